"""Layer norm of rows whose common offset is large against their deviations: the mean is corrected,
so nothing grows with the offset but what the first mean leaves behind, squared."""
import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import layer_norm_fwd
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
WIDTHS = [8, 63, 512, 1000, 1024, 1411, 2048, 3001, 4096, 7168, 8191, 12000, 16384, 16391, 40000]


def _bounds(x, weight, bias, eps, dtype):
    """(value, bound) of y, mean and rstd in 64 bits. u is half a step of fp32, d the depth of a
    row's sum. The first mean mu is off by e <= (d + 2) u mean|x|. The deviations from it, each
    rounded once, are summed for the rest r = mean(x - mu), off by
    c <= (d + 3) u (mean|x - mean| + e), and their squares for var = mean((x - mu)^2) - r^2."""
    u = ref.U
    d = max(32, -(-x.shape[1] // 1024)) + 22
    mean = x.mean(1, keepdim=True)
    dev = x - mean
    var = (dev * dev).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    e = (d + 2) * u * x.abs().mean(1, keepdim=True)
    c = (d + 3) * u * (dev.abs().mean(1, keepdim=True) + e)
    dmean = c + u * (mean.abs() + c)
    # each deviation: rounded at x - mu and at v - r, and r's own error
    ddev = 2 * u * (dev.abs() + e + c) + c
    # squares: v rounded (2 u), the sum (d + 1) and the division, of mean((x - mu)^2) = var + e^2;
    # r^2 with |r| <= e + c; the subtraction and the addition of eps
    dvar = (d + 5) * u * (var + e * e) + 2 * e * c + c * c + u * (e + c) ** 2 + 2 * u * (var + eps)
    low = (var + eps - dvar).clamp(min=1e-300)
    drstd = torch.maximum(1 / torch.sqrt(low) - rstd, rstd - 1 / torch.sqrt(var + eps + dvar)) + 4 * u * rstd
    n = dev * rstd
    dn = ddev * (rstd + drstd) + dev.abs() * drstd + 2 * u * n.abs()
    y = n * weight + bias
    dy = dn * weight.abs() + 2 * u * (y.abs() + (n * weight).abs())
    return ((y, ref.rounded(y, dy, dtype)), (mean[:, 0], dmean[:, 0] + ref.TINY[torch.float32]),
            (rstd[:, 0], drstd[:, 0] + u * rstd[:, 0]))


def _check(x, dt):
    cols = x.shape[1]
    g = torch.Generator().manual_seed(cols)
    w, b = torch.randn(cols, generator=g) + 1, torch.randn(cols, generator=g)
    x = x.to(ref.TYPES[dt])
    mean, rstd = torch.empty(len(x), device=DEV), torch.empty(len(x), device=DEV)
    d = x.to(DEV)
    y = layer_norm_fwd(d, w.to(DEV), b.to(DEV), torch.empty_like(d), mean, rstd)
    vy, vm, vr = _bounds(x.double(), w.double(), b.double(), 1e-5, ref.TYPES[dt])
    ref.check(mean, *vm, "mean")
    ref.check(rstd, *vr, "rstd")
    ref.check(y, *vy, "y")


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_constant_rows(cols, dt):
    """A constant row is its bias, whatever the constant; values whose sums are not exact."""
    say(f"[norm offset] constant, {cols} {dt}")
    value = torch.tensor([0.3, -4097.3, 1000.1, 1.0 / 3, 60000.7, -0.001])
    _check(value[:, None].expand(6, cols).contiguous(), dt)


@pytest.mark.parametrize("cols", WIDTHS)
def test_offsets(cols):
    """Unit deviations on offsets of up to 10^6, of one sign and of both."""
    say(f"[norm offset] {cols} f32")
    g = torch.Generator().manual_seed(cols + 1)
    offset = torch.tensor([1e5, -3e5, 1e6, 777777.7, -1e6, 0.0])
    x = torch.randn(6, cols, generator=g) + offset[:, None]
    _check(x, "f32")
