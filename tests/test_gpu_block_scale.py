"""The block operators past 32-bit offsets, and an autograd capture that is refused."""
import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import LayerNorm, layer_norm_bwd, layer_norm_fwd, linear_act, moe_experts
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.mark.parametrize("cols", [7168, 7169])
def test_layer_norm_past_4_gib(cols):
    rows = (1 << 32) // (2 * cols) + 5
    say(f"[scale] layer norm {rows} x {cols}")
    x = torch.zeros(rows, cols, dtype=BF, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    pick = [0, rows // 2, rows - 2, rows - 1]
    for r in pick:
        x[r] = torch.randn(cols, generator=g, device=DEV).to(BF)
    w = torch.randn(cols, generator=g, device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    y = layer_norm_fwd(x, w, w, torch.empty_like(x), mean, rstd)
    wide = x[pick].cpu().double(), w.cpu().double()
    (v, bound), _, _ = ref.layer_norm(wide[0], wide[1], wide[1], 1e-5, BF)
    ref.check(y[pick], v, bound, "y")
    gy = y.zero_()                                    # only these rows have a gradient
    for r in pick:
        gy[r] = torch.randn(cols, generator=g, device=DEV).to(BF)
    gx, gw, gb = layer_norm_bwd(gy, x, w, mean, rstd, torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))
    v = ref.layer_norm_grads(gy[pick].cpu().double(), wide[0], wide[1], mean[pick].cpu().double(),
                             rstd[pick].cpu().double(), BF, torch.float32)
    ref.check(gx[pick], *v[0], "grad_x")
    # the other rows add zeros: no term of the bound but these rows'
    ref.check(gw, *v[1], "grad_weight")
    ref.check(gb, *v[2], "grad_bias")
    assert not gx[1:rows // 2].any()


def test_linear_past_4_gib():
    m, n, k = 530000, 4104, 8
    say(f"[scale] linear {m} x {n} x {k}")
    g = torch.Generator(device=DEV).manual_seed(2)
    x, w = torch.randn(m, k, generator=g, device=DEV).to(BF), torch.randn(n, k, generator=g, device=DEV).to(BF)
    r = torch.zeros(m, n, dtype=BF, device=DEV)
    r[-300:] = 1.0
    y = linear_act(x, w, torch.empty(m, n, dtype=BF, device=DEV), residual=r)
    for rows in (slice(0, 300), slice(m // 2, m // 2 + 300), slice(m - 300, m)):
        v, bound, _ = ref.linear_act(x[rows].cpu().double(), w.cpu().double(), None, None, r[rows].cpu().double(), BF)
        ref.check(y[rows], v, bound, f"rows {rows}")


@pytest.mark.parametrize("tokens", [1, 40])
def test_experts_past_4_gib(tokens):
    hidden, inter, experts = 7168, 2048, 90           # 5.3 GB of w_up
    say(f"[scale] experts {tokens} tokens")
    g = torch.Generator(device=DEV).manual_seed(3)
    wu = torch.zeros(experts, 2 * inter, hidden, dtype=BF, device=DEV)
    wd = torch.zeros(experts, hidden, inter, dtype=BF, device=DEV)
    wu[-1] = (torch.randn(2 * inter, hidden, generator=g, device=DEV) * 0.02).to(BF)
    wd[-1] = (torch.randn(hidden, inter, generator=g, device=DEV) * 0.02).to(BF)
    x = torch.randn(tokens, hidden, generator=g, device=DEV).to(BF)
    ids = torch.zeros(tokens, 4, dtype=torch.int32, device=DEV)
    ids[:, 2] = experts - 1
    probs = torch.rand(tokens, 4, generator=g, device=DEV)
    y = moe_experts(x, wu, wd, ids, probs, torch.empty_like(x), limit=7.0)
    few = slice(0, min(tokens, 3))
    v, bound = ref.experts(x[few].cpu().double(), wu[-1:].cpu().double(), wd[-1:].cpu().double(),
                           torch.zeros(len(x[few]), 1, dtype=torch.int32), probs[few, 2:3].cpu().double(), "swiglu", 7.0,
                           None, BF)
    ref.check(y[few], v, bound, "last expert")


def test_captured_autograd_is_refused():
    """An autograd backward into leaves during a capture raises, with an eager graph of the same
    leaves alive, and leaves the process able to go on; the direct calls can be captured
    (test_gpu_layer_norm)."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(200, 520, generator=g).to(BF).to(DEV).requires_grad_()
    w = torch.randn(520, generator=g).to(DEV).requires_grad_()
    gy = torch.randn(200, 520, generator=g).to(BF).to(DEV)
    eager = LayerNorm.apply(x, w, None, 1e-5)         # stays alive over the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(graph):
            torch.autograd.grad(LayerNorm.apply(x, w, None, 1e-5), (x, w), gy)
    torch.cuda.synchronize()
    first = torch.autograd.grad(eager, (x, w), gy)
    again = torch.autograd.grad(LayerNorm.apply(x, w, None, 1e-5), (x, w), gy)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
