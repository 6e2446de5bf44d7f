"""Weights to 4 bits, packed, and read back, against their definition (gated_reference): every
output is a whole number or exact, so they are equal."""
import pytest
import torch

import gated_reference as gated
from memory_bound_elementwise_amd import MoeBlockError, fp4_dequantize, fp4_pack, fp4_quantize, fp4_shapes
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = [torch.bfloat16, torch.float16, torch.float32]


def _empty(lead, n, k, fill=165):
    """Codes and scales with a guard on both sides."""
    out = []
    for shape in fp4_shapes(n, k):
        size = torch.Size((*lead, *shape)).numel()
        whole = torch.full((size + 128,), fill, dtype=torch.uint8, device=DEV)
        out.append((whole, whole[64:-64].view(*lead, *shape)))
    return out


def _guards_hold(*pairs):
    torch.cuda.synchronize()
    for whole, _ in pairs:
        assert (whole[:64] == 165).all() and (whole[-64:] == 165).all()


def _quantize(w):
    (c0, codes), (s0, scales) = _empty(w.shape[:-2], *w.shape[-2:])
    fp4_quantize(w.to(DEV), codes, scales)
    _guards_hold((c0, codes), (s0, scales))
    return codes, scales


def _values(codes, scales, shape):
    n = torch.Size(shape).numel()
    whole = torch.full((n + 16,), 77.0, dtype=torch.bfloat16, device=DEV)
    out = fp4_dequantize(codes, scales, whole[8:-8].view(shape))
    torch.cuda.synchronize()
    assert (whole[:8] == 77).all() and (whole[-8:] == 77).all()
    return out.cpu().double()


def _same(a, b):
    nan = torch.isnan(b)
    assert torch.equal(torch.isnan(a), nan)
    assert torch.equal(a[~nan], b[~nan]) and torch.equal(torch.signbit(a[~nan]), torch.signbit(b[~nan]))


def _check(w):
    codes, scales = _quantize(w)
    ref_codes, ref_bytes = gated.quantize(w)
    flat_c, flat_b = ref_codes.view(-1, *w.shape[-2:]), ref_bytes.view(-1, w.shape[-2], w.shape[-1] // 32)
    bad = flat_b == 255                                     # a group of NaN: only its byte counts
    laid = [gated.lay_out(c, b) for c, b in zip(flat_c, flat_b)]
    assert torch.equal(scales.cpu().view(-1, *scales.shape[-3:]), torch.stack([s for _, s in laid]))
    if not bad.any():
        assert torch.equal(codes.cpu().view(-1, *codes.shape[-3:]), torch.stack([c for c, _ in laid]))
    _same(_values(codes, scales, w.shape), gated.values(ref_codes, ref_bytes))


@pytest.mark.parametrize("n,k", [(1, 32), (15, 64), (16, 128), (17, 160), (40, 96), (33, 1056), (64, 384)])
@pytest.mark.parametrize("kind", KINDS)
def test_sizes(n, k, kind):
    say(f"[fp4] {n} x {k} {kind}")
    g = torch.Generator().manual_seed(n + k)
    _check(torch.randn(n, k, generator=g).to(kind))
    _check((torch.randn(3, n, k, generator=g) * 0.02).to(kind))


@pytest.mark.parametrize("kind", KINDS)
def test_borders(kind):
    """Every middle between two elements and its neighbours in the type, groups whose largest is at
    the border of two powers, both signs, zeros of both signs."""
    steps = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.5]).to(kind)
    up = torch.nextafter(steps, torch.full_like(steps, 9))
    down = torch.nextafter(steps, torch.full_like(steps, -9))
    rows = []
    for v in (steps, up, down):
        for top in (4.0, 6.0, 6.96875, 7.0, 3.5, 3.484375, 8.0):
            for sign in (1, -1):
                row = torch.cat((v * sign, v * -sign))
                row[0] = top * sign
                rows.append(row)
    w = torch.stack(rows).to(kind)
    zeros = torch.zeros(2, 32, dtype=kind)
    zeros[1] = -zeros[1]
    w = torch.cat((w, zeros))
    for e in (0, -3, 4) + ((-100, 100) if kind is not torch.float16 else ()):
        _check(w * 2.0 ** e)


def test_range_and_not_finite():
    """The smallest and largest weights of each type; groups with an infinity or a NaN."""
    for kind in KINDS:
        f = torch.finfo(kind)
        w = torch.randn(12, 64, generator=torch.Generator().manual_seed(1)).to(kind)
        w[0, :32] = f.max
        w[1, :32] = -f.max
        w[2, :32] *= f.tiny
        w[3, :32] = f.smallest_normal * f.eps if kind is not torch.float16 else 2.0 ** -24   # the least subnormal
        w[4, 5] = float("inf")
        w[5, 40] = float("nan")
        w[6, 33] = float("-inf")
        w[7] = f.max * torch.linspace(-1, 1, 64).to(kind)
        _check(w)


def test_every_code_and_scale():
    """pack and read back: every element with every byte, past bf16's range and NaN too."""
    codes = torch.arange(16, dtype=torch.uint8).repeat(256, 4)[:, :64]
    codes[:, 32:] = codes[:, 32:].flip(1)
    exponents = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 2)
    exponents[:, 1] = exponents[:, 1].flip(0)
    (c0, c), (s0, s) = _empty((), 256, 64)
    fp4_pack(gated.pairs(codes).to(DEV), exponents.to(DEV), c, s)
    _guards_hold((c0, c), (s0, s))
    want = gated.lay_out(codes, exponents)
    assert torch.equal(c.cpu(), want[0]) and torch.equal(s.cpu(), want[1])
    _same(_values(c, s, (256, 64)), gated.values(codes, exponents))


@pytest.mark.parametrize("lead,n,k", [((), 5, 32), ((3,), 40, 416), ((2,), 16, 128)])
def test_pack(lead, n, k):
    g = torch.Generator().manual_seed(n)
    codes = torch.randint(0, 16, (*lead, n, k), generator=g, dtype=torch.uint8)
    exponents = torch.randint(100, 150, (*lead, n, k // 32), generator=g, dtype=torch.uint8)
    (c0, c), (s0, s) = _empty(lead, n, k)
    fp4_pack(gated.pairs(codes).contiguous().to(DEV), exponents.to(DEV), c, s)
    _guards_hold((c0, c), (s0, s))
    laid = [gated.lay_out(a, b) for a, b in zip(codes.view(-1, n, k), exponents.view(-1, n, k // 32))]
    assert torch.equal(c.cpu().view(-1, *c.shape[-3:]), torch.stack([a for a, _ in laid]))
    assert torch.equal(s.cpu().view(-1, *s.shape[-3:]), torch.stack([b for _, b in laid]))
    _same(_values(c, s, (*lead, n, k)), gated.values(codes, exponents))


def test_error_bound():
    """|w - value| <= half the distance between the elements around it."""
    w = torch.randn(64, 512, generator=torch.Generator().manual_seed(2))
    codes, scales = _quantize(w)
    v = _values(codes, scales, w.shape)
    _, byte = gated.quantize(w)
    unit = 2.0 ** (byte.double() - 127).repeat_interleave(32, 1)
    a = w.double().abs() / unit
    assert (a < 7).all()
    half = torch.where(a <= 2, 0.25, torch.where(a <= 4, 0.5, 1.0)) * unit
    assert ((w.double() - v).abs() <= half).all()


def test_past_4_gib():
    """Offsets beyond 32 bits on both sides: the last matrix of a stack of 4.6 GB."""
    say("[fp4] 5 matrices of 16384 x 28032")
    n, k = 16384, 28032
    w = torch.zeros(5, n, k, dtype=torch.bfloat16, device=DEV)
    last = torch.randn(64, k, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    w[4, -64:] = last.to(DEV)
    codes, scales = (torch.empty(5, *s, dtype=torch.uint8, device=DEV) for s in fp4_shapes(n, k))
    fp4_quantize(w, codes, scales)
    ref = gated.lay_out(*gated.quantize(last))
    assert torch.equal(codes[4, -4:].cpu(), ref[0]) and torch.equal(scales[4, -4:].cpu(), ref[1])
    w.fill_(3)
    fp4_dequantize(codes, scales, w)
    assert torch.equal(w[4, -64:].cpu().double(), gated.values(*gated.quantize(last)))
    assert not w[:4].any() and not w[4, :-64].any()


def test_streams_capture_and_refusals():
    w = torch.randn(40, 256, device=DEV).to(torch.bfloat16)
    codes, scales = _quantize(w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    s.wait_stream(torch.cuda.current_stream())
    fp4_quantize(w, c2, s2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(w)
    with torch.cuda.graph(graph):
        fp4_quantize(w, c2, s2)
        fp4_dequantize(c2, s2, out)
    for _ in range(3):
        w.mul_(-0.7)
        graph.replay()
        torch.cuda.synchronize()
        codes, scales = _quantize(w)
        assert torch.equal(c2, codes) and torch.equal(out, fp4_dequantize(codes, scales, torch.empty_like(w)))
    with pytest.raises(ValueError):                          # k not a multiple of 32
        fp4_quantize(w[:, :40].contiguous(), codes, scales)
    with pytest.raises(ValueError):
        fp4_quantize(w, codes[:1], scales)
    with pytest.raises(ValueError):
        fp4_quantize(w.t(), codes, scales)
    with pytest.raises(TypeError):
        fp4_dequantize(codes, scales, w.float())
    with pytest.raises(TypeError):
        fp4_quantize(w, codes.view(torch.int8), scales)
    with pytest.raises(MoeBlockError):                       # scales over the codes
        fp4_quantize(w, codes, codes.view(-1)[:scales.numel()].view(scales.shape))
