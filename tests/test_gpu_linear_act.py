"""The matrix product with bias, activation and residual against 64 bits (block_reference)."""
import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import MoeBlockError, linear_act, linear_act_workspace
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ACTS = ["none", "silu", "gelu", "squared_relu"]


def _inputs(m, n, k, dt, seed, bias=True, residual=True):
    g = torch.Generator().manual_seed(seed)
    t = ref.TYPES[dt]
    x = torch.randn(m, k, generator=g).to(t)
    w = (torch.randn(n, k, generator=g) * (2 / k ** 0.5)).to(t)
    b = torch.randn(n, generator=g).to(t) if bias else None
    r = torch.randn(m, n, generator=g).to(t) if residual else None
    return x, w, b, r


def _run(x, w, b, r, act, **kw):
    dev = [None if t is None else t.to(DEV) for t in (x, w, b, r)]
    # rows before and after y must stay as they are
    whole = torch.full((x.shape[0] + 2, w.shape[0]), 77.0, dtype=x.dtype, device=DEV)
    y = linear_act(dev[0], dev[1], whole[1:-1], bias=dev[2], activation=act, residual=dev[3], **kw)
    torch.cuda.synchronize()
    assert (whole[0] == 77).all() and (whole[-1] == 77).all()
    return y


def _check(m, n, k, dt, act, bias=True, residual=True):
    say(f"[linear] m {m} n {n} k {k} {dt} {act} bias {bias} residual {residual}")
    x, w, b, r = _inputs(m, n, k, dt, m + 3 * n + 7 * k, bias, residual)
    y = _run(x, w, b, r, act)
    wide = [None if t is None else t.double() for t in (x, w, b)]
    v, bound, _ = ref.linear_act(*wide, act, None if r is None else r.double(), x.dtype)
    ref.check(y, v, bound, f"linear {m}x{n}x{k} {dt} {act}")


# rows on both sides of every variant's border; n and k that end inside a tile or a step
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 127, 129, 255, 257, 300])
@pytest.mark.parametrize("n,k", [(8, 8), (24, 40), (264, 136), (128, 256), (520, 1032)])
def test_shapes(m, n, k):
    _check(m, n, k, "bf16" if (m + n) % 2 else "f16", ACTS[(m + k) % 4])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("m", [3, 70])
def test_activations_bias_residual(m, dt, act):
    for bias, residual in ((True, True), (True, False), (False, True), (False, False)):
        _check(m, 136, 200, dt, act, bias, residual)


@pytest.mark.parametrize("m,n,k", [(1, 64, 7168), (40, 72, 4096), (96, 64, 7168), (600, 520, 1408), (200, 2056, 64)])
def test_long_and_wide(m, n, k):
    _check(m, n, k, "bf16", "silu")
    _check(m, n, k, "f16", "none")


@pytest.mark.parametrize("m", [4, 100])
def test_infinities_and_nan_stay_in_their_rows(m):
    """A non-finite row of x reaches its own row of y, one of W its own column."""
    x, w, b, r = _inputs(m, 64, 96, "bf16", 1)
    clean = _run(x, w, b, r, "silu")
    x2, w2 = x.clone(), w.clone()
    x2[1, 5] = float("nan")
    x2[2, 95] = float("inf")
    w2[17, 3] = float("nan")
    y = _run(x2, w2, b, r, "silu")
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 17]).all()
    assert not torch.isfinite(y[2]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1:3] = False
    keep[:, 17] = False
    assert torch.equal(y[keep], clean[keep])


def test_overflow_to_infinity():
    """A value past the type's range rounds to infinity."""
    x, w = torch.full((2, 64), 200.0, dtype=torch.float16), torch.full((8, 64), 20.0, dtype=torch.float16)
    for m in (2, 80):
        y = _run(x[:1].expand(m, 64).contiguous(), w, None, None, "none")   # 256000
        assert torch.isinf(y).all()


def test_no_rows_and_refusals():
    x, w, b, r = [t.to(DEV) for t in _inputs(2, 16, 24, "bf16", 1)]
    y = torch.empty_like(r)
    linear_act(x[:0], w, y[:0])
    with pytest.raises(MoeBlockError):               # y over the residual
        linear_act(x, w, r, residual=r)
    with pytest.raises(MoeBlockError):               # k not a multiple of 8
        linear_act(x[:, :20].contiguous(), w[:, :20].contiguous(), y)
    with pytest.raises(ValueError):
        linear_act(x, w.t(), y)
    with pytest.raises(RuntimeError):
        linear_act(x.requires_grad_(), w, y)


def test_same_bits_streams_and_capture():
    """Every replay of a captured call, and calls at once on two streams with a workspace each,
    give the eager call's bits."""
    for m, n, k in ((5, 520, 2048), (70, 136, 4096), (500, 264, 512)):
        x, w, b, r = [t.to(DEV) for t in _inputs(m, n, k, "bf16", m)]
        want = linear_act(x, w, torch.empty_like(r), bias=b, activation="gelu", residual=r)
        need = linear_act_workspace(m, n, k)
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
            for _ in range(3):
                y = torch.empty_like(r)
                s.wait_stream(torch.cuda.current_stream())
                linear_act(x, w, y, bias=b, activation="gelu", residual=r, stream=s, workspace=ws)
                outs.append(y)
        torch.cuda.synchronize()
        for y in outs:
            assert torch.equal(y.view(torch.int16), want.view(torch.int16))
        y = torch.empty_like(r)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            linear_act(x, w, y, bias=b, activation="gelu", residual=r)
        for i in range(3):
            x.mul_(0.5)
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            again = linear_act(x, w, torch.empty_like(r), bias=b, activation="gelu", residual=r)
            assert torch.equal(y.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("m,n,k", [(4090, 4088, 72), (3100, 4104, 136), (4600, 4096, 40), (1500, 2056, 200), (6720, 1408, 24)])
def test_many_tiles(m, n, k):
    """Enough tiles for every tile size and height, ragged on every side; the 64-bit product
    runs on the GPU (float64 matmul)."""
    say(f"[linear] m {m} n {n} k {k}")
    for dt, act in (("bf16", "silu"), ("f16", "none")):
        x, w, b, r = _inputs(m, n, k, dt, m)
        y = _run(x, w, b, r, act)
        wide = [t.to(DEV).double() for t in (x, w, b, r)]
        v, bound, _ = ref.linear_act(wide[0], wide[1], wide[2], act, wide[3], x.dtype)
        ref.check(y, v.cpu(), bound.cpu(), f"linear {m}x{n}x{k} {dt} {act}")
