"""Layer norm, forward and backward, against 64 bits (block_reference), through the public
entry points."""
import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import LayerNorm, layer_norm_bwd, layer_norm_bwd_workspace, layer_norm_fwd
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TD = ref.TYPES


def _rows(rows, cols, dt, seed, offset=0.5, std=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std + offset
    return x.to(TD[dt])


def _weights(cols, wt, seed):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn(cols, generator=g) * 0.3 + 1).to(TD[wt]), (torch.randn(cols, generator=g) * 0.3).to(TD[wt]))


def _fwd(x, w, b, eps=1e-5, stats=True):
    dev = [None if t is None else t.to(DEV) for t in (x, w, b)]
    y = torch.full_like(dev[0], 77.0)
    mean = torch.full((x.shape[0],), 77.0, device=DEV) if stats else None
    rstd = torch.full_like(mean, 77.0) if stats else None
    layer_norm_fwd(*dev, y, mean, rstd, eps=eps)
    torch.cuda.synchronize()
    return y, mean, rstd


def _check_fwd(x, w, b, dt, eps=1e-5):
    y, mean, rstd = _fwd(x, w, b, eps)
    wide = [None if t is None else t.double() for t in (x, w, b)]
    (vy, by), (vm, bm), (vr, br) = ref.layer_norm(*wide, eps, TD[dt])
    ref.check(mean, vm, bm, "mean")
    ref.check(rstd, vr, br, "rstd")
    ref.check(y, vy, by, "y")


# widths on both sides of every variant's border, odd ones and ones that end inside a group of eight
WIDTHS = [1, 2, 7, 8, 63, 512, 513, 1000, 1024, 1411, 2048, 2049, 4096, 4099, 7168, 8192, 8200, 16384, 16391, 40007]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dt,wt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
def test_forward(dt, wt, cols):
    w, b = _weights(cols, wt, cols)
    for rows in (1, 5):
        _check_fwd(_rows(rows, cols, dt, cols + rows), w, b, dt)


@pytest.mark.parametrize("rows", [2, 3, 4, 257, 1030])
@pytest.mark.parametrize("cols", [24, 1411, 4096])
def test_forward_many_rows(rows, cols):
    w, b = _weights(cols, "f32", 3)
    _check_fwd(_rows(rows, cols, "bf16", rows), w, b, "bf16")


@pytest.mark.parametrize("cols", [9, 7168, 20000])
def test_forward_without_weight_bias_or_statistics(cols):
    x = _rows(3, cols, "bf16", 1)
    w, b = _weights(cols, "bf16", 2)
    for ww, bb in ((None, None), (w, None), (None, b)):
        _check_fwd(x, ww, bb, "bf16")
    y, _, _ = _fwd(x, w, b, stats=False)
    assert torch.equal(y.view(torch.int16), _fwd(x, w, b)[0].view(torch.int16))


def test_forward_offset_rows_constant_rows_and_specials():
    """A large common offset, a constant row (its variance is 0, so eps decides), rows with an
    infinity or a NaN (the whole row is NaN, its neighbours are not)."""
    x = _rows(8, 1000, "f32", 5)
    x[1] += 4096.0
    x[2] = 3.25
    x[3, 17] = float("inf")
    x[4, 999] = float("nan")
    x[5] = 0.0
    w, b = _weights(1000, "f32", 6)
    y, mean, rstd = _fwd(x, w, b)
    fine = [0, 1, 2, 5, 6, 7]
    (vy, by), _, _ = ref.layer_norm(x[fine].double(), w.double(), b.double(), 1e-5, torch.float32)
    ref.check(y[fine], vy, by, "finite rows")
    assert torch.isnan(y[[3, 4]]).all() and torch.isnan(rstd[[3, 4]]).all()
    assert torch.equal(y[2].cpu(), b) and torch.equal(y[5].cpu(), b)
    y, _, _ = _fwd(x[[2]], w, b, eps=0.0)           # 0 / 0, as the formula has it
    assert torch.isnan(y).all()


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dt,wt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_backward(dt, wt, cols):
    for rows in (1, 6):
        _check_bwd(rows, cols, dt, wt)


def _check_bwd(rows, cols, dt, wt, want=(True, True, True), weight=True):
    say(f"[norm bwd] {rows} x {cols} {dt} {wt}")
    x, gy = _rows(rows, cols, dt, cols + rows), _rows(rows, cols, dt, cols + rows + 1, 0.1, 1.0)
    w = _weights(cols, wt, cols)[0] if weight else None
    wide = x.double()
    mean = wide.mean(1).float()
    rstd = (1 / torch.sqrt(wide.var(1, unbiased=False) + 1e-5)).float()
    out = [torch.full_like(x, 77.0, device=DEV), torch.full((cols,), 77.0, dtype=TD[wt], device=DEV),
           torch.full((cols,), 77.0, dtype=TD[wt], device=DEV)]
    out = [o if k else None for o, k in zip(out, want)]
    layer_norm_bwd(gy.to(DEV), x.to(DEV), None if w is None else w.to(DEV), mean.to(DEV), rstd.to(DEV), *out)
    torch.cuda.synchronize()
    values = ref.layer_norm_grads(gy.double(), wide, None if w is None else w.double(), mean.double(), rstd.double(),
                                  TD[dt], TD[wt])
    for o, (v, bound), name in zip(out, values, ("grad_x", "grad_weight", "grad_bias")):
        if o is not None:
            ref.check(o, v, bound, f"{name} {rows}x{cols} {dt} {wt}")
    return out


@pytest.mark.parametrize("rows", [2, 15, 16, 17, 255, 256, 257, 4100])
@pytest.mark.parametrize("cols", [40, 1000, 2048, 4096])
def test_backward_many_rows(rows, cols):
    _check_bwd(rows, cols, "bf16", "f32")


@pytest.mark.parametrize("cols", [7168, 20000])
def test_backward_many_wide_rows(cols):
    _check_bwd(600, cols, "bf16", "bf16")


@pytest.mark.parametrize("cols", [100, 7168, 17000])
@pytest.mark.parametrize("want", [(True, False, False), (False, True, True), (False, False, True), (True, True, False)])
def test_backward_of_some_outputs(cols, want):
    _check_bwd(19, cols, "bf16", "f32", want)
    _check_bwd(19, cols, "bf16", "f32", want, weight=False)


def test_no_rows():
    w = torch.ones(64, device=DEV)
    x = torch.empty(0, 64, device=DEV)
    st = torch.empty(0, device=DEV)
    layer_norm_fwd(x, w, w, torch.empty_like(x), st, st.clone())
    gw, gb = torch.full((64,), 5.0, device=DEV), torch.full((64,), 5.0, device=DEV)
    layer_norm_bwd(x, x, w, st, st, torch.empty_like(x), gw, gb)
    torch.cuda.synchronize()
    assert not gw.any() and not gb.any()


@pytest.mark.parametrize("shape", [(3, 5, 40), (7, 1411), (64,)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_autograd(shape, dt):
    g = torch.Generator().manual_seed(9)
    x = torch.randn(shape, generator=g).to(dt).to(DEV).requires_grad_()
    w = (torch.randn(shape[-1], generator=g) + 1).to(DEV).requires_grad_()
    b = torch.randn(shape[-1], generator=g).to(DEV).requires_grad_()
    gy = torch.randn(shape, generator=g).to(dt).to(DEV)
    LayerNorm.apply(x, w, b, 1e-5).backward(gy)
    leaves = [t.detach().cpu().double().requires_grad_() for t in (x, w, b)]
    xx, ww, bb = leaves
    c = xx - xx.mean(-1, keepdim=True)
    (c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * ww + bb).backward(gy.cpu().double())
    flat = [t.reshape(-1, shape[-1]) for t in (gy.cpu().double(), xx.detach())]
    mean = flat[1].mean(1)
    rstd = 1 / torch.sqrt(flat[1].var(1, unbiased=False) + 1e-5)
    bounds = ref.layer_norm_grads(*flat, ww.detach(), mean, rstd, dt, torch.float32)
    # the statistics are the kernel's own here: each off by at most 2^6 u relative, which moves
    # every term of the gradients by at most 2^9 u of the row's largest
    slack = 2.0 ** 9 * ref.U
    for t, leaf, (_, bound) in zip((x, w, b), leaves, bounds):
        s = slack * leaf.grad.abs().max() * 4
        ref.check(t.grad, leaf.grad, bound.reshape(leaf.shape) + s, "autograd")


def test_backward_against_differences():
    """Central differences of the 64-bit forward, on the kernel's fp32 gradient."""
    g = torch.Generator().manual_seed(2)
    x, w, b, gy = (torch.randn(s, generator=g).double() for s in ((2, 11), (11,), (11,), (2, 11)))

    def value(xx, ww, bb):
        c = xx - xx.mean(-1, keepdim=True)
        return ((c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * ww + bb) * gy).sum()

    leaves = [t.float().to(DEV).requires_grad_() for t in (x, w, b)]
    LayerNorm.apply(*leaves).backward(gy.float().to(DEV))
    base = [t.float().double() for t in (x, w, b)]
    for which, leaf in enumerate(leaves):
        got = leaf.grad.cpu().double().reshape(-1)
        for i in range(got.numel()):
            d = []
            for sign in (1, -1):
                moved = [t.clone() for t in base]
                moved[which].reshape(-1)[i] += sign * 1e-5
                d.append(value(*moved))
            # differences: h^2 of the third derivative (values of order 1) and 1e-16 / h
            assert abs((d[0] - d[1]) / 2e-5 - got[i]) < 2e-5


def test_same_bits_and_concurrent_workspaces():
    """The same call gives the same bits; two streams with a workspace each do not disturb one
    another; an explicit stream with tensors of the default one."""
    x, gy = _rows(3000, 2048, "bf16", 1).to(DEV), _rows(3000, 2048, "bf16", 2).to(DEV)
    w = torch.ones(2048, device=DEV)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(3000, device=DEV), torch.empty(3000, device=DEV)
    layer_norm_fwd(x, w, None, y, mean, rstd)
    want = layer_norm_bwd(gy, x, w, mean, rstd, torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    need = layer_norm_bwd_workspace(3000, 2048)
    spaces = [torch.empty(need, dtype=torch.uint8, device=DEV), None]
    outs = []
    for _ in range(3):
        for s, ws in zip(streams, spaces):
            out = (torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))
            s.wait_stream(torch.cuda.current_stream())
            layer_norm_bwd(gy, x, w, mean, rstd, *out, stream=s, workspace=ws)
            outs.append(out)
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_captured_forward_and_backward():
    """A captured pair replayed with new inputs, eager work between the replays."""
    x, gy = _rows(300, 1000, "bf16", 1).to(DEV), _rows(300, 1000, "bf16", 2).to(DEV)
    w = torch.rand(1000, device=DEV)
    y, gx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(300, device=DEV), torch.empty(300, device=DEV)
    gw, gb = torch.empty_like(w), torch.empty_like(w)

    def step():
        layer_norm_fwd(x, w, w, y, mean, rstd)
        layer_norm_bwd(gy, x, w, mean, rstd, gx, gw, gb)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(_rows(300, 1000, "bf16", 10 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, mean, rstd, gx, gw, gb)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, mean, rstd, gx, gw, gb)):
            assert torch.equal(a, b)
