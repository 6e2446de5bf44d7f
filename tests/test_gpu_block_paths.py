"""The block operators' variants on inputs that make each workgroup take several turns, and
the expert layer's own choice of experts."""
import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import (layer_norm_bwd, layer_norm_fwd, linear_act, moe_experts,
                                          moe_layer, moe_route)
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
TD = ref.TYPES


# ---------------------------------------------------------------------------
# Layer norm: more rows than workgroups take in one turn
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(700, 8200), (700, 12001), (700, 16384), (700, 16391), (2500, 4099), (2500, 8191),
                                       (5000, 2041), (9000, 1000), (9000, 333)])
@pytest.mark.parametrize("dt,wt", [("bf16", "f32"), ("f16", "f32"), ("f32", "f32")])
def test_layer_norm_several_rows_a_workgroup(rows, cols, dt, wt):
    say(f"[norm rows] {rows} x {cols} {dt} {wt}")
    g = torch.Generator(device=DEV).manual_seed(cols)
    x = (torch.randn(rows, cols, generator=g, device=DEV) * 2 + 0.5).to(TD[dt])
    gy = torch.randn(rows, cols, generator=g, device=DEV).to(TD[dt])
    w, b = (torch.randn(cols, generator=g, device=DEV).to(TD[wt]) for _ in range(2))
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    y = layer_norm_fwd(x, w, b, torch.empty_like(x), mean, rstd)
    gx, gw, gb = layer_norm_bwd(gy, x, w, mean, rstd, torch.empty_like(x), torch.empty_like(w), torch.empty_like(b))
    # every row of the forward pass and of grad_x, and all rows' sums
    (vy, by), (vm, bm), (vr, br) = ref.layer_norm(x.cpu().double(), w.cpu().double(), b.cpu().double(), 1e-5, TD[dt])
    ref.check(y, vy, by, "y")
    ref.check(mean, vm, bm, "mean")
    ref.check(rstd, vr, br, "rstd")
    grads = ref.layer_norm_grads(gy.cpu().double(), x.cpu().double(), w.cpu().double(), mean.cpu().double(),
                                 rstd.cpu().double(), TD[dt], TD[wt])
    for got, (v, bound), name in zip((gx, gw, gb), grads, ("grad_x", "grad_weight", "grad_bias")):
        ref.check(got, v, bound, name)


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m,n,k", [(4090, 4088, 1032), (3100, 4104, 520), (6720, 1408, 776), (1500, 2056, 2056)])
def test_large_tiles_many_steps(m, n, k):
    """Every tile size and height over many steps of k; the 64-bit product runs on the GPU."""
    say(f"[linear] m {m} n {n} k {k}")
    g = torch.Generator(device=DEV).manual_seed(m)
    for dt, act in (("bf16", "gelu"), ("f16", "squared_relu")):
        x, w = (torch.randn(s, k, generator=g, device=DEV).to(TD[dt]) for s in (m, n))
        w *= 0.03125
        b, r = torch.randn(n, generator=g, device=DEV).to(TD[dt]), torch.randn(m, n, generator=g, device=DEV).to(TD[dt])
        y = linear_act(x, w, torch.empty_like(r), bias=b, activation=act, residual=r)
        v, bound, _ = ref.linear_act(x.double(), w.double(), b.double(), act, r.double(), TD[dt])
        ref.check(y, v.cpu(), bound.cpu(), f"linear {m}x{n}x{k} {dt}")


@pytest.mark.parametrize("m,k", [(4, 96), (100, 96), (40, 4096)])
def test_infinite_row_of_x(m, k):
    """An infinity in a row of x makes every column of its row of y an infinity or NaN."""
    g = torch.Generator(device=DEV).manual_seed(m)
    x, w = torch.randn(m, k, generator=g, device=DEV).to(BF), torch.randn(64, k, generator=g, device=DEV).to(BF)
    x[2, k - 1] = float("inf")
    y = linear_act(x, w, torch.empty(m, 64, dtype=BF, device=DEV))
    assert torch.equal(y[2], torch.where(w[:, k - 1] > 0, float("inf"), float("-inf")).to(BF))
    assert torch.isfinite(y[:2]).all() and torch.isfinite(y[3:]).all()


# ---------------------------------------------------------------------------
# The expert layer that chooses for itself (a few tokens, up to 64 experts, small grids)
# ---------------------------------------------------------------------------
def _layer(x, router, wu, wd, top_k, dtype, **kw):
    """moe_layer, and moe_route with moe_experts: (ids, probs, y) of each. Rows are 7 before."""
    tokens = len(x)
    got = []
    for whole in (True, False):
        ids = torch.full((tokens, top_k), 7, dtype=torch.int32, device=DEV)
        probs = torch.full((tokens, top_k), 7.0, device=DEV)
        y = torch.full((tokens, wd.shape[1]), 7.0, dtype=dtype, device=DEV)
        renorm, valid = kw["renormalize"], kw.get("valid_tokens")
        if whole:
            moe_layer(x, router, wu, wd, y, ids, probs, **kw)
        else:
            moe_route(x, router, ids, probs, renormalize=renorm, valid_tokens=valid)
            rest = {k: v for k, v in kw.items() if k != "renormalize"}
            moe_experts(x, wu, wd, ids, probs, y, **rest)
        got.append((ids, probs, y))
    return got


def _same(a, b):
    # bits, so that NaN counts as itself
    return all(torch.equal(p.view(torch.int16 if p.dtype == BF else torch.int32),
                           q.view(torch.int16 if q.dtype == BF else torch.int32)) for p, q in zip(a, b))


@pytest.mark.parametrize("tokens", [1, 2, 3, 4])
@pytest.mark.parametrize("experts,top_k,inter", [(8, 4, 136), (6, 6, 72), (64, 8, 40), (64, 64, 24), (1, 1, 264), (33, 2, 8)])
def test_choice_inside_the_layer(tokens, experts, top_k, inter):
    say(f"[choice] {tokens} tokens, {experts} experts, top {top_k}, inter {inter}")
    hidden = 264
    g = torch.Generator(device=DEV).manual_seed(tokens + experts)
    x = torch.randn(tokens, hidden, generator=g, device=DEV).to(BF)
    r = torch.randn(tokens, hidden, generator=g, device=DEV).to(BF)
    for rdt, dtype, act, renorm in ((BF, BF, "swiglu", True), (torch.float32, torch.float32, "squared_relu", False),
                                    (torch.float32, BF, "squared_relu", True), (BF, torch.float32, "swiglu", False)):
        router = (torch.randn(experts, hidden, generator=g, device=DEV) * hidden ** -0.5).to(rdt)
        wu = torch.randn(experts, 2 * inter if act == "swiglu" else inter, hidden, generator=g, device=DEV).to(BF) * 0.125
        wd = torch.randn(experts, hidden, inter, generator=g, device=DEV).to(BF) * 0.125
        kw = dict(activation=act, limit=7.0, renormalize=renorm, residual=r)
        one, two = _layer(x, router, wu, wd, top_k, dtype, **kw)
        assert _same(one, two)
        want, (p, bound) = ref.route(x.cpu().double(), router.cpu().double(), top_k, renorm)
        assert torch.equal(one[0].cpu(), want)
        ref.check(one[1], p, bound, "probs")
        v, bound = ref.experts(x.cpu().double(), wu.cpu().double(), wd.cpu().double(), want, one[1].cpu().double(), act, 7.0,
                               r.cpu().double(), dtype)
        ref.check(one[2], v, bound, "layer")
        # equal logits, a token that is NaN, one that is zero
        x2, router2 = x.clone(), router.clone()
        router2[experts // 2:] = router2[:experts - experts // 2].clone()
        x2[tokens // 2, 5] = float("nan")
        x2[0, :] = 0
        one, two = _layer(x2, router2, wu, wd, top_k, dtype, **kw)
        assert _same(one, two)
        if tokens > 1:
            assert one[0][0].tolist() == list(range(top_k)) and one[0][tokens // 2].tolist() == list(range(top_k))
            assert torch.isnan(one[1][tokens // 2]).all()
        for n in range(-1, tokens + 2):
            valid = torch.tensor([n], dtype=torch.int32, device=DEV)
            some, apart = _layer(x, router, wu, wd, top_k, dtype, valid_tokens=valid, **kw)
            assert _same(some, apart)
            n = min(max(n, 0), tokens)
            whole = _layer(x, router, wu, wd, top_k, dtype, **kw)[0]
            for a, b in zip(some, whole):
                assert torch.equal(a[:n], b[:n]) and (a[n:] == 7).all()


def test_layer_with_fp32_router_and_output():
    """The same where the choice has a kernel of its own."""
    hidden, inter, experts, top_k, tokens = 520, 264, 100, 6, 30
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g, device=DEV).to(BF)
    router = torch.randn(experts, hidden, generator=g, device=DEV) * hidden ** -0.5
    wu = torch.randn(experts, 2 * inter, hidden, generator=g, device=DEV).to(BF) * 0.125
    wd = torch.randn(experts, hidden, inter, generator=g, device=DEV).to(BF) * 0.125
    one, two = _layer(x, router, wu, wd, top_k, torch.float32, activation="swiglu", limit=7.0, renormalize=True)
    assert _same(one, two)
    want, (p, bound) = ref.route(x.cpu().double(), router.cpu().double(), top_k, True)
    assert torch.equal(one[0].cpu(), want)
    ref.check(one[1], p, bound, "probs")
    v, bound = ref.experts(x.cpu().double(), wu.cpu().double(), wd.cpu().double(), want, one[1].cpu().double(), "swiglu", 7.0,
                           None, torch.float32)
    ref.check(one[2], v, bound, "layer")
