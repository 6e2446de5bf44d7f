"""The product and the expert layer with weights in 4 bits, against 64 bits (block_reference,
gated_reference)."""
import math

import pytest
import torch

import block_reference as ref
import gated_reference as gated
from memory_bound_elementwise_amd import (MoeBlockError, fp4_pack, fp4_shapes, layer_norm_fwd, linear_act_fp4,
                                          linear_act_fp4_workspace, moe_experts_fp4, moe_experts_fp4_workspace,
                                          moe_gate_fwd, moe_route)
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
ACTS = ["none", "silu", "gelu", "squared_relu"]


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF)


def _weights(g, *shape, std=1.0):
    """Values in 64 bits, and the laid-out codes and scales on the GPU."""
    codes, exponents = gated.quantize(torch.randn(*shape, generator=g) * std)
    return gated.values(codes, exponents), _pack(codes, exponents)


def _pack(codes, exponents):
    lead, (n, k) = codes.shape[:-2], codes.shape[-2:]
    to = [torch.empty(*lead, *s, dtype=torch.uint8, device=DEV) for s in fp4_shapes(n, k)]
    fp4_pack(gated.pairs(codes).contiguous().to(DEV), exponents.contiguous().to(DEV), *to)
    return to


# ---------------------------------------------------------------------------
# Product
# ---------------------------------------------------------------------------
def _linear(x, w, b, r, act, n, **kw):
    whole = torch.full((x.shape[0] + 2, n), 77.0, dtype=BF, device=DEV)
    y = linear_act_fp4(x.to(DEV), *w, whole[1:-1], bias=None if b is None else b.to(DEV), activation=act,
                       residual=None if r is None else r.to(DEV), **kw)
    torch.cuda.synchronize()
    assert (whole[0] == 77).all() and (whole[-1] == 77).all()
    return y


def _check_linear(m, n, k, act, bias=True, residual=True):
    say(f"[linear_fp4] m {m} n {n} k {k} {act} bias {bias} residual {residual}")
    g = torch.Generator().manual_seed(m + 3 * n + 7 * k)
    x = _normal(g, m, k)
    v, w = _weights(g, n, k, std=2 / k ** 0.5)
    b, r = _normal(g, n) if bias else None, _normal(g, m, n) if residual else None
    y = _linear(x, w, b, r, act, n)
    want, bound, _ = ref.linear_act(x.double(), v, None if b is None else b.double(), act,
                                    None if r is None else r.double(), BF)
    ref.check(y, want, bound, f"linear {m}x{n}x{k} {act}")


# rows on both sides of every variant's border; n and k that end inside a tile or a step
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 130])
@pytest.mark.parametrize("n,k", [(8, 32), (24, 64), (264, 160), (128, 256), (520, 1056)])
def test_linear_sizes(m, n, k):
    _check_linear(m, n, k, ACTS[(m + k // 32) % 4])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 20, 70])
def test_linear_epilogue(m, act):
    for bias, residual in ((True, True), (True, False), (False, True), (False, False)):
        _check_linear(m, 136, 224, act, bias, residual)


@pytest.mark.parametrize("m,n,k", [(1, 64, 7168), (1, 16, 16384), (2, 4096, 2048), (5, 2056, 1408), (16, 1040, 4096),
                                   (40, 72, 4096), (64, 264, 7168), (96, 64, 7168), (600, 520, 1408),
                                   (1100, 8200, 288), (600, 4104, 1056), (1009, 2048, 4096), (50, 4104, 160), (1, 16400, 160), (4, 16384, 96), (5, 8200, 288),
                                   (7, 8232, 3104), (16, 8192, 64)])
def test_linear_long_and_wide(m, n, k):
    _check_linear(m, n, k, "silu")


@pytest.mark.parametrize("m,n,k", [(2050, 4088, 160), (2100, 4104, 32), (1030, 8200, 288), (4100, 2056, 1056)])
def test_linear_many_tiles(m, n, k):
    """Enough tiles for the widest ones, ragged on every side; the 64-bit product runs on the GPU
    (float64 matmul)."""
    say(f"[linear_fp4] m {m} n {n} k {k}")
    g = torch.Generator().manual_seed(m)
    x, b, r = _normal(g, m, k), _normal(g, n), _normal(g, m, n)
    v, w = _weights(g, n, k, std=k ** -0.5)
    y = _linear(x, w, b, r, "silu", n)
    want, bound, _ = ref.linear_act(x.to(DEV).double(), v.to(DEV), b.to(DEV).double(), "silu", r.to(DEV).double(), BF)
    ref.check(y, want.cpu(), bound.cpu(), f"linear {m}x{n}x{k}")


def test_linear_scales():
    """Each group by its own scale, exactly: the smallest powers too; a NaN group reaches its own
    column alone."""
    g = torch.Generator().manual_seed(9)
    n, k = 48, 288
    codes = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8)
    exponents = torch.randint(0, 40, (n, k // 32), generator=g, dtype=torch.uint8)
    exponents[5] = 0
    x = (torch.randn(3, k, generator=g) * 2.0 ** 100).to(BF)
    for m in (3, 80):
        xs = x.repeat(27, 1)[:m].contiguous()
        y = _linear(xs, _pack(codes, exponents), None, None, None, n)
        want, bound, _ = ref.linear_act(xs.double(), gated.values(codes, exponents), None, "none", None, BF)
        ref.check(y, want, bound, "scales")
        spoilt = exponents.clone()
        spoilt[17, 2] = 255
        z = _linear(xs, _pack(codes, spoilt), None, None, None, n)
        assert torch.isnan(z[:, 17]).all()
        keep = torch.arange(n) != 17
        assert torch.equal(z[:, keep], y[:, keep])


@pytest.mark.parametrize("m", [4, 20, 100])
def test_linear_not_finite(m):
    """A NaN of x stays in its row; an infinity gives infinities where its weight is not zero."""
    g = torch.Generator().manual_seed(2)
    x, (v, w) = _normal(g, m, 96), _weights(g, 64, 96)
    clean = _linear(x, w, None, None, None, 64)
    x2 = x.clone()
    x2[1, 5], x2[2, 95], x2[3, 40] = float("nan"), float("inf"), float("-inf")
    y = _linear(x2, w, None, None, None, 64).cpu().float()
    assert torch.isnan(y[1]).all()
    for row, k, sign in ((2, 95, 1), (3, 40, -1)):
        s = v[:, k].sign() * sign
        assert torch.isnan(y[row][s == 0]).all() and torch.equal(y[row][s != 0], (s * math.inf).float()[s != 0])
    keep = [i for i in range(m) if i not in (1, 2, 3)]
    assert torch.equal(y[keep], clean.cpu().float()[keep])


def test_linear_rows_do_not_touch():
    """A row's bits do not depend on the other rows of its call."""
    g = torch.Generator().manual_seed(3)
    x, (_, w) = _normal(g, 64, 512), _weights(g, 128, 512)
    whole = _linear(x, w, None, None, "silu", 128)
    other = x.clone()
    other[::2] = 100
    assert torch.equal(_linear(other, w, None, None, "silu", 128)[1::2], whole[1::2])


def test_linear_refusals():
    g = torch.Generator().manual_seed(4)
    x, (_, w), r = _normal(g, 2, 64).to(DEV), _weights(g, 16, 64), torch.zeros(2, 16, dtype=BF, device=DEV)
    y = torch.empty_like(r)
    linear_act_fp4(x[:0], *w, y[:0])
    with pytest.raises(MoeBlockError):               # y over the residual
        linear_act_fp4(x, *w, r, residual=r)
    with pytest.raises(MoeBlockError):               # n not a multiple of 8
        linear_act_fp4(x, *w, y[:, :12].contiguous())
    with pytest.raises(ValueError):                  # k not a multiple of 32
        linear_act_fp4(x[:, :40].contiguous(), *w, y)
    with pytest.raises(ValueError):                  # codes of another matrix
        linear_act_fp4(x, w[0][:, :, :512], w[1], y)
    with pytest.raises(TypeError):
        linear_act_fp4(x.half(), *w, y)
    with pytest.raises(RuntimeError):
        linear_act_fp4(x.requires_grad_(), *w, y)


# ---------------------------------------------------------------------------
# Experts
# ---------------------------------------------------------------------------
def _experts(x, up, down, ids, probs, dtype=BF, residual=None, **kw):
    whole = torch.full((x.shape[0] + 2, x.shape[1]), 77.0, dtype=dtype, device=DEV)
    y = moe_experts_fp4(x.to(DEV), *up, *down, ids.to(DEV), probs.to(DEV), whole[1:-1],
                        residual=None if residual is None else residual.to(DEV), **kw)
    torch.cuda.synchronize()
    assert (whole[0] == 77).all() and (whole[-1] == 77).all()
    return y


def _layer(g, experts, hidden, inter, act):
    ups = 2 * inter if act == "swiglu" else inter
    return _weights(g, experts, ups, hidden, std=2 * hidden ** -0.5), _weights(g, experts, hidden, inter, std=inter ** -0.5)


def _choice(g, tokens, experts, top_k):
    ids = torch.stack([torch.randperm(experts, generator=g)[:top_k] for _ in range(tokens)]).to(torch.int32)
    return ids, torch.rand(tokens, top_k, generator=g) + 0.05


def _check_experts(tokens, hidden, inter, experts, top_k, act, limit=math.inf, dtype=BF, residual=True, ids=None):
    say(f"[experts_fp4] {tokens} tokens, {hidden} x {inter}, {experts} experts, top {top_k}, {act}, limit {limit}")
    g = torch.Generator().manual_seed(tokens + hidden + inter + experts)
    (vu, wu), (vd, wd) = _layer(g, experts, hidden, inter, act)
    x = _normal(g, tokens, hidden)
    some, probs = _choice(g, tokens, experts, top_k)
    ids = some if ids is None else ids
    r = _normal(g, tokens, hidden) if residual else None
    y = _experts(x, wu, wd, ids, probs, dtype, r, activation=act, limit=limit)
    want, bound = gated.experts(x.double(), vu, vd, ids, probs.double(), act, limit, None if r is None else r.double(), dtype)
    ref.check(y, want, bound, "experts")
    return y


@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 16, 33])
@pytest.mark.parametrize("hidden,inter,experts,top_k", [(32, 32, 1, 1), (96, 64, 5, 3), (160, 288, 8, 8), (512, 128, 16, 2),
                                                        (256, 416, 4, 4)])
def test_experts_sizes(tokens, hidden, inter, experts, top_k):
    _check_experts(tokens, hidden, inter, experts, top_k, "swiglu", 7.0)
    _check_experts(tokens, hidden, inter, experts, top_k, "squared_relu", dtype=torch.float32, residual=False)


# tokens an expert: both sides of what one, two and four groups of columns hold, and more
@pytest.mark.parametrize("tokens", [6, 10, 11, 17, 20, 21, 32, 40, 64, 65, 130, 256])
def test_tokens_of_an_expert(tokens):
    ids = torch.zeros(tokens, 2, dtype=torch.int32)
    ids[:, 1] = torch.arange(tokens) % 3
    for experts in (3, 90, 600):                      # an average of many, some and few tokens an expert
        _check_experts(tokens, 64, 64, experts, 2, "swiglu", 7.0, ids=ids)


def test_experts_elsewhere_and_twice():
    """Ids outside the experts contribute nothing, a repeated one twice; tokens without any expert
    give the residual."""
    ids = torch.tensor([[0, 1, 1], [-1, 5, 2 ** 31 - 1], [4, 4, 4], [3, -2 ** 31, 0]], dtype=torch.int32)
    for dtype in (BF, torch.float32):
        y = _check_experts(4, 128, 96, 5, 3, "swiglu", 2.0, dtype, ids=ids)
    none = torch.full((3, 2), 9, dtype=torch.int32)
    y = _check_experts(3, 64, 32, 4, 2, "swiglu", residual=False, ids=none)
    assert (y == 0).all()


def test_wide_experts():
    _check_experts(2, 2048, 1408, 4, 2, "swiglu", 7.0)
    _check_experts(9, 1024, 2048, 3, 2, "squared_relu")


@pytest.mark.parametrize("valid", [-1, 0, 1, 6, 11, 50])
def test_experts_valid_tokens(valid):
    g = torch.Generator().manual_seed(5)
    (_, wu), (_, wd) = _layer(g, 6, 64, 64, "swiglu")
    x, (ids, probs) = _normal(g, 11, 64), _choice(g, 11, 6, 3)
    n = min(max(valid, 0), 11)
    ids[n:] = 1                                       # behind the end: whatever they say
    y = _experts(x, wu, wd, ids, probs, valid_tokens=torch.tensor([valid], dtype=torch.int32, device=DEV))
    assert (y[n:] == 77).all()
    if n:
        assert torch.equal(y[:n], _experts(x[:n], wu, wd, ids[:n], probs[:n])[:n])


def test_activation_keeps_its_bits():
    """Weights of one: the output is the fp32 activation itself, to its last bit or two, where 16
    bits of it would be off by 2^-17."""
    hidden = inter = 32
    up = torch.zeros(1, inter, hidden)
    up[0, :, 0] = 1
    down = torch.zeros(1, hidden, inter)
    down[0] = torch.eye(hidden)
    wu, wd = _pack(*gated.quantize(up)), _pack(*gated.quantize(down))
    x = torch.zeros(7, hidden, dtype=BF)
    x[:, 0] = torch.tensor([1.0, 1.0078125, 3.015625, 0.00390625, 1.9921875, 1e10, 1e-15]).to(BF)
    p = torch.tensor([1 / 3, 0.1, 0.7, 1e-3, 1.0, 0.9, 0.3])[:, None]
    y = _experts(x, wu, wd, torch.zeros(7, 1, dtype=torch.int32), p, torch.float32, activation="squared_relu")
    h = (x[:, :1].double() ** 2).float().double() * p.double()      # the square is exact in fp32
    assert ((y.cpu().double() - h).abs() <= h * 2.0 ** -23).all()


def test_experts_not_finite():
    """A token's NaN and infinities stay its own."""
    g = torch.Generator().manual_seed(6)
    (_, wu), (_, wd) = _layer(g, 4, 64, 64, "swiglu")
    x, (ids, probs) = _normal(g, 9, 64), _choice(g, 9, 4, 2)
    clean = _experts(x, wu, wd, ids, probs)
    x2, p2 = x.clone(), probs.clone()
    x2[2, 7], x2[5, 1], p2[7, 0] = float("nan"), float("inf"), float("inf")
    y = _experts(x2, wu, wd, ids, p2)
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[5]).all() and not torch.isfinite(y[7]).all()
    keep = [0, 1, 3, 4, 6, 8]
    assert torch.equal(y[keep], clean[keep])


def test_experts_refusals():
    g = torch.Generator().manual_seed(7)
    (_, wu), (_, wd) = _layer(g, 4, 64, 32, "swiglu")
    x, (ids, probs) = _normal(g, 2, 64).to(DEV), [t.to(DEV) for t in _choice(g, 2, 4, 2)]
    y = torch.empty_like(x)
    moe_experts_fp4(x[:0], *wu, *wd, ids[:0], probs[:0], y[:0])
    with pytest.raises(ValueError):
        moe_experts_fp4(x, *wu, *wd, ids, probs, y, limit=0.0)
    with pytest.raises(ValueError):                  # the weights of another number of experts
        moe_experts_fp4(x, *wu, *(t[:3] for t in wd), ids, probs, y)
    with pytest.raises(MoeBlockError):               # y over x
        moe_experts_fp4(x, *wu, *wd, ids, probs, x)
    with pytest.raises(ValueError):
        moe_experts_fp4(x, *wu, *wd, ids, probs, y, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(RuntimeError):
        moe_experts_fp4(x, *wu, *wd, ids, probs.requires_grad_(), y)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
def test_same_bits_streams_and_capture():
    """Every replay of a captured run, and runs at once on two streams with workspaces of their own,
    give the eager bits."""
    g = torch.Generator().manual_seed(8)
    for tokens in (1, 12, 70):
        (_, wu), (_, wd) = _layer(g, 8, 128, 96, "swiglu")
        _, wl = _weights(g, 128, 128, std=0.1)
        x, (ids, probs) = _normal(g, tokens, 128).to(DEV), [t.to(DEV) for t in _choice(g, tokens, 8, 3)]

        def run(stream=None, ws=(None, None)):
            y, z = torch.empty_like(x), torch.empty_like(x)
            linear_act_fp4(x, *wl, z, activation="silu", residual=x, stream=stream, workspace=ws[0])
            moe_experts_fp4(x, *wu, *wd, ids, probs, y, limit=7.0, residual=x, stream=stream, workspace=ws[1])
            return y, z
        want = run()
        sizes = (linear_act_fp4_workspace(tokens, 128, 128), moe_experts_fp4_workspace(tokens, 128, 96, 8, 3))
        streams, got = [torch.cuda.Stream() for _ in range(2)], []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            ws = [torch.empty(max(n, 1), dtype=torch.uint8, device=DEV) for n in sizes]
            with torch.cuda.stream(s):
                got += [run(s, ws) for _ in range(3)]
        torch.cuda.synchronize()
        for out in got:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = run()
        for _ in range(3):
            x.mul_(0.75)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, run()))


@pytest.mark.parametrize("tokens", [1, 21])
def test_a_block(tokens):
    """Norm, gated router, shared expert and routed experts in 4 bits, as a decoding step runs them:
    each operator against 64 bits of the one before it as it came out."""
    g = torch.Generator().manual_seed(11)
    hidden, inter, experts, top_k = 512, 256, 16, 4
    r = _normal(g, tokens, hidden).to(DEV)
    nw, nb = (_normal(g, hidden, std=0.2) + 1).to(DEV), _normal(g, hidden, std=0.2).to(DEV)
    router, bias = _normal(g, experts, hidden, std=0.06).to(DEV), (torch.randn(experts, generator=g) * 0.1).to(DEV)
    v1, s1 = _weights(g, inter, hidden, std=hidden ** -0.5)
    v2, s2 = _weights(g, hidden, inter, std=inter ** -0.5)
    (vu, wu), (vd, wd) = _layer(g, experts, hidden, inter, "swiglu")
    how = dict(scores="sigmoid", groups=4, top_groups=2, group_top=2, renormalize=True, scale=2.5)

    n = layer_norm_fwd(r, nw, nb, torch.empty_like(r))
    a = linear_act_fp4(n, *s1, torch.empty(tokens, inter, dtype=BF, device=DEV), activation="squared_relu")
    shared = linear_act_fp4(a, *s2, torch.empty_like(r), residual=r)
    ids, probs = torch.empty(tokens, top_k, dtype=torch.int32, device=DEV), torch.empty(tokens, top_k, device=DEV)
    moe_route(n, router, ids, probs, bias=bias, **how)
    y = moe_experts_fp4(n, *wu, *wd, ids, probs, torch.empty_like(r), limit=7.0, residual=shared)

    n64, r64 = n.cpu().double(), r.cpu().double()
    want, bound, _ = ref.linear_act(n64, v1, None, "squared_relu", None, BF)
    ref.check(a, want, bound, "shared expert, first product")
    want, bound, _ = ref.linear_act(a.cpu().double(), v2, None, "none", r64, BF)
    ref.check(shared, want, bound, "shared expert")
    logits = n64 @ router.cpu().double().t()
    chosen, (p, bound) = gated.gate(logits, top_k, bias=bias.cpu(), **how)
    assert torch.equal(ids.cpu(), chosen)
    ref.check(probs, p, bound, "probs")
    ids2, probs2 = torch.empty_like(ids), torch.empty_like(probs)      # the same gate from 32-bit logits
    moe_gate_fwd(logits.float().to(DEV), ids2, probs2, bias=bias, **how)
    assert torch.equal(ids2, ids) and torch.allclose(probs2, probs, rtol=1e-5)
    want, bound = gated.experts(n64, vu, vd, ids.cpu(), probs.cpu().double(), "swiglu", 7.0, shared.cpu().double(), BF)
    ref.check(y, want, bound, "experts")
