"""The router, the expert products for a few tokens and both in one call, against 64 bits
(block_reference)."""
import math

import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import (LayerNorm, MoeBlockError, layer_norm_fwd, linear_act, moe_experts,
                                          moe_layer, moe_layer_workspace, moe_route)
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _normal(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


# ---------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------
def _route(x, router, top_k, renorm, **kw):
    ids = torch.full((x.shape[0], top_k), -7, dtype=torch.int32, device=DEV)
    probs = torch.full((x.shape[0], top_k), -7.0, device=DEV)
    moe_route(x.to(DEV), router.to(DEV), ids, probs, renormalize=renorm, **kw)
    torch.cuda.synchronize()
    return ids.cpu(), probs


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 40, 130])
@pytest.mark.parametrize("hidden,experts,top_k", [(8, 1, 1), (24, 5, 5), (264, 64, 8), (1000, 65, 3), (512, 256, 8),
                                                  (136, 300, 64), (2056, 1024, 2), (7168, 64, 8)])
def test_route(tokens, hidden, experts, top_k):
    say(f"[route] {tokens} tokens, hidden {hidden}, {experts} experts, top {top_k}")
    g = torch.Generator().manual_seed(tokens * 7 + hidden)
    x = _normal(g, tokens, hidden)
    for rdt in (BF, torch.float32):
        router = _normal(g, experts, hidden, std=hidden ** -0.5, dtype=rdt)
        for renorm in (False, True):
            ids, probs = _route(x, router, top_k, renorm)
            want, (p, bound) = ref.route(x.double(), router.double(), top_k, renorm)
            assert torch.equal(ids, want)
            ref.check(probs, p, bound, "probs")


def test_route_ties_zeros_and_far_logits():
    """Equal logits go to the lower expert; zero rows tie everywhere; logits far apart."""
    g = torch.Generator().manual_seed(3)
    x = _normal(g, 6, 64)
    x[1] = 0
    x[2] *= 200
    router = _normal(g, 40, 64)
    router[20:] = router[:20]                  # every logit twice
    router[7] = -router[7].abs()
    for renorm in (False, True):
        ids, probs = _route(x, router, 9, renorm)
        want, (p, bound) = ref.route(x.double(), router.double(), 9, renorm)
        assert torch.equal(ids, want)
        ref.check(probs, p, bound, "probs")
    assert ids[1].tolist() == list(range(9))


def test_route_neighbouring_logits():
    """Logits that differ by 2^-40 relative, which 32-bit sums cannot tell apart."""
    x = torch.zeros(2, 64, dtype=BF)
    x[:, 0], x[:, 1] = 1.0, 2.0 ** -20
    router = torch.zeros(5, 64, dtype=BF)
    router[:, 0] = 1.0
    router[:, 1] = torch.tensor([1, 3, 2, 5, 4]).to(BF) * 2.0 ** -20
    ids, _ = _route(x, router, 5, True)
    assert ids.tolist() == [[3, 4, 1, 2, 0]] * 2


def test_route_not_finite():
    """NaN comes before any number; a token's NaN or infinity stays its own."""
    g = torch.Generator().manual_seed(4)
    x = _normal(g, 5, 32)
    router = _normal(g, 6, 32)
    x[1, 3] = float("nan")
    x[3, 0] = float("inf")
    clean = _route(x[[0, 2, 4]], router, 3, False)
    ids, probs = _route(x, router, 3, False)
    assert torch.equal(ids[[0, 2, 4]], clean[0]) and torch.equal(probs[[0, 2, 4]], clean[1])
    assert ids[1].tolist() == [0, 1, 2] and torch.isnan(probs[1]).all()
    assert torch.isnan(probs[3, 0])


@pytest.mark.parametrize("valid", [-3, 0, 1, 7, 20, 99])
def test_route_valid_tokens(valid):
    g = torch.Generator().manual_seed(5)
    x, router = _normal(g, 20, 128), _normal(g, 16, 128, std=0.1)
    ids, probs = _route(x, router, 4, True, valid_tokens=torch.tensor([valid], dtype=torch.int32, device=DEV))
    whole_ids, whole_probs = _route(x, router, 4, True)
    n = min(max(valid, 0), 20)
    assert torch.equal(ids[:n], whole_ids[:n]) and torch.equal(probs[:n], whole_probs[:n])
    assert (ids[n:] == -7).all() and (probs[n:] == -7).all()


# ---------------------------------------------------------------------------
# Experts
# ---------------------------------------------------------------------------
def _weights(g, experts, hidden, inter, act):
    ups = 2 * inter if act == "swiglu" else inter
    return (_normal(g, experts, ups, hidden, std=2 * hidden ** -0.5), _normal(g, experts, hidden, inter, std=inter ** -0.5))


def _experts(x, wu, wd, ids, probs, dtype=BF, residual=None, **kw):
    whole = torch.full((x.shape[0] + 2, x.shape[1]), 77.0, dtype=dtype, device=DEV)
    y = moe_experts(x.to(DEV), wu.to(DEV), wd.to(DEV), ids.to(DEV), probs.to(DEV), whole[1:-1],
                    residual=None if residual is None else residual.to(DEV), **kw)
    torch.cuda.synchronize()
    assert (whole[0] == 77).all() and (whole[-1] == 77).all()
    return y


def _check_experts(tokens, hidden, inter, experts, top_k, act, limit=math.inf, dtype=BF, residual=True, ids=None, seed=0):
    say(f"[experts] {tokens} tokens, {hidden} x {inter}, {experts} experts, top {top_k}, {act}, limit {limit}")
    g = torch.Generator().manual_seed(seed + tokens + hidden + inter)
    x = _normal(g, tokens, hidden)
    wu, wd = _weights(g, experts, hidden, inter, act)
    if ids is None:
        ids = torch.stack([torch.randperm(experts, generator=g)[:top_k] for _ in range(tokens)]).to(torch.int32)
    probs = torch.rand(tokens, top_k, generator=g)
    r = _normal(g, tokens, hidden) if residual else None
    y = _experts(x, wu, wd, ids, probs, dtype, r, activation=act, limit=limit)
    v, bound = ref.experts(x.double(), wu.double(), wd.double(), ids, probs.double(), act, limit,
                           None if r is None else r.double(), dtype)
    ref.check(y, v, bound, "experts")


@pytest.mark.parametrize("tokens", [1, 2, 5, 16, 17, 40])
@pytest.mark.parametrize("hidden,inter", [(8, 8), (24, 40), (136, 264), (520, 128)])
@pytest.mark.parametrize("act", ["swiglu", "squared_relu"])
def test_experts(tokens, hidden, inter, act):
    _check_experts(tokens, hidden, inter, 6, 3, act, limit=1.5)


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 64, 8), (64, 2, 2), (130, 2, 1), (128, 8, 8),
                                                  (1024, 3, 1), (33, 33, 31), (7, 1024, 5), (128, 256, 1),
                                                  (65, 40, 2), (100, 128, 3), (128, 64, 8), (90, 12, 2),
                                                  (129, 64, 4), (64, 64, 8), (32, 4, 4)])
def test_experts_counts(tokens, experts, top_k):
    """One expert for every token (several reads of its weights), more experts than pairs, the
    largest number of pairs."""
    _check_experts(tokens, 40, 24, experts, top_k, "swiglu")
    _check_experts(tokens, 40, 24, experts, top_k, "squared_relu", dtype=torch.float32, residual=False)


@pytest.mark.parametrize("tokens,hidden,inter", [(1, 2056, 1032), (3, 7168, 256), (20, 256, 2048), (2, 64, 4104),
                                                  (70, 1032, 136)])
def test_experts_long(tokens, hidden, inter):
    _check_experts(tokens, hidden, inter, 4, 2, "swiglu", limit=7.0)
    _check_experts(tokens, hidden, inter, 4, 2, "squared_relu", dtype=torch.float32)


def test_ids_outside_repeated_and_none():
    """Ids outside the experts contribute nothing, a repeated id counts twice, a token may have
    none at all (its row is the residual, or zero)."""
    ids = torch.tensor([[0, 0, 3], [-1, 4, 2], [-1, -1, 4], [2147483647, -2147483648, 1], [3, 3, 3]], dtype=torch.int32)
    for residual in (True, False):
        for dtype in (BF, torch.float32):
            _check_experts(5, 72, 136, 4, 3, "swiglu", 7.0, dtype, residual, ids)
    g = torch.Generator().manual_seed(1)
    x = _normal(g, 5, 72)
    wu, wd = _weights(g, 4, 72, 136, "swiglu")
    none = torch.full((5, 3), -1, dtype=torch.int32)
    probs = torch.ones(5, 3)
    assert not _experts(x, wu, wd, none, probs).any()
    r = _normal(g, 5, 72)
    assert torch.equal(_experts(x, wu, wd, none, probs, residual=r).cpu(), r)


@pytest.mark.parametrize("valid", [-1, 0, 1, 5, 11, 50, 79, 200])
@pytest.mark.parametrize("tokens,experts", [(11, 3), (11, 200), (80, 16), (150, 8)])
def test_experts_valid_tokens(valid, tokens, experts):
    g = torch.Generator().manual_seed(8)
    x = _normal(g, tokens, 64)
    wu, wd = _weights(g, experts, 64, 72, "swiglu")
    ids = torch.randint(0, experts, (tokens, 2), generator=g, dtype=torch.int32)
    probs = torch.rand(tokens, 2, generator=g)
    n = min(max(valid, 0), tokens)
    whole = _experts(x, wu, wd, ids, probs)
    # what lies behind the last token is not read: ids far outside, NaN
    ids[n:], probs[n:], x[n:] = 1 << 30, float("nan"), float("nan")
    y = _experts(x, wu, wd, ids, probs, valid_tokens=torch.tensor([valid], dtype=torch.int32, device=DEV))
    assert torch.equal(y[:n], whole[:n]) and (y[n:] == 77).all()


def test_repeated_ids_of_many_tokens():
    """The same expert twice in a token, next to each other in its list, in the form for many."""
    ids = torch.randint(-1, 5, (70, 4), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    ids[::3, 1] = ids[::3, 0]
    ids[5] = 2
    ids[6] = -1
    for dtype in (BF, torch.float32):
        _check_experts(70, 72, 136, 4, 4, "swiglu", 7.0, dtype, True, ids)


def test_not_finite_tokens_and_weights():
    """A token's NaN or infinity stays in its row; an unused expert's weights are not read."""
    g = torch.Generator().manual_seed(9)
    x = _normal(g, 6, 64)
    wu, wd = _weights(g, 4, 64, 72, "swiglu")
    ids = torch.tensor([[0, 1]] * 6, dtype=torch.int32)
    probs = torch.rand(6, 2, generator=g)
    clean = _experts(x, wu, wd, ids, probs)
    wu[3], wd[3] = float("nan"), float("nan")
    x[1, 0], x[4, 63] = float("nan"), float("inf")
    probs[2, 1] = float("nan")
    y = _experts(x, wu, wd, ids, probs)
    assert torch.equal(y[[0, 3, 5]], clean[[0, 3, 5]])
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all() and not torch.isfinite(y[4]).any()


def test_large_activations_keep_their_range():
    """Squared ReLU reaches 2^126: h is cut into two bf16 terms without becoming infinite."""
    x = torch.full((1, 8), 2.0 ** 30, dtype=BF)
    wu = torch.zeros(1, 8, 8, dtype=BF)
    wu[0, :, 0] = 2.0 ** 33
    wd = torch.full((1, 8, 8), 2.0 ** -100, dtype=BF)
    y = _experts(x, wu, wd, torch.zeros(1, 1, dtype=torch.int32), torch.tensor([[1.9999999]]), torch.float32,
                 activation="squared_relu")
    want = 8 * float(torch.tensor(1.9999999)) * 2.0 ** 126 * 2.0 ** -100
    assert ((y.cpu().double() / want - 1).abs() < 2.0 ** -15).all()


# ---------------------------------------------------------------------------
# The whole layer, and a block of the operators together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k,act", [(1, 256, 128, 64, 8, "swiglu"),
                                                                   (9, 136, 72, 12, 4, "squared_relu"),
                                                                   (64, 512, 64, 16, 8, "swiglu")])
def test_layer_is_route_and_experts(tokens, hidden, inter, experts, top_k, act):
    g = torch.Generator().manual_seed(tokens)
    x, router = _normal(g, tokens, hidden).to(DEV), _normal(g, experts, hidden, std=hidden ** -0.5).to(DEV)
    wu, wd = [t.to(DEV) for t in _weights(g, experts, hidden, inter, act)]
    r = _normal(g, tokens, hidden).to(DEV)
    ids, probs = torch.empty(tokens, top_k, dtype=torch.int32, device=DEV), torch.empty(tokens, top_k, device=DEV)
    y = moe_layer(x, router, wu, wd, torch.empty_like(x), ids, probs, activation=act, limit=7.0, renormalize=True,
                  residual=r)
    ids2, probs2 = torch.empty_like(ids), torch.empty_like(probs)
    moe_route(x, router, ids2, probs2, renormalize=True)
    y2 = moe_experts(x, wu, wd, ids2, probs2, torch.empty_like(x), activation=act, limit=7.0, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(probs, probs2) and torch.equal(y, y2)
    v, bound = ref.experts(x.cpu().double(), wu.cpu().double(), wd.cpu().double(), ids.cpu(), probs.cpu().double(), act,
                           7.0, r.cpu().double(), BF)
    ref.check(y, v, bound, "layer")


def test_layer_captured_and_on_two_streams():
    """Decoding as a program does it: one captured layer replayed for new tokens and a changing
    number of valid ones, eager calls between; and two streams at once, a workspace each."""
    tokens, hidden, inter, experts, top_k = 12, 256, 136, 16, 4
    g = torch.Generator().manual_seed(1)
    x, router = _normal(g, tokens, hidden).to(DEV), _normal(g, experts, hidden, std=0.1).to(DEV)
    wu, wd = [t.to(DEV) for t in _weights(g, experts, hidden, inter, "swiglu")]
    ids, probs = torch.zeros(tokens, top_k, dtype=torch.int32, device=DEV), torch.zeros(tokens, top_k, device=DEV)
    y = torch.zeros_like(x)
    valid = torch.tensor([tokens], dtype=torch.int32, device=DEV)

    def call(o, i, p, **kw):
        return moe_layer(x, router, wu, wd, o, i, p, limit=7.0, valid_tokens=valid, residual=x, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(y, ids, probs)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y, ids, probs)
    for n in (12, 3, 0, 1, 12):
        x.copy_(_normal(g, tokens, hidden))
        valid.fill_(n)
        for t in (y, ids, probs):
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        o, i, p = torch.full_like(y, 5), torch.full_like(ids, 5), torch.full_like(probs, 5)
        call(o, i, p)
        torch.cuda.synchronize()
        assert torch.equal(y, o) and torch.equal(ids, i) and torch.equal(probs, p)
        assert (y[n:] == 5).all()
    need = moe_layer_workspace(tokens, hidden, inter, experts, top_k)
    got = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        for _ in range(4):
            o, i, p = torch.full_like(y, 5), torch.full_like(ids, 5), torch.full_like(probs, 5)
            s.wait_stream(torch.cuda.current_stream())
            call(o, i, p, stream=s, workspace=ws)
            got.append((o, i, p))
    torch.cuda.synchronize()
    for o, i, p in got:
        assert torch.equal(y, o) and torch.equal(ids, i) and torch.equal(probs, p)


@pytest.mark.parametrize("tokens", [1, 5, 70])
def test_block(tokens):
    """The second half of a block as a serving program runs it: pre-norm, shared expert (two
    products, the second onto the residual stream), routed experts on top."""
    hidden, inter, experts, top_k = 264, 136, 16, 3
    g = torch.Generator().manual_seed(tokens)
    stream = _normal(g, tokens, hidden, std=2.0)
    nw, nb = _normal(g, hidden), _normal(g, hidden)
    s1, s2 = _normal(g, inter, hidden, std=hidden ** -0.5), _normal(g, hidden, inter, std=inter ** -0.5)
    router = _normal(g, experts, hidden, std=hidden ** -0.5)
    wu, wd = _weights(g, experts, hidden, inter, "swiglu")
    d = [t.to(DEV) for t in (stream, nw, nb, s1, s2, router, wu, wd)]
    h = layer_norm_fwd(d[0], d[1], d[2], torch.empty_like(d[0]))
    a = linear_act(h, d[3], torch.empty(tokens, inter, dtype=BF, device=DEV), activation="squared_relu")
    r = linear_act(a, d[4], torch.empty_like(h), residual=d[0])
    ids, probs = torch.empty(tokens, top_k, dtype=torch.int32, device=DEV), torch.empty(tokens, top_k, device=DEV)
    y = moe_layer(h, d[5], d[6], d[7], torch.empty_like(h), ids, probs, limit=7.0, residual=r)
    torch.cuda.synchronize()
    # each step against 64 bits on the step before it
    (v, bound), _, _ = ref.layer_norm(stream.double(), nw.double(), nb.double(), 1e-5, BF)
    ref.check(h, v, bound, "norm")
    h, a, r = h.cpu().double(), a.cpu().double(), r.cpu().double()
    v, bound, _ = ref.linear_act(h, s1.double(), None, "squared_relu", None, BF)
    ref.check(a, v, bound, "shared up")
    v, bound, _ = ref.linear_act(a, s2.double(), None, None, stream.double(), BF)
    ref.check(r, v, bound, "shared down")
    want, (p, bound) = ref.route(h, router.double(), top_k, False)
    assert torch.equal(ids.cpu(), want)
    ref.check(probs, p, bound, "probs")
    v, bound = ref.experts(h, wu.double(), wd.double(), ids.cpu(), probs.cpu().double(), "swiglu", 7.0, r, BF)
    ref.check(y, v, bound, "layer")


def test_refusals():
    g = torch.Generator().manual_seed(1)
    x, router = _normal(g, 4, 64).to(DEV), _normal(g, 8, 64).to(DEV)
    wu, wd = [t.to(DEV) for t in _weights(g, 8, 64, 24, "swiglu")]
    ids, probs = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV)
    with pytest.raises(MoeBlockError):                    # y over x
        moe_experts(x, wu, wd, ids, probs, x)
    with pytest.raises(MoeBlockError):                    # more chosen than experts
        many = torch.zeros(4, 9, dtype=torch.int32, device=DEV)
        moe_route(x, router, many, torch.zeros(4, 9, device=DEV))
    with pytest.raises(MoeBlockError):                    # more than 1024 pairs
        big = torch.zeros(600, 64, dtype=BF, device=DEV)
        moe_experts(big, wu, wd, torch.zeros(600, 2, dtype=torch.int32, device=DEV), torch.zeros(600, 2, device=DEV),
                    torch.empty_like(big))
    with pytest.raises(ValueError):
        moe_experts(x, wu, wd, ids, probs, torch.empty_like(x), limit=0.0)
    with pytest.raises(ValueError):
        moe_layer(x, router, wu, wd, torch.empty_like(x), ids, probs, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(RuntimeError):
        moe_route(x.requires_grad_(), router, ids, probs)
    assert LayerNorm is not None
