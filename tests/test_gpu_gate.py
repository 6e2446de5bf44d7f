"""The gate from given logits, the router with the gate behind it, and the gate's gradient, against
64 bits (gated_reference)."""
import pytest
import torch

import block_reference as ref
import gated_reference as gated
from memory_bound_elementwise_amd import (MoeBlockError, MoeGate, moe_gate_bwd, moe_gate_fwd, moe_route,
                                          moe_route_workspace)
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


def _logits(tokens, experts, dt="f32", std=1.5, seed=0):
    g = torch.Generator().manual_seed(seed + tokens * 1000 + experts)
    return (torch.randn(tokens, experts, generator=g) * std).to(ref.TYPES[dt])


def _bias(experts, seed=0):
    return torch.randn(experts, generator=torch.Generator().manual_seed(seed + experts)) * 0.1


def _gate(logits, top_k, bias=None, **how):
    """Rows in front of and behind the outputs must stay as they are."""
    tokens = logits.shape[0]
    ids = torch.full((tokens + 2, top_k), -7, dtype=torch.int32, device=DEV)
    probs = torch.full((tokens + 2, top_k), -7.0, device=DEV)
    moe_gate_fwd(logits.to(DEV), ids[1:-1], probs[1:-1], bias=None if bias is None else bias.to(DEV), **how)
    torch.cuda.synchronize()
    assert (ids[0] == -7).all() and (ids[-1] == -7).all() and (probs[0] == -7).all() and (probs[-1] == -7).all()
    return ids[1:-1].cpu(), probs[1:-1]


def _check(logits, top_k, scores, bias=None, **how):
    ids, probs = _gate(logits, top_k, bias, scores=scores, **how)
    want, (p, bound) = gated.gate(logits, top_k, scores, bias, **how)
    assert torch.equal(ids, want), (ids, want)
    ref.check(probs, p, bound, "probs")
    return ids, probs


# both sides of every variant's border: experts a lane holds, tokens a wave holds
@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 63, 130])
@pytest.mark.parametrize("experts,top_k", [(1, 1), (5, 5), (60, 6), (64, 8), (65, 3), (256, 8), (257, 9), (1000, 64),
                                           (1024, 2)])
def test_sizes(tokens, experts, top_k):
    say(f"[gate] {tokens} tokens, {experts} experts, top {top_k}")
    for dt in ("f32", "bf16", "f16"):
        for scores in ("softmax", "sigmoid"):
            _check(_logits(tokens, experts, dt), top_k, scores, renormalize=dt == "bf16")
    _check(_logits(tokens, experts), top_k, "sigmoid", _bias(experts), renormalize=True, scale=2.5)


@pytest.mark.parametrize("experts,top_k", [(7, 7), (64, 8), (160, 6), (256, 20), (300, 3)])
def test_many_tokens(experts, top_k):
    """More tokens than waves of a token each, and no multiple of a workgroup's."""
    say(f"[gate] 2055 tokens, {experts} experts, top {top_k}")
    _check(_logits(2055, experts), top_k, "sigmoid", _bias(experts), renormalize=True)
    _check(_logits(2055, experts, "bf16"), top_k, "softmax")


@pytest.mark.parametrize("groups,size,top_groups", [(2, 2, 1), (8, 32, 4), (8, 20, 3), (4, 15, 4), (64, 16, 5), (64, 1, 9),
                                                   (3, 21, 2), (16, 4, 16)])
@pytest.mark.parametrize("tokens", [1, 37, 2054])
def test_groups(tokens, groups, size, top_groups):
    experts = groups * size
    say(f"[gate] {tokens} tokens, {groups} groups of {size}, top {top_groups}")
    if tokens > 1000 and experts > 256:
        tokens = 200
    top_k = min(6, top_groups * size)
    for group_top in (1, 2):
        if group_top > size:
            continue
        for scores in ("softmax", "sigmoid"):
            for bias in (None, _bias(experts)):
                _check(_logits(tokens, experts), top_k, scores, bias, groups=groups, top_groups=top_groups,
                       group_top=group_top, renormalize=scores == "sigmoid", scale=1.5)


@pytest.mark.parametrize("tokens", [4, 2124])
def test_ties(tokens):
    """Equal ranks go to the lower expert, equal groups to the lower one; a bias decides between
    equal scores."""
    logits = torch.zeros(tokens, 96)
    assert _check(logits, 8, "softmax")[0].tolist() == [list(range(8))] * tokens
    ids, _ = _check(logits, 8, "sigmoid", groups=4, top_groups=2, group_top=2)
    assert ids[0].tolist() == list(range(8))
    bias = torch.zeros(96)
    bias[50], bias[70] = 0.25, 0.5
    ids, _ = _check(logits, 3, "sigmoid", bias, groups=4, top_groups=2, group_top=1)
    assert ids[0].tolist() == [70, 50, 0]                   # both in group 2; group 0 is the other one kept
    half = _logits(tokens, 48)
    _check(torch.cat((half, half), 1), 9, "softmax")


def test_neighbouring_scores():
    """Ranks that 32 bits cannot tell apart: sigmoid scores near 1, and a bias that all but cancels."""
    logits = torch.tensor([[18.0, 18.000002, 17.999998, 18.000004], [20.0, 20.25, 20.5, 20.125]])
    _check(logits, 4, "sigmoid")
    _check(logits, 4, "sigmoid", torch.full((4,), 4096.0))
    _check(torch.tensor([[0.0, 1e-8, -1e-8, 2e-8]]).repeat(2054, 1), 4, "softmax")


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [8, 2064])
def test_masked_experts(tokens, scores):
    """Logits of -inf: chosen last, with weight 0, whatever their bias; a row of them has weights 0."""
    for experts in (40, 128):
        logits = _logits(tokens, experts)
        logits[1] = -INF
        logits[2, 3:] = -INF
        logits[3, :-1] = -INF
        logits[4, ::2] = -INF
        bias = _bias(experts)
        bias[::3] = 5.0
        for renorm in (False, True):
            for b in (None, bias):
                ids, probs = _check(logits, 6, scores, b, renormalize=renorm)
                _check(logits, 6, scores, b, renormalize=renorm, groups=4, top_groups=2, group_top=2)
                assert ids[1].tolist() == list(range(6)) and (probs[1] == 0).all() and (probs[2, 3:] == 0).all()
                assert probs[3, 1:].abs().max() == 0
    lowest = _logits(tokens, 40)
    lowest[0] = torch.finfo(torch.float32).min            # the type's lowest value is a number like any other
    lowest[1, 5:] = torch.finfo(torch.float32).min
    _check(lowest, 6, scores, renormalize=True)


@pytest.mark.parametrize("tokens,experts", [(7, 24), (7, 200), (2074, 48), (2074, 200), (9, 900)])
def test_chosen_far_below_the_largest(tokens, experts):
    """A bias that keeps the largest logits out: the chosen ones' softmax is far from fp64's end, also
    where their scores among all experts are past it; the gradient is that of these weights."""
    logits = _logits(tokens, experts)
    logits[::2, :4] += torch.tensor([600.0, 700.0, 900.0, 1e30])
    logits[1::3, 3] += 650.0
    bias = _bias(experts)
    bias[:4] = -INF
    ids, probs = _check(logits, 6, "softmax", bias, renormalize=True, scale=2.0)
    assert (ids > 3).all() and (probs.sum(1) - 2).abs().max() < 1e-6
    g = torch.randn(tokens, 6)
    want, bound = gated.gate_grads(logits, ids, g, "softmax", True, 2.0, torch.float32)
    ref.check(_grads(logits, ids, g, scores="softmax", renormalize=True, scale=2.0), want, bound, "grad_logits")


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_not_finite(scores):
    """NaN comes before any number, +inf is a number for the sigmoid; a token's NaN stays its own."""
    logits = _logits(2054, 70)
    logits[1, 9] = NAN
    logits[3, 20] = INF
    logits[4] = NAN
    for tokens in (6, 2054):
        part = logits[:tokens]
        for how in (dict(), dict(renormalize=True), dict(groups=7, top_groups=2, group_top=2)):
            ids, probs = _check(part, 5, scores, **how)
            clean = [0, 2, 5]
            alone = _gate(part[clean], 5, scores=scores, **how)
            assert torch.equal(ids[clean], alone[0]) and torch.equal(probs[clean], alone[1])
    bias = _bias(70)
    bias[3], bias[4], bias[5] = INF, -INF, NAN
    _check(_logits(20, 70), 64, scores, bias)


@pytest.mark.parametrize("valid", [-3, 0, 1, 7, 20, 99])
def test_valid_tokens(valid):
    v = torch.tensor([valid], dtype=torch.int32, device=DEV)
    n = min(max(valid, 0), 20)
    logits = _logits(20, 48)
    for reps in (1, 110):                                   # 2200 tokens: several a wave
        part = logits.repeat(reps, 1)
        whole = _gate(part, 4, scores="sigmoid")
        ids, probs = _gate(part, 4, scores="sigmoid", valid_tokens=v)
        m = min(max(valid, 0), len(part))
        assert torch.equal(ids[:m], whole[0][:m]) and torch.equal(probs[:m], whole[1][:m])
        assert (ids[m:] == -7).all() and (probs[m:] == -7).all()
    g = torch.randn(20, 4, device=DEV)
    out = torch.full((20, 48), 5.0, device=DEV)
    full = moe_gate_bwd(logits.to(DEV), _gate(logits, 4)[0].to(DEV), g, torch.empty_like(out))
    moe_gate_bwd(logits.to(DEV), _gate(logits, 4)[0].to(DEV), g, out, valid_tokens=v)
    assert torch.equal(out[:n], full[:n]) and (out[n:] == 5).all()


# ---------------------------------------------------------------------------
# Behind the router's product
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tokens", [1, 4, 5, 33, 260])
@pytest.mark.parametrize("hidden,experts,top_k,groups,top_groups", [(24, 5, 5, 1, 1), (264, 64, 8, 8, 3), (2056, 160, 6, 8, 3),
                                                                    (7168, 256, 8, 8, 4), (136, 300, 20, 5, 2)])
def test_route(tokens, hidden, experts, top_k, groups, top_groups):
    say(f"[route] {tokens} tokens, hidden {hidden}, {experts} experts, top {top_k}, {groups} groups")
    g = torch.Generator().manual_seed(tokens + hidden)
    x = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    bias = _bias(experts)
    for rdt in (torch.bfloat16, torch.float32):
        router = (torch.randn(experts, hidden, generator=g) * 1.5 * hidden ** -0.5).to(rdt)
        for scores in ("sigmoid", "softmax"):
            how = dict(scores=scores, groups=groups, top_groups=top_groups, group_top=2 if groups > 1 else 1,
                       renormalize=scores == "sigmoid", scale=2.5)
            ids = torch.full((tokens, top_k), -7, dtype=torch.int32, device=DEV)
            probs = torch.full((tokens, top_k), -7.0, device=DEV)
            moe_route(x.to(DEV), router.to(DEV), ids, probs, bias=bias.to(DEV), **how)
            # fp64 logits; the gate as it stands, in fp64 too
            want, (p, bound) = gated.gate(x.double() @ router.double().t(), top_k, bias=bias, **how)
            assert torch.equal(ids.cpu(), want)
            ref.check(probs, p, bound, "probs")


def test_route_without_a_gate_is_the_router():
    """The default arguments give the plain router's bits, and the gate agrees with it."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(9, 512, generator=g).to(torch.bfloat16).to(DEV)
    router = (torch.randn(48, 512, generator=g) * 0.06).to(torch.bfloat16).to(DEV)

    def route(**how):
        ids, probs = torch.empty(9, 4, dtype=torch.int32, device=DEV), torch.empty(9, 4, device=DEV)
        moe_route(x, router, ids, probs, **how)
        return ids, probs
    plain, gate = route(), route(bias=torch.zeros(48, device=DEV))
    assert torch.equal(plain[0], gate[0]) and torch.allclose(plain[1], gate[1], rtol=2.0 ** -23, atol=0)
    with pytest.raises(MoeBlockError):                       # a group that is not there is refused all the same
        route(top_groups=2)


# ---------------------------------------------------------------------------
# Gradient
# ---------------------------------------------------------------------------
def _grads(logits, ids, g, **how):
    whole = torch.full((logits.shape[0] + 2, logits.shape[1]), 77.0, dtype=logits.dtype, device=DEV)
    flat = whole.view(-1)
    pad = -logits.shape[1] * logits.element_size() % 16      # the gradient starts at 16 bytes
    if pad:
        out = torch.full_like(logits, 77.0, device=DEV)
    else:
        out = whole[1:-1]
    moe_gate_bwd(logits.to(DEV), ids.to(DEV), g.to(DEV), out, **how)
    torch.cuda.synchronize()
    if not pad:
        assert (flat[:logits.shape[1]] == 77).all() and (flat[-logits.shape[1]:] == 77).all()
    return out


@pytest.mark.parametrize("tokens", [1, 2, 5, 130, 2055])
@pytest.mark.parametrize("experts,top_k", [(1, 1), (5, 5), (60, 6), (64, 8), (65, 3), (256, 8), (257, 9), (1000, 64)])
def test_gradient(tokens, experts, top_k):
    say(f"[gate_bwd] {tokens} tokens, {experts} experts, top {top_k}")
    if tokens > 1000 and experts > 256:
        tokens = 150
    for dt in ("f32", "bf16", "f16"):
        logits = _logits(tokens, experts, dt)
        g = torch.randn(tokens, top_k, generator=torch.Generator().manual_seed(1))
        ids = torch.argsort(logits.double(), dim=1, descending=True)[:, :top_k].to(torch.int32).contiguous()
        for scores in ("softmax", "sigmoid"):
            for renorm in (False, True):
                got = _grads(logits, ids, g, scores=scores, renormalize=renorm, scale=2.5)
                want, bound = gated.gate_grads(logits, ids, g, scores, renorm, 2.5, logits.dtype)
                ref.check(got, want, bound, f"grad_logits {scores} {renorm}")


def test_gradient_of_odd_choices():
    """Ids outside the experts contribute nothing, a repeated one twice; masked experts and rows of
    them have zeros; far logits keep their digits."""
    logits = _logits(2054, 40)
    logits[3] = -INF
    logits[4, 1:] = -INF
    logits[5] *= 200
    logits[6] -= 500
    ids = torch.randint(-2, 43, (2054, 7), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    ids[0], ids[1] = 11, -1
    ids[2, 3] = 2 ** 31 - 1
    ids[4] = torch.arange(7)
    g = torch.randn(2054, 7, generator=torch.Generator().manual_seed(3))
    for tokens in (8, 2054):
        for scores in ("softmax", "sigmoid"):
            for renorm in (False, True):
                got = _grads(logits[:tokens], ids[:tokens], g[:tokens], scores=scores, renormalize=renorm)
                want, bound = gated.gate_grads(logits[:tokens], ids[:tokens], g[:tokens], scores, renorm, 1.0, torch.float32)
                ref.check(got, want, bound, f"grad_logits {scores} {renorm}")
                assert (got[1] == 0).all() and (got[3] == 0).all()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(scores, renorm):
    """Central differences of the 64-bit gate with its choice held fixed; step 1e-4, so that the
    differences are off by about 1e-8 of the weights, and the kernel by 2^-24 of its gradient."""
    logits = _logits(6, 12)
    ids, _ = gated.gate(logits, 4, scores)
    g = torch.randn(6, 4, generator=torch.Generator().manual_seed(5))

    def total(l):
        out = torch.zeros(6, dtype=torch.float64)
        for t in range(6):
            p = gated.scores_of(l[t], scores)[ids[t].long()]
            out[t] = ((p / p.sum() if renorm else p) * g[t].double()).sum()
        return out
    want = torch.zeros(6, 12, dtype=torch.float64)
    for i in range(12):
        up, down = logits.double(), logits.double()
        up[:, i] += 1e-4
        down[:, i] -= 1e-4
        want[:, i] = (total(up) - total(down)) / 2e-4
    got = _grads(logits, ids, g, scores=scores, renormalize=renorm)
    assert (got.cpu().double() - want).abs().max() < 1e-7 * max(1.0, float(g.abs().max()) * 4)


def test_autograd():
    """MoeGate: any leading axes, strides and offsets; shared and unused gradients."""
    logits = _logits(24, 96).to(DEV)
    bias = _bias(96).to(DEV)
    how = dict(scores="sigmoid", groups=4, top_groups=2, group_top=2, renormalize=True, scale=2.5)
    want_ids, (p, bound) = gated.gate(logits.cpu(), 6, bias=bias.cpu(), **how)
    wide = torch.zeros(4, 6, 2, 97, device=DEV)
    wide[:, :, 1, 1:] = logits.view(4, 6, 96)
    for src in (logits.clone().view(4, 6, 96), wide[:, :, 1, 1:]):
        leaf = src.detach().requires_grad_()
        probs, ids = MoeGate.apply(leaf, 6, bias, "sigmoid", 4, 2, 2, True, 2.5)
        assert probs.shape == (4, 6, 6) and not ids.requires_grad
        assert torch.equal(ids.view(24, 6).cpu(), want_ids)
        ref.check(probs.view(24, 6), p, bound, "probs")
        up = torch.randn(6, 4, 6, device=DEV).transpose(0, 1)
        probs.backward(up)
        g, gb = gated.gate_grads(logits.cpu(), want_ids, up.reshape(24, 6).cpu(), "sigmoid", True, 2.5, torch.float32)
        ref.check(leaf.grad.reshape(24, 96), g, gb, "grad_logits")
    leaf = logits.clone().requires_grad_()
    probs, _ = MoeGate.apply(leaf, 2)
    (probs.sum() + probs[0].sum()).backward()                # a broadcast gradient
    up = torch.ones(24, 2)
    up[0] = 2
    ids, _ = gated.gate(logits.cpu(), 2, "softmax")
    g, gb = gated.gate_grads(logits.cpu(), ids, up, "softmax", False, 1.0, torch.float32)
    ref.check(leaf.grad, g, gb, "grad_logits")
    half = logits.to(torch.bfloat16).requires_grad_()
    MoeGate.apply(half, 2)[0].sum().backward()
    assert half.grad.dtype == torch.bfloat16
    none = torch.empty(3, 0, 96, device=DEV, requires_grad=True)
    probs, ids = MoeGate.apply(none, 2)
    probs.sum().backward()
    assert probs.shape == ids.shape == (3, 0, 2) and none.grad.shape == none.shape
    one = logits[0].clone().requires_grad_()
    probs, ids = MoeGate.apply(one, 2)
    probs.backward(up[0].to(DEV))
    assert probs.shape == ids.shape == (2,)
    ref.check(one.grad[None], *gated.gate_grads(logits[:1].cpu(), ids[None].cpu(), up[:1], "softmax", False, 1.0,
                                                torch.float32), "grad_logits")


def test_captured_autograd_is_refused():
    """A backward into a leaf inside a capture raises, with an eager graph of the same leaf alive, and
    leaves the process able to go on."""
    leaf = _logits(8, 16).to(DEV).requires_grad_()
    g = torch.randn(8, 2, device=DEV)
    eager, _ = MoeGate.apply(leaf, 2)                        # stays alive over the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(graph):
            torch.autograd.grad(MoeGate.apply(leaf, 2)[0], leaf, g)
    torch.cuda.synchronize()
    first, = torch.autograd.grad(eager, leaf, g)
    again, = torch.autograd.grad(MoeGate.apply(leaf, 2)[0], leaf, g)
    assert torch.equal(first, again)


# ---------------------------------------------------------------------------
# Calls
# ---------------------------------------------------------------------------
def test_same_bits_streams_and_capture():
    """Every replay of a captured run gives the eager bits, also while another stream runs the same."""
    for tokens in (3, 2500):
        logits, bias = _logits(tokens, 96).to(DEV), _bias(96).to(DEV)
        x = torch.randn(tokens, 256, device=DEV).to(torch.bfloat16)
        router = (torch.randn(96, 256, device=DEV) * 0.1).to(torch.bfloat16)
        g = torch.randn(tokens, 6, device=DEV)
        how = dict(scores="sigmoid", renormalize=True)
        group = dict(groups=4, top_groups=2, group_top=2, bias=bias)

        def run(stream=None, workspace=None):
            out = [torch.empty(tokens, 6, dtype=t, device=DEV) for t in (torch.int32, torch.float32) * 2]
            grad = torch.empty_like(logits)
            moe_gate_fwd(logits, out[0], out[1], **how, **group, stream=stream)
            moe_gate_bwd(logits, out[0], g, grad, **how, stream=stream)
            moe_route(x, router, out[2], out[3], **how, **group, stream=stream, workspace=workspace)
            return out + [grad]
        want = run()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            ws = torch.empty(moe_route_workspace(tokens, 256, 96), dtype=torch.uint8, device=DEV)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got += [run(s, ws) for _ in range(2)]
        torch.cuda.synchronize()
        for out in got:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = run()
        for i in range(3):
            logits.mul_(0.75)
            x.mul_(0.5)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, run()))


def test_nothing_and_refusals():
    logits = _logits(4, 16).to(DEV)
    ids, probs = torch.empty(4, 2, dtype=torch.int32, device=DEV), torch.empty(4, 2, device=DEV)
    moe_gate_fwd(logits[:0], ids[:0], probs[:0])
    moe_gate_bwd(logits[:0], ids[:0], probs[:0], logits[:0].clone())
    for bad in (dict(groups=3), dict(groups=0), dict(groups=4, top_groups=5), dict(groups=16, group_top=2), dict(scale=INF),
                dict(group_top=3), dict(groups=16, top_groups=1)):
        with pytest.raises(MoeBlockError):
            moe_gate_fwd(logits, ids, probs, **bad)
    with pytest.raises(ValueError):
        moe_gate_fwd(logits, ids, probs, scores="tanh")
    with pytest.raises(ValueError):
        moe_gate_fwd(logits.t(), ids, probs)
    with pytest.raises(TypeError):
        moe_gate_fwd(logits.double(), ids, probs)
    with pytest.raises(ValueError):
        moe_gate_fwd(logits, ids, probs, bias=torch.zeros(15, device=DEV))
    with pytest.raises(MoeBlockError):                       # the gradient over the logits
        moe_gate_bwd(logits, ids, probs, logits)
