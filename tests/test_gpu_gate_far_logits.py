"""The gate where fp64 scores cannot tell logits apart: softmax scores that run out of exponents,
sigmoid scores of 1, sums of scores near the end of fp64. Expected values are formed from the logits
themselves, on the CPU in 64 bits."""
import pytest
import torch

import block_reference as ref
import gated_reference as gated
from memory_bound_elementwise_amd import MoeGate, moe_gate_bwd, moe_gate_fwd, moe_route
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")
KINDS = [torch.float32, torch.bfloat16, torch.float16]


def _gate(logits, top_k, **how):
    ids = torch.empty(len(logits), top_k, dtype=torch.int32, device=DEV)
    probs = torch.empty(len(logits), top_k, device=DEV)
    moe_gate_fwd(logits.to(DEV), ids, probs, **how)
    return ids.cpu(), probs.cpu()


def _far(tokens, experts, kind, seed=0):
    """Logits thousands apart, and rows where they are large and close together."""
    g = torch.Generator().manual_seed(seed + tokens + experts)
    logits = torch.randn(tokens, experts, generator=g) * 3000
    logits[::3] = 60 + 4 * torch.randn(logits[::3].shape, generator=g)
    logits[1, experts // 2:] = -INF
    return logits.to(kind)


def _largest(logits, top_k):
    """Larger logits first, equal ones in increasing order."""
    return torch.sort(logits.double(), dim=1, descending=True, stable=True)[1][:, :top_k]


def _weights(logits, ids, scores, renormalize):
    """Of the chosen experts, in 64 bits."""
    l = logits.double()
    mine = l.gather(1, ids.long())
    if scores == "softmax":
        top = l.amax(1, keepdim=True)
        e = torch.exp(mine - top)
        return e / (e.sum(1, keepdim=True) if renormalize else torch.exp(l - top).sum(1, keepdim=True))
    s = torch.sigmoid(mine)
    total = s.sum(1, keepdim=True)
    return torch.where(total > 0, s / total, 0.0) if renormalize else s


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,experts,top_k", [(5, 3, 2), (7, 40, 6), (2061, 40, 8), (9, 250, 8), (2061, 250, 8), (6, 700, 20)])
def test_without_a_bias_the_order_is_the_logits(tokens, experts, top_k, kind):
    """Also where their scores are all 0 or all 1."""
    say(f"[gate far] {tokens} tokens, {experts} experts, {kind}")
    logits = _far(tokens, experts, kind)
    want = _largest(logits, top_k)
    for scores in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            ids, probs = _gate(logits, top_k, scores=scores, renormalize=renormalize, scale=2.0)
            assert torch.equal(ids.long(), want)
            p = 2 * _weights(logits, ids, scores, renormalize)
            ref.check(probs, p, ref.rounded(p, p.abs() * gated.WIDE, torch.float32), "probs")
        # one group a expert of several, all of them kept, or those of the largest logits
        if experts % 5 == 0:
            ids, _ = _gate(logits, top_k, scores=scores, groups=5, group_top=2)
            assert torch.equal(ids.long(), want)
            kept = 2
            worth = logits.double().view(tokens, 5, -1).amax(2)
            inside = torch.zeros(tokens, 5, dtype=torch.bool).scatter_(1, _largest(worth, kept), True)
            hidden = torch.where(inside.repeat_interleave(experts // 5, 1), logits.double(), -INF)
            few = min(top_k, 2)
            rows = (hidden > -INF).sum(1) >= few
            ids, _ = _gate(logits, few, scores=scores, groups=5, top_groups=kept)
            assert torch.equal(ids.long()[rows], _largest(hidden, few)[rows])


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_the_router_has_one_order(scores):
    """Arguments that have nothing to do with the choice leave it as it is."""
    rows = torch.tensor([[1000.0, 1, 5, -3], [-2000, 900, -1536, 40], [64, 66, 72, 70], [0, -900, -800, -1000]])
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    x[:, :4] = torch.eye(4)
    router = torch.zeros(4, 8, dtype=torch.bfloat16)
    router[:, :4] = rows.t()
    assert torch.equal((x.double() @ router.double().t()), rows.double())
    want = _largest(rows, 3).to(torch.int32)
    for renormalize in (False, True):
        plain = None
        for how in (dict(), dict(scale=2.5), dict(groups=2), dict(groups=2, group_top=2), dict(group_top=2)):
            ids, probs = torch.empty(4, 3, dtype=torch.int32, device=DEV), torch.empty(4, 3, device=DEV)
            moe_route(x.to(DEV), router.to(DEV), ids, probs, scores=scores, renormalize=renormalize, **how)
            assert torch.equal(ids.cpu(), want), (how, ids)
            probs = probs / how.get("scale", 1.0)
            plain = probs if plain is None else plain
            assert torch.allclose(probs, plain, rtol=2.0 ** -22, atol=0)


def test_not_a_number_comes_first():
    logits = torch.full((2, 6), -900.0)
    logits[:, 4] = 10.0
    logits[0, 2] = float("nan")
    ids, _ = _gate(logits, 2, scores="sigmoid")
    assert ids.tolist() == [[2, 4], [4, 0]]


# sums of sigmoid scores between fp64's smallest number and 2^-840
@pytest.mark.parametrize("tokens,experts", [(6, 30), (6, 200), (2060, 30), (2060, 200), (6, 600)])
def test_sigmoid_near_the_end_of_fp64(tokens, experts):
    """There s = e^l within fp64, and the renormalised weights are the softmax of the chosen logits; the
    gradient is that of these weights."""
    g = torch.Generator().manual_seed(tokens + experts)
    logits = torch.randn(tokens, experts, generator=g) * 2
    logits[::2] -= torch.linspace(590, 738, len(logits[::2]))[:, None]
    how = dict(scores="sigmoid", renormalize=True, scale=1.5)
    far = torch.arange(0, tokens, 2)
    up = torch.randn(tokens, 5, generator=g)
    for bias in (None, torch.randn(experts, generator=g)):
        ids, probs = _gate(logits, 5, bias=None if bias is None else bias.to(DEV), **how)
        mine = logits.double().gather(1, ids.long())
        s = torch.sigmoid(mine)
        p = s / s.sum(1, keepdim=True)
        p[far] = torch.softmax(mine[far], 1)
        v = p * 1.5
        ref.check(probs, v, ref.rounded(v, v.abs() * gated.WIDE, torch.float32), "probs")
        got = moe_gate_bwd(logits.to(DEV), ids.to(DEV), up.to(DEV), torch.empty_like(logits, device=DEV), **how)
        u = 1.5 * up.double()
        mass = p * (u.abs() + (u * p).abs().sum(1, keepdim=True)) * torch.sigmoid(-mine)
        want = torch.zeros(tokens, experts, dtype=torch.float64)
        want.scatter_(1, ids.long(), p * (u - (u * p).sum(1, keepdim=True)) * torch.sigmoid(-mine))
        loss = torch.zeros_like(want).scatter_(1, ids.long(), mass * gated.WIDE)
        ref.check(got, want, ref.rounded(want, loss, torch.float32), "grad_logits")
        leaf = logits.to(DEV).requires_grad_()
        again, _ = MoeGate.apply(leaf, 5, None if bias is None else bias.to(DEV), "sigmoid", 1, None, 1, True, 1.5)
        again.backward(up.to(DEV))
        assert torch.equal(again.detach().cpu(), probs) and torch.equal(leaf.grad, got)
