"""The gate behind the router's product beyond its plain forms: renormalised softmax weights, tokens past
the valid ones, a prompt's tokens, and chosen experts far below the largest; against 64 bits
(gated_reference)."""
import pytest
import torch

import block_reference as ref
import gated_reference as gated
from memory_bound_elementwise_amd import moe_route
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")


def _inputs(tokens, hidden, experts, kind=torch.bfloat16):
    g = torch.Generator().manual_seed(tokens + hidden + experts)
    x = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    router = (torch.randn(experts, hidden, generator=g) * 1.5 * hidden ** -0.5).to(kind)
    return x, router, torch.randn(experts, generator=g) * 0.1


def _route(x, router, top_k, **how):
    """Rows in front of and behind the outputs must stay as they are."""
    ids = torch.full((len(x) + 2, top_k), -7, dtype=torch.int32, device=DEV)
    probs = torch.full((len(x) + 2, top_k), -7.0, device=DEV)
    moe_route(x.to(DEV), router.to(DEV), ids[1:-1], probs[1:-1],
              **{k: v.to(DEV) if torch.is_tensor(v) else v for k, v in how.items()})
    torch.cuda.synchronize()
    assert (ids[[0, -1]] == -7).all() and (probs[[0, -1]] == -7).all()
    return ids[1:-1].cpu(), probs[1:-1].cpu()


def _check(x, router, top_k, logits=None, **how):
    ids, probs = _route(x, router, top_k, **how)
    logits = x.double() @ router.double().t() if logits is None else logits
    want, (p, bound) = gated.gate(logits, top_k, **how)
    assert torch.equal(ids, want)
    ref.check(probs, p, bound, "probs")
    return ids, probs


# the experts a lane holds on both sides of each border, tokens of a wave each and more of them
@pytest.mark.parametrize("tokens", [1, 6, 70, 2055, 2300])
@pytest.mark.parametrize("experts,top_k,groups,top_groups", [(8, 2, 1, 1), (64, 6, 8, 3), (65, 3, 5, 2), (256, 8, 8, 4), (320, 8, 4, 2)])
def test_renormalised_softmax(tokens, experts, top_k, groups, top_groups):
    say(f"[route] {tokens} tokens, {experts} experts, {groups} groups")
    x, router, bias = _inputs(tokens, 136, experts)
    group_top = 2 if groups > 1 else 1
    how = dict(scores="softmax", renormalize=True, groups=groups, top_groups=top_groups)
    _check(x, router, top_k, bias=bias, group_top=group_top, **how)
    _check(x, router, top_k, scale=2.5, group_top=1, **how)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,experts", [(2049, 48), (2600, 64), (2049, 96), (2601, 256), (2049, 400)])
def test_a_prompt(tokens, experts, kind):
    """More tokens than take a wave each, in every variant."""
    say(f"[route] {tokens} tokens, {experts} experts, {kind}")
    x, router, bias = _inputs(tokens, 264, experts, kind)
    _check(x, router, 8, scores="sigmoid", bias=bias, groups=4, top_groups=2, group_top=2, renormalize=True, scale=2.5)
    _check(x, router, 5, scores="softmax", bias=bias)


@pytest.mark.parametrize("valid", [-2, 0, 1, 3, 19, 20, 77])
def test_valid_tokens(valid):
    v = torch.tensor([valid], dtype=torch.int32)
    for tokens, experts in ((3, 64), (20, 64), (20, 256), (20, 300), (2100, 64), (2100, 200)):
        x, router, bias = _inputs(tokens, 72, experts)
        n = min(max(valid, 0), tokens)
        how = dict(scores="sigmoid", bias=bias, groups=4, top_groups=3, group_top=2, renormalize=True)
        whole = _route(x, router, 4, **how)
        x[n:] = float("nan")                                 # behind the end: whatever they say
        ids, probs = _route(x, router, 4, valid_tokens=v, **how)
        assert torch.equal(ids[:n], whole[0][:n]) and torch.equal(probs[:n], whole[1][:n])
        assert (ids[n:] == -7).all() and (probs[n:] == -7).all()


# hidden of one part of k and of several
@pytest.mark.parametrize("hidden", [8, 4096])
@pytest.mark.parametrize("tokens,experts", [(5, 24), (5, 200), (2060, 40), (2060, 200), (5, 600)])
def test_chosen_far_below_the_largest(tokens, experts, hidden):
    """A bias that keeps the largest logits out: the chosen experts' weights are the softmax of their own
    logits, also where their scores among all experts are past fp64's end."""
    g = torch.Generator().manual_seed(tokens + experts)
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16)
    router = torch.zeros(experts, hidden, dtype=torch.bfloat16)
    # the logits are x[:, 0] router[:, 0] + x[:, 1] router[:, 1], of the first four experts large
    x[:, 0] = torch.randn(tokens, generator=g).to(torch.bfloat16)
    x[:, -1] = torch.tensor([0.0, 1.0, 0.75])[torch.arange(tokens) % 3]
    router[:, 0] = torch.randn(experts, generator=g).to(torch.bfloat16)
    router[:4, -1] = torch.tensor([600.0, 800.0, 1000.0, 2.0 ** 40])
    bias = torch.randn(experts, generator=g) * 0.1
    bias[:4] = -INF
    ids, probs = _check(x, router, 6, bias=bias, scores="softmax", renormalize=True, scale=2.0)
    assert (ids > 3).all() and (probs.sum(1) - 2).abs().max() < 1e-6
