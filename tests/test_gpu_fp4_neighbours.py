"""Weights in 4 bits next to groups of NaN: loads that run past a block of rows, a part of k or a matrix
must bring zeros, not what lies there (zero times NaN would show)."""
import pytest
import torch

from memory_bound_elementwise_amd import fp4_shapes, linear_act_fp4, moe_experts_fp4
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _weights(g, lead, n, k):
    codes, scales = (torch.empty(*lead, *s, dtype=torch.uint8) for s in fp4_shapes(n, k))
    codes.random_(0, 256, generator=g)
    scales.random_(118, 124, generator=g)
    return codes.to(DEV), scales.to(DEV)


@pytest.mark.parametrize("m", [1, 3, 9, 16, 17, 40, 70, 200])
@pytest.mark.parametrize("n,k", [(48, 32), (80, 160), (272, 288), (144, 1056), (48, 4224)])
def test_linear(m, n, k):
    say(f"[fp4 neighbours] {m} x {n} x {k}")
    g = torch.Generator().manual_seed(m + n + k)
    codes, scales = _weights(g, (), n, k)
    x = torch.randn(m, k, generator=g).to(BF).to(DEV)

    def run():
        return linear_act_fp4(x, codes, scales, torch.empty(m, n, dtype=BF, device=DEV)).view(m, -1, 16)
    clean = run()
    scales[1::2] = 255                                       # every second block of 16 rows
    y = run()
    assert torch.equal(y[:, ::2], clean[:, ::2]) and torch.isfinite(clean).all() and torch.isnan(y[:, 1::2]).all()


# tokens, experts, top_k, hidden, inter: each form of both products, k of one tile, of odd numbers of tiles, in parts
@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", [
    (1, 8, 2, 96, 32), (1, 4, 2, 160, 1056), (3, 16, 2, 288, 160), (9, 4, 3, 96, 288), (6, 16, 4, 1056, 96),
    (40, 16, 4, 96, 160), (70, 6, 2, 64, 96), (40, 64, 8, 416, 160), (40, 8, 4, 96, 2208), (12, 64, 8, 96, 1056),
    (140, 12, 4, 160, 288)])
@pytest.mark.parametrize("act", ["swiglu", "squared_relu"])
def test_experts(tokens, experts, top_k, hidden, inter, act):
    say(f"[fp4 neighbours] {tokens} tokens, {experts} experts, top {top_k}, {hidden} x {inter} {act}")
    g = torch.Generator().manual_seed(tokens + hidden + inter)
    up = _weights(g, (experts,), 2 * inter if act == "swiglu" else inter, hidden)
    down = _weights(g, (experts,), hidden, inter)
    x = torch.randn(tokens, hidden, generator=g).to(BF).to(DEV)
    probs = torch.rand(tokens, top_k, generator=g).to(DEV) + 0.1

    def run(ids):
        return moe_experts_fp4(x, *up, *down, ids, probs, torch.empty(tokens, hidden, device=DEV), activation=act, limit=7.0)
    ids = torch.stack([torch.randperm(experts, generator=g)[:top_k] for _ in range(tokens)]).to(torch.int32).to(DEV)
    clean = run(ids)
    kept = down[1].clone()
    down[1][:, 1::2] = 255                                   # every second block of 16 columns of the output
    y = run(ids)
    a, b = clean.view(tokens, -1, 16), y.view(tokens, -1, 16)
    assert torch.isfinite(clean).all() and torch.equal(b[:, ::2], a[:, ::2]) and torch.isnan(b[:, 1::2]).all()
    down[1].copy_(kept)
    # every second expert, of which some tokens have none
    some = ids.clone()
    some[::2] = some[::2] // 2 * 2
    clean = run(some)
    up[1][1::2] = 255
    down[1][1::2] = 255
    y = run(some)
    free = (some % 2 == 0).all(1)
    assert free[0] and torch.equal(y[free], clean[free])
    assert torch.isnan(y[~free]).all()
