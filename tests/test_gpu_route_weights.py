"""The router's softmax weights are fp64 rounded once."""
import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import moe_route
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("scale", [1.0, 6.0, 40.0])
@pytest.mark.parametrize("tokens,hidden,experts,top_k", [(1, 256, 64, 8), (3, 64, 6, 6), (4, 4096, 200, 20), (17, 264, 64, 64),
                                                         (40, 1000, 65, 3), (5, 64, 1024, 64), (130, 136, 256, 8)])
def test_weights_are_rounded_once(tokens, hidden, experts, top_k, scale):
    """scale spreads the logits, to about e^-100 between the first and the last chosen."""
    say(f"[route weights] {tokens} tokens, hidden {hidden}, {experts} experts, top {top_k}, scale {scale}")
    g = torch.Generator().manual_seed(tokens + experts)
    x = (torch.randn(tokens, hidden, generator=g) * scale).to(torch.bfloat16)
    for dtype in (torch.bfloat16, torch.float32):
        router = (torch.randn(experts, hidden, generator=g) * hidden ** -0.5).to(dtype)
        terms = x.double().abs() @ router.double().abs().t()
        # a logit is off by hidden 2^-53 of its terms; a weight by twice the largest such error of
        # its token, the differences' rounding and a few steps of fp64, then half a step of fp32
        loss = ref.U + 4 * hidden * 2.0 ** -53 * terms.max(1, keepdim=True).values + 2.0 ** -44
        for renorm in (False, True):
            want, (p, _) = ref.route(x.double(), router.double(), top_k, renorm)
            ids = torch.empty(tokens, top_k, dtype=torch.int32, device=DEV)
            probs = torch.empty(tokens, top_k, device=DEV)
            moe_route(x.to(DEV), router.to(DEV), ids, probs, renormalize=renorm)
            assert torch.equal(ids.cpu(), want)
            ref.check(probs, p, p * loss + 2.0 ** -149, "probs")
