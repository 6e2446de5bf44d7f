"""The gate's gradient to its last bit in 16-bit types, and nothing written beside it."""
import pytest
import torch

from memory_bound_elementwise_amd import moe_gate_bwd, moe_gate_fwd
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F16 = torch.bfloat16, torch.float16
INF = float("inf")
# bits of the significand, exponent of the smallest normal number
FORMAT = {BF: (8, -126), F16: (11, -14)}


def _round(v, kind):
    """v (double) to kind's nearest number, ties to even, in one step; as double. Also where the nearest
    two are closer than 2^-40 of a step to equally near: there the kernel's fp64 may take either."""
    bits, least = FORMAT[kind]
    power = torch.frexp(v)[1].to(torch.float64) - 1
    step = 2.0 ** (power.clamp(min=least) - (bits - 1))
    q = v / step                                            # a power of two: exact
    return torch.round(q) * step, ((q - torch.floor(q)) - 0.5).abs() < 2.0 ** -40 * (1 + q.abs())


@pytest.mark.parametrize("kind,short", [(BF, 8), (F16, 11)])
@pytest.mark.parametrize("renormalize", [False, True])
def test_one_rounding(kind, short, renormalize):
    """Gradients less than 2^-24 away from the middle between two numbers of the type: rounded to fp32 on
    the way they would be the middle itself, and go to the even neighbour."""
    step = 2.0 ** -short                                     # half the distance of numbers above 1
    # the products are 1 + step + step b - b^2 and 1 + 3 step - 3 step b - b^2
    b = 2.0 ** -18 if kind is BF else 2.0 ** -15
    cases = [(1 + step - b, 1 + b, 1 + 2 * step), (1 + 3 * step + b, 1 - b, 1 + 2 * step)]
    for g, scale, want in cases:
        exact = g * scale                                    # 48 bits
        assert 0 < abs(exact - (1 + step)) < 2.0 ** -24 or 0 < abs(exact - (1 + 3 * step)) < 2.0 ** -24
        assert torch.tensor(g).double().item() == g and torch.tensor(scale).double().item() == scale
        for sign in (1, -1):
            logits = torch.zeros(3, 5, dtype=kind, device=DEV)      # sigmoid: s = 1/2, ds/dl = 1/4
            ids = torch.tensor([[2, 4]] * 3, dtype=torch.int32, device=DEV)
            up = torch.tensor([[g * sign, 0.0]] * 3, device=DEV)
            out = moe_gate_bwd(logits, ids, up, torch.empty_like(logits), scores="sigmoid", renormalize=renormalize, scale=scale)
            # renormalised: p = 1/2, d = g - g / 2, times 1 - s
            part = 0.125 if renormalize else 0.25
            row = torch.zeros(5, dtype=torch.float64)
            row[2] = sign * want * part
            if renormalize:
                row[4] = -row[2]
            assert torch.equal(out.cpu().double(), row.repeat(3, 1)), (out, row)


@pytest.mark.parametrize("kind", [BF, F16])
def test_every_element_is_the_nearest(kind):
    """A million gradients against their 64-bit values."""
    g = torch.Generator().manual_seed(4)
    logits = (torch.randn(4096, 256, generator=g) * 2).to(kind)
    ids = torch.argsort(logits.double(), dim=1, descending=True)[:, :8].to(torch.int32).contiguous()
    up = torch.randn(4096, 8, generator=g) * 100
    out = moe_gate_bwd(logits.to(DEV), ids.to(DEV), up.to(DEV), torch.empty_like(logits, device=DEV))
    s = torch.softmax(logits.double(), 1)
    v = up.double() * s.gather(1, ids.long())
    want = -s * v.sum(1, keepdim=True)
    want.scatter_add_(1, ids.long(), v)
    nearest, middle = _round(want, kind)
    wrong = (out.cpu().double() != nearest) & ~middle
    # where terms cancel, fp64's own loss is more than the middle's margin
    mass = s * v.abs().sum(1, keepdim=True)
    mass.scatter_add_(1, ids.long(), v.abs())
    cancelled = want.abs() < mass * 2.0 ** -6
    assert int(cancelled.sum()) < want.numel() // 20
    assert int((wrong & ~cancelled).sum()) == 0


@pytest.mark.parametrize("kind", [BF, F16])
def test_range(kind):
    """Beyond the largest number an infinity, below the smallest a zero, subnormals in between."""
    largest, tiny = torch.finfo(kind).max, 2.0 ** (FORMAT[kind][1] - FORMAT[kind][0] + 1)  # the least subnormal
    past = largest * (1 + 2.0 ** -10) * (1 + 2.0 ** -8)              # past the middle to the next power of two
    for scale, values, want in ((2.0 ** 20, (largest, -largest, past, -past), (largest, -largest, INF, -INF)),
                                (1.0, (3 * tiny, -tiny, tiny / 2, -0.75 * tiny), (3 * tiny, -tiny, 0.0, -tiny))):
        logits = torch.zeros(1, 4, dtype=kind, device=DEV)
        ids = torch.arange(4, dtype=torch.int32, device=DEV)[None]
        up = torch.tensor([values], dtype=torch.float64) * 4 / scale
        out = moe_gate_bwd(logits, ids, up.float().to(DEV), torch.empty_like(logits), scores="sigmoid", scale=scale)
        assert out[0].tolist() == list(want)


# ragged widths, whose last rows end inside a vector
@pytest.mark.parametrize("tokens", [1, 2, 5, 131, 2055])
@pytest.mark.parametrize("experts,top_k", [(1, 1), (5, 5), (60, 6), (63, 4), (65, 3), (255, 8), (257, 9), (1001, 20)])
def test_nothing_beside_it_is_written(tokens, experts, top_k):
    say(f"[gate_bwd] {tokens} tokens, {experts} experts")
    if tokens > 1000 and experts > 256:
        tokens = 150
    for kind in (torch.float32, BF, F16):
        g = torch.Generator().manual_seed(tokens + experts)
        logits = torch.randn(tokens, experts, generator=g).to(kind).to(DEV)
        ids, probs = torch.empty(tokens, top_k, dtype=torch.int32, device=DEV), torch.empty(tokens, top_k, device=DEV)
        moe_gate_fwd(logits, ids, probs)
        n = tokens * experts
        for scores, renormalize in (("softmax", False), ("softmax", True), ("sigmoid", False)):
            flat = torch.full((n + 128,), 77.0, dtype=kind, device=DEV)
            moe_gate_bwd(logits, ids, probs, flat[64:64 + n].view(tokens, experts), scores=scores, renormalize=renormalize)
            assert (flat[:64] == 77).all() and (flat[64 + n:] == 77).all() and not (flat[64:64 + n] == 77).any()
            if tokens > 1:                                  # and behind the valid tokens
                flat.fill_(77)
                v = torch.tensor([tokens - 1], dtype=torch.int32, device=DEV)
                moe_gate_bwd(logits, ids, probs, flat[64:64 + n].view(tokens, experts), scores=scores,
                             renormalize=renormalize, valid_tokens=v)
                assert (flat[:64] == 77).all() and (flat[64 + n - experts:] == 77).all()
