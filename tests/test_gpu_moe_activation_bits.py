"""The expert layer's activations keep the 24 bits of fp32 on their way through the down product."""
import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import moe_experts
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16

# tokens, experts, slots: both forms of the down product, with one, two and four groups of
# eight tokens to an expert, four and eight waves
FORMS = [(1, 4, 1), (12, 1, 1), (40, 1, 1), (3, 7, 2), (64, 64, 2), (64, 16, 2), (128, 8, 1), (128, 16, 1), (128, 64, 1),
         (200, 5, 1)]


def _ids(tokens, experts, slots, g):
    """One expert a token; its other slots are empty."""
    ids = torch.full((tokens, slots), -1, dtype=torch.int32)
    ids[torch.arange(tokens), torch.randint(0, slots, (tokens,), generator=g)] = \
        torch.randint(0, experts, (tokens,), generator=g, dtype=torch.int32)
    return ids


@pytest.mark.parametrize("width", [40, 136, 1032])
@pytest.mark.parametrize("tokens,experts,slots", FORMS)
def test_activation_keeps_24_bits(tokens, experts, slots, width):
    """x has one power of two a token and w_down one a row, so z, and h times w_down, are exact:
    y is h = z^2 p itself, one fp32 rounding of a square of 16 bits times a weight of 24, bit
    for bit."""
    say(f"[activation bits] {tokens} tokens, {experts} experts, {slots} slots, {width}")
    g = torch.Generator().manual_seed(tokens + width)
    ids = _ids(tokens, experts, slots, g)
    probs = torch.rand(tokens, slots, generator=g) + 0.01
    x = torch.zeros(tokens, width, dtype=BF)
    x[:, 0] = 2.0 ** torch.randint(-3, 4, (tokens,), generator=g)
    wu = torch.zeros(experts, width, width, dtype=BF)
    wu[:, :, 0] = torch.randn(experts, width, generator=g).to(BF)
    scale = 2.0 ** torch.randint(-2, 3, (experts, width), generator=g) * (torch.rand(experts, width, generator=g) - 0.5).sign()
    wd = torch.diag_embed(scale).to(BF)
    y = moe_experts(x.to(DEV), wu.to(DEV), wd.to(DEV), ids.to(DEV), probs.to(DEV),
                    torch.empty(tokens, width, dtype=torch.float32, device=DEV), activation="squared_relu").cpu()
    at = ids.argmax(1)
    e, p = ids.gather(1, at[:, None])[:, 0].long(), probs.gather(1, at[:, None])
    z = (wu[e, :, 0].double() * x[:, :1].double()).clamp(min=0)
    h = (z * z * p.double()).float()               # exact in 64 bits: 16 + 24 bits
    assert torch.equal(y, h * scale[e].float())


def _experts64(x, wu, wd, ids, probs, act, limit):
    """(y, bound) in 64 bits; the bound is of fp32 arithmetic, with h in fp32 and its three terms
    in the down product's sums (twice as many products of a column, each good to 2 u)."""
    tokens, hidden = x.shape
    experts, _, inter = wd.shape
    y, dy, mass = (torch.zeros(tokens, hidden, dtype=torch.float64) for _ in range(3))
    for e in range(experts):
        t, j = torch.where(ids == e)
        if not t.numel():
            continue
        z, dz = ref.product(x[t], wu[e])
        if act == "swiglu":
            gate, up = z[:, :inter].clamp(max=limit), z[:, inter:].clamp(-limit, limit)
            s, ds = ref.activation("silu", gate, dz[:, :inter])
            h = s * up
            dh = ds * up.abs() + s.abs() * dz[:, inter:] + ds * dz[:, inter:] + ref.U * h.abs()
        else:
            h, dh = ref.activation("squared_relu", z, dz)
        p = probs[t, j][:, None]
        h, dh = h * p, (dh + ref.U * h.abs()) * p.abs()
        heavy = (h.abs() + dh) @ wd[e].abs().t()
        y.index_add_(0, t, h @ wd[e].t())
        dy.index_add_(0, t, dh @ wd[e].abs().t() + (4 * inter + 4) * ref.U * heavy)
        mass.index_add_(0, t, heavy)
    # a token's pairs, parts and shares one after the other
    dy += (ids.shape[1] * 16 + 4) * ref.U * mass
    return y, ref.rounded(y, dy, torch.float32)


@pytest.mark.parametrize("tokens,experts,slots", [(1, 4, 3), (9, 5, 3), (16, 2, 2), (40, 3, 2), (64, 16, 4), (100, 40, 4),
                                                  (128, 8, 3), (130, 6, 4)])
@pytest.mark.parametrize("hidden,inter", [(24, 8), (136, 24)])
@pytest.mark.parametrize("act", ["swiglu", "squared_relu"])
def test_fp32_output(tokens, experts, slots, hidden, inter, act):
    """Short sums, so that the bound is near fp32's own step."""
    say(f"[fp32 output] {tokens} tokens, {experts} experts, {slots} slots, {hidden} x {inter}, {act}")
    g = torch.Generator().manual_seed(tokens + hidden)
    x = torch.randn(tokens, hidden, generator=g).to(BF)
    ups = 2 * inter if act == "swiglu" else inter
    wu = (torch.randn(experts, ups, hidden, generator=g) * 2 * hidden ** -0.5).to(BF)
    wd = (torch.randn(experts, hidden, inter, generator=g) * inter ** -0.5).to(BF)
    ids = torch.randint(-1, experts, (tokens, slots), generator=g, dtype=torch.int32)
    probs = torch.rand(tokens, slots, generator=g)
    y = moe_experts(x.to(DEV), wu.to(DEV), wd.to(DEV), ids.to(DEV), probs.to(DEV),
                    torch.empty(tokens, hidden, dtype=torch.float32, device=DEV), activation=act, limit=1.5)
    v, bound = _experts64(x.double(), wu.double(), wd.double(), ids, probs.double(), act, 1.5)
    ref.check(y, v, bound, "fp32 output")


@pytest.mark.parametrize("tokens,experts,slots", FORMS)
def test_infinite_weights_and_activations(tokens, experts, slots):
    """An infinite weight of the down product gives an infinity of the activation's sign (NaN for
    an activation of 0), however few bits the activation has; an infinite activation likewise."""
    say(f"[infinite weights] {tokens} tokens, {experts} experts, {slots} slots")
    width, inf = 72, float("inf")
    g = torch.Generator().manual_seed(tokens)
    ids = _ids(tokens, experts, slots, g)
    probs = torch.tensor([1.0, -0.5, 1.0 / 3, -2.0 ** -20])[torch.randint(0, 4, (tokens, slots), generator=g)]
    x = torch.zeros(tokens, width, dtype=BF)
    x[:, 0] = 1.0
    wu = torch.zeros(experts, width, width, dtype=BF)
    wu[:, :, 0] = torch.randint(-1, 4, (experts, width), generator=g).to(BF)
    wd = torch.randn(experts, width, width, generator=g).to(BF)
    rows = torch.arange(0, width, 3)
    wd[:, rows, torch.randint(0, width, (len(rows),), generator=g)] = inf
    wd[:, rows[::2], 5] = -inf

    def both(w_up, p):
        y = moe_experts(x.to(DEV), w_up.to(DEV), wd.to(DEV), ids.to(DEV), p.to(DEV),
                        torch.empty(tokens, width, dtype=torch.float32, device=DEV), activation="squared_relu").cpu()
        at = ids.argmax(1)
        z = w_up[ids.gather(1, at[:, None])[:, 0].long(), :, 0].double().clamp(min=0)
        h = z * z * p.gather(1, at[:, None]).double()
        w = wd[ids.gather(1, at[:, None])[:, 0].long()].double()
        # elementwise in 64 bits; a sum with infinities of both signs, or 0 times one, is NaN
        want = (w * h[:, None, :]).sum(2)
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        there = torch.isinf(want)
        assert torch.equal(torch.where(there, y.double(), 0.0), torch.where(there, want, 0.0))
        assert torch.isfinite(y[torch.isfinite(want)]).all()
        return want

    want = both(wu, probs)
    assert torch.isinf(want).any() or tokens == 1
    positive = wu.clone()
    positive[:, :, 0] = positive[:, :, 0].clamp(min=1)
    assert torch.isinf(both(positive, probs)).any()
    wd = wd.nan_to_num(posinf=1.0, neginf=1.0).abs() + 1
    assert torch.isinf(both(positive, probs * inf)).all()


@pytest.mark.parametrize("tokens,experts,slots", [(64, 16, 4), (64, 64, 8), (128, 64, 8), (128, 16, 2)])
def test_same_bits_where_waves_share(tokens, experts, slots):
    """The waves of a workgroup share the activations' loads: every call gives the same bits, and
    a token with one expert the same whatever its place among the others."""
    say(f"[same bits] {tokens} tokens, {experts} experts, {slots} slots")
    hidden, inter = 2056, 1032
    g = torch.Generator(device=DEV).manual_seed(tokens + slots)
    x = torch.randn(tokens, hidden, generator=g, device=DEV).to(BF)
    wu = (torch.randn(experts, 2 * inter, hidden, generator=g, device=DEV) * 2 * hidden ** -0.5).to(BF)
    wd = (torch.randn(experts, hidden, inter, generator=g, device=DEV) * inter ** -0.5).to(BF)
    # one expert a token in its first slot, so that a row is one expert's sum alone
    ids = torch.full((tokens, slots), -1, dtype=torch.int32, device=DEV)
    ids[:, 0] = torch.randint(0, experts, (tokens,), generator=g, device=DEV, dtype=torch.int32)
    probs = torch.rand(tokens, slots, generator=g, device=DEV)

    def call(rows):
        return moe_experts(x[rows], wu, wd, ids[rows], probs[rows],
                           torch.empty(len(x[rows]), hidden, dtype=torch.float32, device=DEV), limit=7.0)

    want = call(slice(None))
    for _ in range(10):
        assert torch.equal(call(slice(None)), want)
    order = torch.randperm(tokens, generator=g, device=DEV)
    assert torch.equal(call(order), want[order])
    # every slot taken
    ids[:] = torch.randint(0, experts, ids.shape, generator=g, device=DEV, dtype=torch.int32)
    want = call(slice(None))
    for _ in range(10):
        assert torch.equal(call(slice(None)), want)
