"""Infinite weights in 4 bits (bytes 253 and 254 of the exponent with the larger elements) through
every form of the expert layer: an infinity of the product's sign, however few bits the activation
has, and NaN where the sum in 64 bits has one."""
import pytest
import torch

from memory_bound_elementwise_amd import fp4_pack, fp4_shapes, moe_experts_fp4
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
INF = float("inf")

# tokens, experts, top_k, hidden, inter: a pair at a time, in one part of k and in four; five pairs at a
# time; by expert with one and with several groups of columns; by expert in parts of k
FORMS = [(1, 8, 2, 64, 64), (1, 4, 2, 64, 1056), (6, 16, 2, 96, 64), (9, 4, 3, 64, 288), (40, 16, 4, 96, 64), (70, 3, 2, 64, 96),
         (40, 8, 4, 96, 2176)]


def _pack(codes, exponents):
    lead, (n, k) = codes.shape[:-2], codes.shape[-2:]
    to = [torch.empty(*lead, *s, dtype=torch.uint8, device=DEV) for s in fp4_shapes(n, k)]
    pairs = codes[..., 0::2] | codes[..., 1::2] << 4
    fp4_pack(pairs.contiguous().to(DEV), exponents.contiguous().to(DEV), *to)
    return to


def _values(codes, exponents):
    """In 64 bits, infinite past bf16's range."""
    level = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    v = level[codes.long()] * (2.0 ** (exponents.double() - 127)).repeat_interleave(32, -1)
    return torch.where(v.abs() > torch.finfo(BF).max, v.sign() * INF, v)


def _exact(x, up, down, ids, probs):
    """Squared ReLU; each product and sum as 64 bits have them, infinities and NaN included."""
    y = torch.zeros(x.shape[0], down.shape[1], dtype=torch.float64)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            z = up[e][:, 0] * x[t, 0]                      # the other elements of x are zeros
            h = z.clamp(min=0) ** 2 * probs[t, j]
            y[t] += (down[e] * h).sum(1)
    return y


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", FORMS)
@pytest.mark.parametrize("byte,codes_past", [(253, (6, 7)), (254, (4, 5, 6, 7))])
def test_infinite_down_weights(tokens, experts, top_k, hidden, inter, byte, codes_past):
    say(f"[fp4 infinite] {tokens} tokens, {experts} experts, top {top_k}, {hidden} x {inter}, byte {byte}")
    g = torch.Generator().manual_seed(tokens + byte)

    def pick(values, *shape):
        return torch.tensor(values)[torch.randint(0, len(values), shape, generator=g)]
    ids = torch.stack([torch.randperm(experts, generator=g)[:top_k] for _ in range(tokens)]).to(torch.int32)
    # of one bit, of two, of all 24
    probs = pick([1.0, 0.75, 1.0 / 3, 2.0 ** -20], tokens, top_k)
    x = torch.zeros(tokens, hidden, dtype=BF)
    x[:, 0] = 1.0
    up = torch.zeros(experts, inter, hidden, dtype=torch.uint8)
    up_exp = torch.full((experts, inter, hidden // 32), 127, dtype=torch.uint8)
    down = torch.randint(0, 16, (experts, hidden, inter), generator=g, dtype=torch.uint8)
    down_exp = torch.randint(125, 129, (experts, hidden, inter // 32), generator=g, dtype=torch.uint8)
    rows = torch.arange(0, hidden, 3)
    down[:, rows, :32] = 0                                 # a group that is infinite at one place or two
    at = torch.randint(0, 32, (experts, len(rows)), generator=g)
    past = pick(codes_past, experts, len(rows), 1).to(torch.uint8)
    past[:, 1::3] += 8                                     # negative in some rows
    down[:, rows] = down[:, rows].scatter(2, at[..., None], past)
    down[:, rows[2::3], 5] = codes_past[0] + 8             # of both signs in others
    down_exp[:, rows, 0] = byte

    def both(up, up_exp, probs):
        y = moe_experts_fp4(x.to(DEV), *_pack(up, up_exp), *_pack(down, down_exp), ids.to(DEV), probs.to(DEV),
                            torch.empty(tokens, hidden, dtype=torch.float32, device=DEV), activation="squared_relu")
        want = _exact(x.double(), _values(up, up_exp), _values(down, down_exp), ids, probs.double())
        y = y.cpu().double()
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        there = torch.isinf(want)
        assert torch.equal(torch.where(there, y, 0.0), torch.where(there, want, 0.0))
        assert torch.isfinite(y[torch.isfinite(want)]).all()
        return want

    up[:, :, 0] = pick([10, 0, 2, 4, 5], experts, inter).to(torch.uint8)          # -1, 0, 1, 2, 3
    both(up, up_exp, probs)                                # 0 times an infinity among them
    up[:, :, 0] = pick([2, 4, 5], experts, inter).to(torch.uint8)
    want = both(up, up_exp, probs)
    assert (want == INF).any() and (want == -INF).any() and torch.isnan(want).any()
    both(up, up_exp, -probs)
    # an infinite weight of the up product: the activation is infinite
    down_exp[:] = 127
    down[:] = down % 8
    down[:, :, ::7] = 2
    up_exp[:, ::5, 0] = byte
    up[:, ::5, 0] = codes_past[0]
    want = both(up, up_exp, probs)
    assert not torch.isfinite(want).any()
