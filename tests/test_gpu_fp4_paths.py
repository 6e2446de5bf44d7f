"""The variants of the expert layer with weights in 4 bits, each at sizes that take it, against 64
bits: waves that share columns and waves that split k, one to four groups of columns and more than
they hold, several units a workgroup, ragged ends; and operands past 2^31 and 2^32 elements."""
import pytest
import torch

import block_reference as ref
from memory_bound_elementwise_amd import (fp4_dequantize, fp4_pack, fp4_quantize, fp4_shapes, linear_act, linear_act_fp4,
                                          moe_experts_fp4, moe_gate_bwd, moe_gate_fwd)
from parity import say
from test_gpu_fp4_products import _check_experts, _choice, _layer, _normal, _weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _skewed(tokens, experts, top_k, seed):
    """Most tokens at the first few experts, some experts with none."""
    g = torch.Generator().manual_seed(seed)
    ids = (torch.rand(tokens, top_k, generator=g) ** 4 * experts).to(torch.int32)
    return ids


# (hidden, inter, experts): which of the two products has waves that share columns
@pytest.mark.parametrize("hidden,inter,experts,top_k", [(1056, 288, 64, 8), (512, 1056, 64, 8), (1312, 1184, 40, 4), (2080, 96, 32, 2)])
@pytest.mark.parametrize("tokens", [2, 3, 16, 40])
def test_shared_columns(tokens, hidden, inter, experts, top_k):
    _check_experts(tokens, hidden, inter, experts, top_k, "swiglu", 7.0)
    _check_experts(tokens, hidden, inter, experts, top_k, "squared_relu", dtype=torch.float32, residual=False,
                   ids=_skewed(tokens, experts, top_k, tokens))


@pytest.mark.parametrize("tokens,top_k", [(64, 8), (128, 8), (256, 4), (1024, 1)])
def test_one_expert_has_them_all(tokens, top_k):
    """More tokens than four groups of columns hold; their weights are read again."""
    for inter in (64, 224):
        ids = torch.full((tokens, top_k), 300, dtype=torch.int32)
        ids[:, top_k // 2:] = torch.arange(tokens * (top_k - top_k // 2)).view(tokens, -1).to(torch.int32) % 310 + 90
        _check_experts(tokens, 96, inter, 400, top_k, "swiglu", 7.0, ids=ids)


@pytest.mark.parametrize("tokens", [1, 5, 9])
def test_top_k_of_sixty_four(tokens):
    """As many pairs as one workgroup adds up, and more."""
    _check_experts(tokens, 64, 64, 64, 64, "squared_relu")


# inter of 16 steps and more, in two, four and eight parts, the last one shorter or not
@pytest.mark.parametrize("inter", [2048, 2080, 2176, 4224, 8192, 8224])
@pytest.mark.parametrize("tokens", [9, 40])
def test_down_in_parts(tokens, inter):
    _check_experts(tokens, 96, inter, 8, 4, "squared_relu")
    ids = _skewed(tokens, 8, 4, inter)
    ids[3] = -1
    ids[5:7, 1:] = 8
    _check_experts(tokens, 544, inter, 8, 4, "swiglu", 7.0, dtype=torch.float32, residual=False, ids=ids)


@pytest.mark.parametrize("valid", [0, 5, 20])
def test_down_in_parts_of_some_tokens(valid):
    g = torch.Generator().manual_seed(valid)
    tokens, hidden, inter, experts, top_k = 20, 96, 4224, 8, 4
    (_, wu), (_, wd) = _layer(g, experts, hidden, inter, "swiglu")
    x, (ids, probs) = _normal(g, tokens, hidden).to(DEV), (t.to(DEV) for t in _choice(g, tokens, experts, top_k))
    whole = moe_experts_fp4(x, *wu, *wd, ids, probs, torch.empty(tokens, hidden, device=DEV), limit=7.0)
    x[valid:] = float("nan")
    ids[valid:] = 1 << 30
    y = torch.full((tokens, hidden), 77.0, device=DEV)
    moe_experts_fp4(x, *wu, *wd, ids, probs, y, limit=7.0, valid_tokens=torch.tensor([valid], dtype=torch.int32, device=DEV))
    assert torch.equal(y[:valid], whole[:valid]) and (y[valid:] == 77).all()


def test_bits_do_not_depend_on_the_batch():
    """A token's bits in a batch of one composition are those in another of the same sizes."""
    g = torch.Generator().manual_seed(3)
    tokens, hidden, inter, experts, top_k = 24, 1056, 288, 64, 8
    (_, wu), (_, wd) = _layer(g, experts, hidden, inter, "swiglu")
    x, (ids, probs) = _normal(g, tokens, hidden), _choice(g, tokens, experts, top_k)

    def run(x, ids):
        return moe_experts_fp4(x.to(DEV), *wu, *wd, ids.to(DEV), probs.to(DEV), torch.empty(tokens, hidden, device=DEV), limit=7.0)
    whole = run(x, ids)
    x2, ids2 = x.clone(), ids.clone()
    x2[::2] = 3
    ids2[::2] = ids[1]
    assert torch.equal(run(x2, ids2)[1::2], whole[1::2])


@pytest.mark.parametrize("m", [1, 7, 40, 300])
def test_the_same_as_wide_weights(m):
    """The product with the weights' bf16 values is the same sum in another order."""
    g = torch.Generator().manual_seed(m)
    w = torch.randn(264, 1056, generator=g).to(BF).to(DEV)
    codes, scales = (torch.empty(s, dtype=torch.uint8, device=DEV) for s in fp4_shapes(264, 1056))
    fp4_quantize(w, codes, scales)
    wide = fp4_dequantize(codes, scales, torch.empty_like(w))
    x = _normal(g, m, 1056).to(DEV)
    a = linear_act_fp4(x, codes, scales, torch.empty(m, 264, dtype=BF, device=DEV)).double()
    b = linear_act(x, wide, torch.empty(m, 264, dtype=BF, device=DEV)).double()
    # each is within its sum's loss (2 k 2^-24 of the terms) and half a step of the exact value
    mass = x.double().abs() @ wide.double().abs().t()
    lim = 2 * (2 * 1056 * ref.U * mass) + (a.abs() + b.abs()) * ref.half_step(BF) * (1 + 2.0 ** -7)
    assert ((a - b).abs() <= lim).all()


def test_long_k():
    """A sum of 2^15 terms a row through every variant of the product."""
    g = torch.Generator().manual_seed(9)
    k = 1 << 15
    v, w = _weights(g, 24, k, std=k ** -0.5)
    for m in (1, 6, 20, 70):
        say(f"[linear_fp4] m {m} n 24 k {k}")
        x = _normal(g, m, k)
        y = linear_act_fp4(x.to(DEV), *w, torch.empty(m, 24, dtype=BF, device=DEV))
        want, bound, _ = ref.linear_act(x.double(), v, None, "none", None, BF)
        ref.check(y, want, bound, f"linear {m}")


# ---------------------------------------------------------------------------
# Far ends of large operands: the same call over a view of the end gives the same bits
# ---------------------------------------------------------------------------
def _pair(experts, n, k):
    return [torch.empty(experts, *s, dtype=torch.uint8, device=DEV) for s in fp4_shapes(n, k)]


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_weights_past_32_bits(dtype):
    experts, n, k = 136, 8192, 4096  # 4.56e9 elements
    w = torch.empty(experts, n, k, dtype=dtype, device=DEV)
    for e in range(experts):
        w[e].normal_()
    whole, end = _pair(experts, n, k), _pair(2, n, k)
    fp4_quantize(w, *whole)
    fp4_quantize(w[-2:], *end)
    for a, b in zip(whole, end):
        assert torch.equal(a[-2:], b)
        assert not torch.equal(a[-1], a[7])  # 7 = 135 - 2^32 / (8192 x 4096)
    del w
    wide = torch.empty(experts, n, k, dtype=BF, device=DEV)
    fp4_dequantize(*whole, wide)
    assert torch.equal(wide[-2:], fp4_dequantize(*end, torch.empty(2, n, k, dtype=BF, device=DEV)))
    pairs = torch.randint(0, 256, (experts, n, k // 2), dtype=torch.uint8, device=DEV)
    exponents = torch.randint(120, 130, (experts, n, k // 32), dtype=torch.uint8, device=DEV)
    fp4_pack(pairs, exponents, *whole)
    fp4_pack(pairs[-2:], exponents[-2:], *end)
    for a, b in zip(whole, end):
        assert torch.equal(a[-2:], b)


@pytest.mark.parametrize("tokens,top_k", [(1, 4), (2, 8), (24, 8)])
def test_experts_past_32_bits(tokens, top_k):
    experts, hidden, inter = 160, 4096, 8192  # the codes of up_* are 5.4e9 bytes
    g = torch.Generator().manual_seed(tokens)
    wu, wd = _pair(experts, 2 * inter, hidden), _pair(experts, hidden, inter)
    for codes, scales in (wu, wd):
        codes.random_(0, 256)
        scales.random_(118, 122)
    x, ids, probs = _normal(g, tokens, hidden).to(DEV), *(t.to(DEV) for t in _choice(g, tokens, 16, top_k))

    def run(wu, wd, ids):
        return moe_experts_fp4(x, *wu, *wd, ids, probs, torch.empty(tokens, hidden, device=DEV), limit=7.0)
    y = run(wu, wd, ids + (experts - 16))
    assert torch.isfinite(y).all() and (y != 0).any()
    # the same experts at the front of a layer of the same sizes, which so takes the same variant
    assert torch.equal(y, run([t.roll(16, 0) for t in wu], [t.roll(16, 0) for t in wd], ids))


def test_linear_past_32_bits():
    m, n, k = 65544, 65544, 64  # y has 4.3e9 elements
    codes, scales = (t[0] for t in _pair(1, n, k))
    codes.random_(0, 256)
    scales.random_(118, 122)
    w = fp4_dequantize(codes, scales, torch.empty(n, k, dtype=BF, device=DEV)).double()
    x = torch.randn(m, k, device=DEV).to(BF)
    y = linear_act_fp4(x, codes, scales, torch.empty(m, n, dtype=BF, device=DEV))
    for at in (0, 32760, 65536 - 40, m - 300):
        rows = x[at:at + 300].double()
        want, mass = rows @ w.t(), rows.abs() @ w.abs().t()
        lim = 2 * k * ref.U * mass + want.abs() * ref.half_step(BF) * (1 + 2.0 ** -7)
        assert ((y[at:at + 300].double() - want).abs() <= lim).all()


@pytest.mark.parametrize("experts", [256, 512])
def test_gate_past_32_bits(experts):
    tokens, top_k = min((1 << 32) // experts + 1029, 1 << 24), 4  # 2^32 logits and more
    logits = torch.empty(tokens, experts, dtype=BF, device=DEV)
    for part in logits.split(1 << 20):
        part.normal_()
    ids = torch.empty(tokens, top_k, dtype=torch.int32, device=DEV)
    probs, grads = torch.empty(tokens, top_k, device=DEV), torch.randn(tokens, top_k, device=DEV)
    moe_gate_fwd(logits, ids, probs, renormalize=True)
    dx = moe_gate_bwd(logits, ids, grads, torch.empty_like(logits), renormalize=True)
    for at in (0, (1 << 31) // experts - 700, tokens - 2100):
        rows = slice(at, at + 2100)
        i, p = torch.empty_like(ids[rows]), torch.empty_like(probs[rows])
        moe_gate_fwd(logits[rows], i, p, renormalize=True)
        assert torch.equal(i, ids[rows]) and torch.equal(p, probs[rows])
        part = moe_gate_bwd(logits[rows], i, grads[rows], torch.empty_like(logits[rows]), renormalize=True)
        assert torch.equal(part, dx[rows])
