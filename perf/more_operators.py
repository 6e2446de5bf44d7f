"""Cases for the operators that routing and 4-bit weights add to the Mixture-of-Experts block: the
gate (softmax or sigmoid scores, a bias for balance, groups of experts, top-k, renormalised
weights), its gradient, the router product in front of it, the quantiser of weights to 4 bits with
group scales, the product with such weights and the expert layer for a few tokens with such weights.

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits (the gate's
scores in 64, since its choice of experts is made between neighbouring values), rounded once at
the end. With ``own`` true it makes the calls of this package.

The 4-bit format is the open microscaling one: elements of a sign, two bits of exponent and one of
mantissa (0, 0.5, 1, 1.5, 2, 3, 4, 6), and a power of two, its exponent plus 127 in a byte, for each
32 neighbours of a row.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # a handful of decoded tokens over a small set of experts: latency
        {"name": "gate_few", "op": "gate", "tokens": 5, "experts": 64, "top_k": 6, "scores": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_top": 1, "renorm": False, "scale": 1.0, "type": "f32", "masked": False},
        # a training step's tokens, balanced by a bias and kept to half of the groups
        {"name": "gate_batch", "op": "gate", "tokens": 6720, "experts": 256, "top_k": 8, "scores": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "type": "f32",
         "masked": False},
        # the same step's backward
        {"name": "gate_bwd_batch", "op": "gate_bwd", "tokens": 6720, "experts": 256, "top_k": 8, "scores": "sigmoid",
         "renorm": True, "scale": 2.5, "type": "f32", "masked": False},
        # a ragged batch over an odd number of experts: every logit has a gradient
        {"name": "gate_bwd_odd", "op": "gate_bwd", "tokens": 1009, "experts": 60, "top_k": 6, "scores": "softmax",
         "renorm": False, "scale": 1.0, "type": "bf16", "masked": False},
        # one decoded token's routing at the model width: latency
        {"name": "route_token", "op": "route", "tokens": 1, "hidden": 7168, "experts": 256, "top_k": 8,
         "scores": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5,
         "masked": False},
        # a batch of decoded tokens
        {"name": "route_many", "op": "route", "tokens": 128, "hidden": 4096, "experts": 160, "top_k": 6,
         "scores": "softmax", "bias": False, "groups": 8, "top_groups": 3, "group_top": 1, "renorm": False,
         "scale": 16.0, "masked": False},
        # a small projection quantised and read back, rows that end inside a tile
        {"name": "quantize_small", "op": "quantize", "matrices": 1, "n": 1411, "k": 1408, "type": "bf16"},
        # the first products of eight experts, from fp32 master weights
        {"name": "quantize_experts", "op": "quantize", "matrices": 8, "n": 4096, "k": 7168, "type": "f32"},
        # a shared expert's first product for one decoded token: a weight stream
        {"name": "linear_token", "op": "linear", "m": 1, "k": 7168, "n": 4096, "act": "silu", "bias": True,
         "residual": False},
        # a ragged prompt through a shared expert's second product, added to the residual stream
        {"name": "linear_prompt", "op": "linear", "m": 1009, "k": 1408, "n": 7168, "act": "none", "bias": False,
         "residual": True},
        # one decoded token: eight experts' weights streamed once
        {"name": "experts_token", "op": "experts", "tokens": 1, "hidden": 7168, "inter": 2048, "experts": 64,
         "top_k": 8, "act": "swiglu", "limit": 7.0, "residual": True},
        # a decoding batch that reaches nearly every expert
        {"name": "experts_batch", "op": "experts", "tokens": 64, "hidden": 7168, "inter": 2048, "experts": 64,
         "top_k": 8, "act": "swiglu", "limit": 7.0, "residual": True},
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return int(max(lo, min(hi, v))) // step * step


def _draw_gate(rng):
    groups = rng.choice([1, 1, 2, 4, 8])
    size = _spread(rng, max(4, 8 // groups), 256 // groups)
    top_groups = rng.randint(1, groups)
    return {"experts": groups * size, "top_k": rng.randint(1, min(8, top_groups * size)),
            "scores": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
            "top_groups": top_groups, "group_top": rng.randint(1, 2), "renorm": rng.random() < 0.5,
            "scale": rng.choice([1.0, 2.5]), "masked": rng.random() < 0.2}


def draw(rng):
    op = rng.choice(["gate", "gate_bwd", "route", "quantize", "linear", "linear", "experts", "experts"])
    if op in ("gate", "gate_bwd"):
        g = _draw_gate(rng)
        if op == "gate_bwd":
            g = {key: g[key] for key in ("experts", "top_k", "scores", "renorm", "scale", "masked")}
        return {"op": op, "tokens": _spread(rng, 1, 6720), "type": rng.choice(["f32", "f32", "bf16", "f16"]), **g}
    if op == "route":
        return {"op": op, "tokens": _spread(rng, 1, 256), "hidden": _spread(rng, 128, 7168, 8), **_draw_gate(rng),
                "masked": False}
    if op == "quantize":
        return {"op": op, "matrices": rng.randint(1, 8), "n": _spread(rng, 16, 4096), "k": _spread(rng, 64, 7168, 32),
                "type": rng.choice(["bf16", "f16", "f32"])}
    if op == "linear":
        return {"op": op, "m": _spread(rng, 1, 1009), "k": _spread(rng, 128, 7168, 32), "n": _spread(rng, 128, 4096, 8),
                "act": rng.choice(["none", "silu", "gelu", "squared_relu"]), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5}
    act = rng.choice(["swiglu", "swiglu", "squared_relu"])
    return {"op": op, "tokens": _spread(rng, 1, 64), "hidden": _spread(rng, 128, 7168, 32),
            "inter": _spread(rng, 128, 2048, 32), "experts": _spread(rng, 8, 64), "top_k": rng.randint(1, 8),
            "act": act, "limit": rng.choice([7.0, math.inf]) if act == "swiglu" else math.inf,
            "residual": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# The 4-bit format, in elementary operations
# ---------------------------------------------------------------------------
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(w):
    """w [n, k] in 32 bits as elements (uint8 [n, k], a code each) and exponents (uint8 [n, k / 32])."""
    v = w.view(w.shape[0], -1, GROUP)
    top = v.abs().amax(2)
    part, power = torch.frexp(top)  # top = part 2^power, part in [0.5, 1)
    # the smallest power of two whose largest element, 6, is the nearest one to all of the group
    power = (power - 3 + (part >= 0.875)).clamp(-127, 125)
    v = torch.ldexp(v, -power[..., None])
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(v)).to(torch.uint8)  # ties went to the even code
    return code.view(w.shape), (power + 127).to(torch.uint8)


def _pairs(code):
    """Two elements a byte, the first in its lower half."""
    return code[..., 0::2] | code[..., 1::2] << 4


def _values(elements, exponents):
    """The weights of packed elements [..., n, k / 2] and exponents [..., n, k / 32], in 32 bits."""
    level = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), device=elements.device)
    codes = torch.stack((elements & 15, elements >> 4), -1).flatten(-2)
    scale = torch.exp2(exponents.float() - 127.0)
    return level[codes.int()] * scale.repeat_interleave(GROUP, -1)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0, kind="bf16"):
        t = torch.randn(*shape, generator=g, device=DEV, dtype=TYPES[kind])
        return t.mul_(std) if std != 1.0 else t

    def weights(matrices, n, k, std):
        """Weights as a checkpoint holds them, or laid out for the package's kernels."""
        if own:
            import memory_bound_elementwise_amd as mbe
            shapes = mbe.fp4_shapes(n, k)
            out = [torch.empty(matrices, *shape, dtype=torch.uint8, device=DEV) for shape in shapes]
        else:
            out = [torch.empty(matrices, n, k // (2 if i == 0 else GROUP), dtype=torch.uint8, device=DEV) for i in (0, 1)]
        for i in range(matrices):
            codes, exponents = _quantize(normal(n, k, std=std, kind="f32"))
            if own:
                mbe.fp4_pack(_pairs(codes), exponents, out[0][i], out[1][i])
            else:
                out[0][i], out[1][i] = _pairs(codes), exponents
        return out

    s = dict(case)
    op = case["op"]
    if op in ("gate", "gate_bwd", "route"):
        t, e = case["tokens"], case["experts"]
        s["bias_v"] = normal(e, std=0.1, kind="f32") if case.get("bias") else None
        if op == "route":
            s["x"] = normal(t, case["hidden"])
            s["router"] = normal(e, case["hidden"], std=1.5 / math.sqrt(case["hidden"]))
            return s
        logits = normal(t, e, std=1.5, kind="f32")
        if case["masked"]:  # experts that are not there to be had, a tenth of them
            logits[:, torch.rand(e, generator=g, device=DEV) < 0.1] = -math.inf
        s["logits"] = logits.to(TYPES[case["type"]])
        if op == "gate_bwd":  # what the forward chose
            order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)[1]
            s["ids"] = order[:, :case["top_k"]].to(torch.int32).contiguous()
            s["grad_probs"] = normal(t, case["top_k"], kind="f32")
    elif op == "quantize":
        w = normal(case["matrices"], case["n"], case["k"], std=1 / math.sqrt(case["k"]), kind="f32")
        s["w"] = w.to(TYPES[case["type"]])
    elif op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = normal(m, k)
        s["w"] = [t[0] for t in weights(1, n, k, 1 / math.sqrt(k))]
        s["bias_v"] = normal(n, std=0.5) if case["bias"] else None
        s["res"] = normal(m, n) if case["residual"] else None
    else:
        t, h, inter, e, k = (case[key] for key in ("tokens", "hidden", "inter", "experts", "top_k"))
        s["x"] = normal(t, h)
        # gate and up spread like the activation's own inputs, so that some of them clamp
        gated = case["act"] == "swiglu"
        s["w_up"] = weights(e, 2 * inter if gated else inter, h, (3.0 if gated else 1.0) / math.sqrt(h))
        s["w_down"] = weights(e, h, inter, 1 / math.sqrt(inter))
        ranked, order = torch.sort(normal(t, e, kind="f32"), dim=1, descending=True, stable=True)
        k = min(k, e)
        s["ids"] = order[:, :k].to(torch.int32).contiguous()
        s["probs"] = torch.softmax(ranked[:, :k], 1).contiguous()
        s["res"] = normal(t, h) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _plain_gate(s, logits):
    """Scores, and the choice of experts, in 64 bits."""
    t, e = logits.shape
    masked = logits == -math.inf
    if s["scores"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    rank = score if s["bias_v"] is None else score + s["bias_v"].double()
    rank = torch.where(masked, -math.inf, rank)
    if s["groups"] > 1:
        each = rank.view(t, s["groups"], -1)
        worth = torch.sort(each, dim=2, descending=True, stable=True)[0][:, :, :s["group_top"]].sum(2)
        best = torch.sort(worth, dim=1, descending=True, stable=True)[1][:, :s["top_groups"]]
        kept = torch.zeros_like(worth, dtype=torch.bool).scatter_(1, best, True)
        # the experts of other groups come after everything, masked ones too
        order = torch.sort(rank, dim=1, descending=True, stable=True)[1]
        inside = kept.repeat_interleave(e // s["groups"], 1).gather(1, order)
        order = order.gather(1, torch.sort((~inside).to(torch.int8), dim=1, stable=True)[1])
    else:
        order = torch.sort(rank, dim=1, descending=True, stable=True)[1]
    ids = order[:, :s["top_k"]]
    probs = score.gather(1, ids)
    if s["renorm"]:
        total = probs.sum(1, keepdim=True)
        probs = torch.where(total > 0, probs / total, 0.0)
    return {"ids": ids.to(torch.int32), "probs": (probs * s["scale"]).float()}


def _plain_gate_bwd(s):
    logits, ids, g = s["logits"].float(), s["ids"].long(), s["grad_probs"] * s["scale"]
    if s["scores"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
        slope = score * (1 / (1 + torch.exp(logits)))
    else:
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    chosen = score.gather(1, ids)
    if s["renorm"]:
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total > 0, total, math.inf)
        p = chosen / total
        d_score = (g - (g * p).sum(1, keepdim=True)) / total
    else:
        d_score = g
    dense = torch.zeros_like(score).scatter_(1, ids, d_score)
    if s["scores"] == "sigmoid":
        grad = dense * slope
    else:
        grad = score * (dense - (dense * score).sum(1, keepdim=True))
    return {"grad_logits": grad.to(s["logits"].dtype)}


def _plain_quantize(s):
    out = []
    for w in s["w"]:
        codes, exponents = _quantize(w.float())
        out.append(_values(_pairs(codes), exponents).to(torch.bfloat16))
    return {"values": torch.stack(out)}


def _plain_linear(s):
    z = s["x"].float() @ _values(*s["w"]).t()
    if s["bias_v"] is not None:
        z = z + s["bias_v"].float()
    if s["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    elif s["act"] == "gelu":
        z = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    elif s["act"] == "squared_relu":
        z = z.clamp(min=0).square()
    if s["res"] is not None:
        z = z + s["res"].float()
    return {"y": z.to(s["x"].dtype)}


def _plain_act(s, z):
    if s["act"] == "squared_relu":
        return z.clamp(min=0).square()
    gate, up = z.chunk(2, dim=-1)
    gate, up = gate.clamp(max=s["limit"]), up.clamp(-s["limit"], s["limit"])
    return gate / (1 + torch.exp(-gate)) * up


def _plain_experts(s):
    x, ids, probs = s["x"].float(), s["ids"].long(), s["probs"]
    y = torch.zeros_like(x) if s["res"] is None else s["res"].float()
    if ids.numel() <= s["experts"]:  # the chosen experts' weights, a token and slot at a time
        for t in range(ids.shape[0]):
            for j in range(ids.shape[1]):
                at = ids[t, j:j + 1]
                up, down = (_values(*(part.index_select(0, at)[0] for part in s[key])) for key in ("w_up", "w_down"))
                h = _plain_act(s, x[t:t + 1] @ up.t()) * probs[t, j]
                y = y.index_add(0, torch.full((1,), t, device=x.device), h @ down.t())
    else:  # every expert over every token, the ones not chosen weighted with zero
        p = torch.zeros(x.shape[0], s["experts"], device=x.device).scatter_(1, ids, probs)
        for e in range(s["experts"]):
            up, down = (_values(*(part[e] for part in s[key])) for key in ("w_up", "w_down"))
            y = y + (_plain_act(s, x @ up.t()) * p[:, e:e + 1]) @ down.t()
    return {"y": y.to(s["x"].dtype)}


# ---------------------------------------------------------------------------
# The package's calls
# ---------------------------------------------------------------------------
def _own(s):
    import memory_bound_elementwise_amd as mbe

    op = s["op"]
    if op in ("gate", "route"):
        t = s["tokens"]
        ids = torch.empty(t, s["top_k"], dtype=torch.int32, device=DEV)
        probs = torch.empty(t, s["top_k"], dtype=torch.float32, device=DEV)
        how = dict(scores=s["scores"], bias=s["bias_v"], groups=s["groups"], top_groups=s["top_groups"],
                   group_top=s["group_top"], renormalize=s["renorm"], scale=s["scale"])
        if op == "gate":
            mbe.moe_gate_fwd(s["logits"], ids, probs, **how)
        else:
            mbe.moe_route(s["x"], s["router"], ids, probs, **how)
        return {"ids": ids, "probs": probs}
    if op == "gate_bwd":
        grad = mbe.moe_gate_bwd(s["logits"], s["ids"], s["grad_probs"], torch.empty_like(s["logits"]),
                                scores=s["scores"], renormalize=s["renorm"], scale=s["scale"])
        return {"grad_logits": grad}
    if op == "quantize":
        w = s["w"]
        codes, scales = (torch.empty(w.shape[0], *shape, dtype=torch.uint8, device=DEV)
                         for shape in mbe.fp4_shapes(s["n"], s["k"]))
        mbe.fp4_quantize(w, codes, scales)
        return {"values": mbe.fp4_dequantize(codes, scales, torch.empty(w.shape, dtype=torch.bfloat16, device=DEV))}
    x = s["x"]
    if op == "linear":
        y = torch.empty(s["m"], s["n"], dtype=x.dtype, device=DEV)
        return {"y": mbe.linear_act_fp4(x, *s["w"], y, bias=s["bias_v"], activation=s["act"], residual=s["res"])}
    y = mbe.moe_experts_fp4(x, *s["w_up"], *s["w_down"], s["ids"], s["probs"], torch.empty_like(x),
                            activation=s["act"], limit=s["limit"], residual=s["res"])
    return {"y": y}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "gate":
        return _plain_gate(state, state["logits"].double())
    if op == "route":
        return _plain_gate(state, state["x"].double() @ state["router"].double().t())
    if op == "gate_bwd":
        return _plain_gate_bwd(state)
    if op == "quantize":
        return _plain_quantize(state)
    return _plain_linear(state) if op == "linear" else _plain_experts(state)


def work(case):
    op = case["op"]
    if op in ("gate", "gate_bwd", "route"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        if op == "route":
            h = case["hidden"]
            return {"bytes": 2 * (t * h + e * h) + 4 * e * case["bias"] + 8 * t * k, "flops": 2 * t * e * h}
        size = 4 if case["type"] == "f32" else 2
        if op == "gate":
            return {"bytes": t * e * size + 4 * e * case["bias"] + 8 * t * k, "flops": 8 * t * e}
        dense = case["scores"] == "softmax" and not case["renorm"]
        return {"bytes": t * size * (e + (e if dense else k)) + 8 * t * k, "flops": 8 * t * (e if dense else k)}
    if op == "quantize":  # the weights in, 4.25 bits each out and in again, 16-bit values out
        n = case["matrices"] * case["n"] * case["k"]
        return {"bytes": int(n * ((4 if case["type"] == "f32" else 2) + 2 * 17 / 32 + 2)), "flops": 4 * n}
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * (m * k + m * n * (2 if case["residual"] else 1) + (n if case["bias"] else 0)) + n * k * 17 // 32,
                "flops": 2 * m * n * k}
    t, h, e, inter, k = case["tokens"], case["hidden"], case["experts"], case["inter"], min(case["top_k"], case["experts"])
    ups = 2 * inter if case["act"] == "swiglu" else inter
    reached = e * (1 - (1 - k / e) ** t)  # distinct experts, as independent choices give them
    return {"bytes": int(reached * (ups + inter) * h * 17 / 32) + 2 * t * h * (3 if case["residual"] else 2) + 8 * t * k,
            "flops": 2 * t * k * (ups + inter) * h}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _checkpoint(case, seed):
    """The inputs with the weights as a checkpoint holds them."""
    global own
    kept, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = kept


def _wide(elements, exponents):
    """Packed weights in 64 bits, from the bits of the format: sign, two of exponent, one of mantissa."""
    code = torch.empty(*elements.shape[:-1], 2 * elements.shape[-1], dtype=torch.int16, device=elements.device)
    code[..., 0::2], code[..., 1::2] = elements.bitwise_and(0xF), elements.bitwise_right_shift(4)
    mantissa, power = (code & 1).double(), (code >> 1 & 3).double()
    size = torch.where(power == 0, mantissa / 2, (1 + mantissa / 2) * 2 ** (power - 1))
    size = torch.where(code >= 8, -size, size).unflatten(-1, (-1, GROUP))
    return (size * (2.0 ** (exponents.double() - 127)).unsqueeze(-1)).flatten(-2)


def _exact_chosen(case, score, rank):
    """The k experts of each row that a walk through them in order of worth keeps."""
    t, e = score.shape
    size = e // case["groups"]
    if case["groups"] > 1:
        parts = rank.reshape(t, case["groups"], size)
        worth = torch.topk(parts, case["group_top"], dim=2)[0].sum(2)
        place = torch.argsort(torch.argsort(-worth, dim=1, stable=True), dim=1)
        out = place.repeat_interleave(size, 1) >= case["top_groups"]
    else:
        out = torch.zeros_like(rank, dtype=torch.bool)
    first = torch.argsort(-rank, dim=1, stable=True)
    late = torch.gather(out, 1, first).to(torch.int64) * e + torch.arange(e, device=rank.device)
    return torch.gather(first, 1, torch.argsort(late, dim=1))[:, :case["top_k"]]


def exact(case, seed):
    s = _checkpoint(case, seed)
    op = case["op"]
    if op in ("gate", "route", "gate_bwd"):
        if op == "route":
            logits = torch.matmul(s["x"].to(torch.float64), s["router"].to(torch.float64).T)
        else:
            logits = s["logits"].to(torch.float64)
        sigmoid = case["scores"] == "sigmoid"
        score = torch.sigmoid(logits) if sigmoid else torch.softmax(logits, dim=1)
        if op == "gate_bwd":
            at = s["ids"].to(torch.int64)
            g = s["grad_probs"].to(torch.float64) * case["scale"]
            mine = torch.gather(score, 1, at)
            if case["renorm"]:
                total = mine.sum(1, keepdim=True)
                g = torch.where(total > 0, (g * total - torch.linalg.vecdot(g, mine)[:, None]) / total ** 2, 0.0)
            if sigmoid:
                back = g * mine * torch.sigmoid(-torch.gather(logits, 1, at))
                return {"grad_logits": torch.zeros_like(score).scatter_add_(1, at, back)}
            mean = torch.linalg.vecdot(g, mine)[:, None]
            return {"grad_logits": (-mean * score).scatter_add_(1, at, g * mine)}
        rank = score if s["bias_v"] is None else torch.add(score, s["bias_v"].to(torch.float64))
        rank = rank.masked_fill(torch.isneginf(logits), -math.inf)
        weight = torch.gather(score, 1, _exact_chosen(case, score, rank))
        if case["renorm"]:
            weight = torch.nan_to_num(weight / weight.sum(1, keepdim=True))
        return {"ids": None, "probs": case["scale"] * weight}
    if op == "quantize":
        values = []
        level = torch.tensor(_LEVELS, dtype=torch.float64, device=DEV)
        between = (level[1:] + level[:-1]) / 2
        for w in s["w"].to(torch.float64):
            v = w.reshape(-1, GROUP)
            top = v.abs().amax(1, keepdim=True)
            power = torch.floor(torch.log2(top.clamp(min=1e-300) / 7.0)) + 1  # top < 7 2^power, the smallest such
            power = torch.where(top >= 7.0 * 2.0 ** power, power + 1, power)
            power = torch.where(top < 7.0 * 2.0 ** (power - 1), power - 1, power)
            v = v * 2.0 ** -power
            up = torch.bucketize(v.abs(), between, right=True)   # a tie to the higher code,
            low = torch.bucketize(v.abs(), between)              # and to the lower one
            code = torch.where(up % 2 == 0, up, low)
            values.append((torch.sign(v) * level[code] * 2.0 ** power).reshape(w.shape))
        return {"values": torch.stack(values)}
    x = s["x"].to(torch.float64)
    if op == "linear":
        z = torch.matmul(x, _wide(*s["w"]).T)
        if case["bias"]:
            z += s["bias_v"].to(torch.float64)
        if case["act"] == "silu":
            z *= torch.sigmoid(z)
        elif case["act"] == "gelu":
            z *= torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
        elif case["act"] == "squared_relu":
            z = torch.where(z > 0, z * z, torch.zeros_like(z))
        if case["residual"]:
            z += s["res"].to(torch.float64)
        return {"y": z}
    y = s["res"].to(torch.float64) if case["residual"] else torch.zeros_like(x)
    for e in range(case["experts"]):  # an expert at a time
        t, slot = torch.where(s["ids"] == e)
        if not t.numel():
            continue
        z = torch.matmul(x[t], _wide(s["w_up"][0][e], s["w_up"][1][e]).T)
        if case["act"] == "squared_relu":
            a = torch.where(z > 0, z * z, torch.zeros_like(z))
        else:
            gate, up = z[:, :case["inter"]], z[:, case["inter"]:]
            gate = torch.minimum(gate, torch.full_like(gate, case["limit"]))
            a = gate * torch.sigmoid(gate) * up.clip(-case["limit"], case["limit"])
        a = a * s["probs"][t, slot].to(torch.float64)[:, None]
        y.index_add_(0, t, torch.matmul(a, _wide(s["w_down"][0][e], s["w_down"][1][e]).T))
    return {"y": y}
