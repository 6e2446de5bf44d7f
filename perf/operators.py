"""Cases for the operators of one Mixture-of-Experts block: layer norm (forward and
backward), a matrix product with bias, activation and residual in its epilogue, the
router (product, top-k, softmax weights) and a whole expert layer for a few tokens.

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits
(the router's logits in 64, since its choice of experts is made between neighbouring
values), rounded once at the end. With ``own`` true it makes the calls of this package.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decoded token's pre-norm: latency only
        {"name": "norm_fwd_token", "op": "norm_fwd", "rows": 1, "cols": 7168, "type": "bf16", "weights": "bf16"},
        # a training step's tokens at the model width, mixed precision (fp32 weights)
        {"name": "norm_fwd_batch", "op": "norm_fwd", "rows": 6720, "cols": 7168, "type": "bf16", "weights": "f32"},
        # the same step's backward
        {"name": "norm_bwd_batch", "op": "norm_bwd", "rows": 6720, "cols": 7168, "type": "bf16", "weights": "f32"},
        # a ragged fp32 batch whose width is odd
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 1009, "cols": 1411, "type": "f32", "weights": "f32"},
        # a shared expert's first product for one decoded token: a weight stream
        {"name": "linear_token", "op": "linear", "m": 1, "k": 7168, "n": 4096, "type": "bf16",
         "act": "silu", "bias": True, "residual": False},
        # a ragged prompt through a shared expert's second product, added to the residual stream
        {"name": "linear_prompt", "op": "linear", "m": 1009, "k": 1408, "n": 2056, "type": "f16",
         "act": "gelu", "bias": True, "residual": True},
        # a full batch at the model width
        {"name": "linear_batch", "op": "linear", "m": 6720, "k": 7168, "n": 4096, "type": "bf16",
         "act": "squared_relu", "bias": True, "residual": True},
        # one decoded token's routing: latency
        {"name": "route_token", "op": "route", "tokens": 1, "hidden": 7168, "experts": 64, "top_k": 8, "renorm": False},
        # a batch of decoded tokens over many experts
        {"name": "route_many", "op": "route", "tokens": 128, "hidden": 4096, "experts": 256, "top_k": 8, "renorm": True},
        # a small model's layer for an odd handful of tokens: latency
        {"name": "moe_small", "op": "moe", "tokens": 3, "hidden": 256, "inter": 256, "experts": 8, "top_k": 2,
         "act": "squared_relu", "limit": math.inf, "renorm": True, "residual": False},
        # one decoded token: eight experts' weights streamed once
        {"name": "moe_token", "op": "moe", "tokens": 1, "hidden": 7168, "inter": 2048, "experts": 64, "top_k": 8,
         "act": "swiglu", "limit": 7.0, "renorm": False, "residual": True},
        # a decoding batch that reaches nearly every expert
        {"name": "moe_batch", "op": "moe", "tokens": 64, "hidden": 7168, "inter": 2048, "experts": 64, "top_k": 8,
         "act": "swiglu", "limit": 7.0, "renorm": True, "residual": True},
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return int(max(lo, min(hi, v))) // step * step


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "linear", "linear", "route", "moe", "moe"])
    if op in ("norm_fwd", "norm_bwd"):
        kind = rng.choice(["bf16", "f16", "f32"])
        cols = _spread(rng, 16, 7168)
        if rng.random() < 0.6:
            cols = cols // 8 * 8
        most = 6720 if kind != "f32" else 3360
        return {"op": op, "rows": _spread(rng, 1, most), "cols": cols, "type": kind,
                "weights": rng.choice([kind, "f32"])}
    if op == "linear":
        return {"op": op, "m": _spread(rng, 1, 6720), "k": _spread(rng, 128, 7168, 8), "n": _spread(rng, 128, 4096, 8),
                "type": rng.choice(["bf16", "f16"]), "act": rng.choice(["none", "silu", "gelu", "squared_relu"]),
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    if op == "route":
        experts = _spread(rng, 8, 256)
        return {"op": op, "tokens": _spread(rng, 1, 256), "hidden": _spread(rng, 128, 7168, 8), "experts": experts,
                "top_k": rng.randint(1, 8), "renorm": rng.random() < 0.5}
    act = rng.choice(["swiglu", "swiglu", "squared_relu"])
    return {"op": op, "tokens": _spread(rng, 1, 64), "hidden": _spread(rng, 128, 7168, 8),
            "inter": _spread(rng, 128, 2048, 8), "experts": _spread(rng, 8, 64), "top_k": rng.randint(1, 8),
            "act": act, "limit": rng.choice([7.0, math.inf]) if act == "swiglu" else math.inf,
            "renorm": rng.random() < 0.5, "residual": rng.random() < 0.5}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0, kind="bf16", mean=0.0):
        # drawn in the tensor's own type: the expert weights are gigabytes
        t = torch.randn(*shape, generator=g, device=DEV, dtype=TYPES[kind])
        if std != 1.0:
            t.mul_(std)
        return t.add_(mean) if mean else t

    s = dict(case)
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        rows, cols, kind, wkind = case["rows"], case["cols"], case["type"], case["weights"]
        # a residual stream: each row with an offset and a scale of its own
        x = normal(rows, cols, kind="f32")
        x.mul_(torch.rand(rows, 1, generator=g, device=DEV) * 3 + 0.5).add_(normal(rows, 1, kind="f32", std=0.5))
        s["x"] = x.to(TYPES[kind])
        s["weight"] = normal(cols, std=0.2, mean=1.0, kind=wkind)
        s["bias"] = normal(cols, std=0.2, kind=wkind)
        if op == "norm_bwd":
            s["grad_y"] = normal(rows, cols, kind=kind)
            wide = s["x"].double()  # what the forward pass saved
            mean = wide.mean(1, keepdim=True)
            var = (wide - mean).square().mean(1)
            s["mean"], s["rstd"] = mean[:, 0].float(), (var + EPS).rsqrt().float()
    elif op == "linear":
        m, k, n, kind = case["m"], case["k"], case["n"], case["type"]
        s["x"] = normal(m, k, kind=kind)
        s["weight"] = normal(n, k, std=1 / math.sqrt(k), kind=kind)
        s["bias_v"] = normal(n, std=0.5, kind=kind) if case["bias"] else None
        s["res"] = normal(m, n, kind=kind) if case["residual"] else None
    else:
        t, h, e = case["tokens"], case["hidden"], case["experts"]
        s["x"] = normal(t, h)
        s["router"] = normal(e, h, std=1 / math.sqrt(h))
        if op == "moe":
            inter = case["inter"]
            ups = 2 * inter if case["act"] == "swiglu" else inter
            # gate and up spread like the activation's own inputs, so that some of them clamp
            s["w_up"] = normal(e, ups, h, std=(3.0 if case["act"] == "swiglu" else 1.0) / math.sqrt(h))
            s["w_down"] = normal(e, h, inter, std=1 / math.sqrt(inter))
            s["res"] = normal(t, h) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    y = (x - mean) * rstd * s["weight"].float() + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_bwd(s):
    gy, rstd = s["grad_y"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    wg = gy * s["weight"].float()
    gx = (wg - wg.mean(1, keepdim=True) - xhat * (wg * xhat).mean(1, keepdim=True)) * rstd
    kind = s["weight"].dtype
    return {"grad_x": gx.to(s["x"].dtype), "grad_weight": (gy * xhat).sum(0).to(kind), "grad_bias": gy.sum(0).to(kind)}


def _plain_linear(s):
    z = s["x"].float() @ s["weight"].float().t()
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


def _plain_route(s):
    logits = s["x"].double() @ s["router"].double().t()
    ranked, order = torch.sort(logits, dim=1, descending=True, stable=True)
    k = min(s["top_k"], logits.shape[1])
    weights = torch.exp(ranked - ranked[:, :1])
    probs = weights[:, :k] / (weights[:, :k] if s["renorm"] else weights).sum(1, keepdim=True)
    return order[:, :k].to(torch.int32), probs.float()


def _plain_act(s, z):
    """z = x W_up^T in 32 bits; the probability is applied by the caller."""
    if s["act"] == "squared_relu":
        return z.clamp(min=0).square()
    gate, up = z.chunk(2, dim=-1)
    gate, up = gate.clamp(max=s["limit"]), up.clamp(-s["limit"], s["limit"])
    return gate / (1 + torch.exp(-gate)) * up


def _plain_moe(s):
    ids, probs = _plain_route(s)
    x, (t, k) = s["x"].float(), ids.shape
    if t * k <= s["experts"]:  # gather the chosen experts' weights
        at = ids.long()
        h = _plain_act(s, (s["w_up"][at].float() @ x[:, None, :, None])[..., 0]) * probs[..., None]
        y = (s["w_down"][at].float() @ h[..., None])[..., 0].sum(1)
    else:  # every expert over every token, the ones not chosen weighted with zero
        p = torch.zeros(t, s["experts"], device=x.device).scatter_(1, ids.long(), probs)
        h = _plain_act(s, x[None] @ s["w_up"].float().transpose(1, 2)) * p.t()[:, :, None]
        y = (h @ s["w_down"].float().transpose(1, 2)).sum(0)
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(s["x"].dtype), "ids": ids, "probs": probs}


# ---------------------------------------------------------------------------
# The package's calls
# ---------------------------------------------------------------------------
def _own(s):
    import memory_bound_elementwise_amd as mbe

    op, x = s["op"], s["x"]
    if op == "norm_fwd":
        rows = x.shape[0]
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        y = mbe.layer_norm_fwd(x, s["weight"], s["bias"], torch.empty_like(x), mean, rstd, eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        gx, gw, gb = mbe.layer_norm_bwd(s["grad_y"], x, s["weight"], s["mean"], s["rstd"], torch.empty_like(x),
                                        torch.empty_like(s["weight"]), torch.empty_like(s["bias"]))
        return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    if op == "linear":
        y = torch.empty(s["m"], s["n"], dtype=x.dtype, device=x.device)
        return {"y": mbe.linear_act(x, s["weight"], y, bias=s["bias_v"], activation=s["act"], residual=s["res"])}
    k = min(s["top_k"], s["experts"])
    ids = torch.empty(s["tokens"], k, dtype=torch.int32, device=x.device)
    probs = torch.empty(s["tokens"], k, dtype=torch.float32, device=x.device)
    if op == "route":
        mbe.moe_route(x, s["router"], ids, probs, renormalize=s["renorm"])
        return {"ids": ids, "probs": probs}
    y = mbe.moe_layer(x, s["router"], s["w_up"], s["w_down"], torch.empty_like(x), ids, probs, activation=s["act"],
                      limit=s["limit"], renormalize=s["renorm"], residual=s["res"])
    return {"y": y, "ids": ids, "probs": probs}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(state)
    if op == "norm_bwd":
        return _plain_norm_bwd(state)
    if op == "linear":
        return _plain_linear(state)
    if op == "route":
        ids, probs = _plain_route(state)
        return {"ids": ids, "probs": probs}
    return _plain_moe(state)


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        n, size = case["rows"] * case["cols"], 4 if case["type"] == "f32" else 2
        vec = case["cols"] * (4 if case["weights"] == "f32" else 2)
        if op == "norm_fwd":  # x, weight, bias in; y, mean, rstd out
            return {"bytes": 2 * n * size + 2 * vec + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * size + 3 * vec + 8 * case["rows"], "flops": 14 * n}
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * (m * k + n * k + m * n * (2 if case["residual"] else 1) + (n if case["bias"] else 0)),
                "flops": 2 * m * n * k}
    t, h, e, k = case["tokens"], case["hidden"], case["experts"], min(case["top_k"], case["experts"])
    size, flops = 2 * (t * h + e * h) + 8 * t * k, 2 * t * e * h
    if op == "moe":
        inter = case["inter"]
        ups = 2 * inter if case["act"] == "swiglu" else inter
        reached = e * (1 - (1 - k / e) ** t)  # distinct experts, as independent choices give them
        size += 2 * reached * (ups + inter) * h + 2 * t * h * (2 if case["residual"] else 1)
        flops += 2 * t * k * (ups + inter) * h
    return {"bytes": size, "flops": flops}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, x = case["op"], s["x"].to(torch.float64)
    if op in ("norm_fwd", "norm_bwd"):
        w, b = s["weight"].to(torch.float64), s["bias"].to(torch.float64)
        var, mu = torch.var_mean(x, dim=1, unbiased=False)
        r = 1 / torch.sqrt(var + EPS)
        if op == "norm_fwd":
            return {"y": torch.addcmul(b, torch.sub(x, mu[:, None]) * r[:, None], w), "mean": mu, "rstd": r}
        n = (x - mu[:, None]) * r[:, None]
        g = s["grad_y"].to(torch.float64)
        c = case["cols"]
        d = g * w
        along = torch.linalg.vecdot(d, n) / c
        gx = r[:, None] * (d - (d.sum(1) / c)[:, None] - n * along[:, None])
        return {"grad_x": gx, "grad_weight": torch.linalg.vecdot(g, n, dim=0), "grad_bias": torch.sum(g, 0)}
    if op == "linear":
        z = torch.matmul(x, s["weight"].to(torch.float64).T)
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
    k = min(case["top_k"], case["experts"])
    logits = torch.matmul(x, s["router"].to(torch.float64).T)
    p = torch.softmax(logits, dim=1)
    chosen = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    weight = torch.gather(p, 1, chosen)
    if case["renorm"]:
        weight = weight / weight.sum(1, keepdim=True)
    if op == "route":
        return {"ids": None, "probs": weight}
    y = s["res"].to(torch.float64) if case["residual"] else torch.zeros_like(x)
    for e in range(case["experts"]):  # an expert at a time
        t, slot = torch.where(chosen == e)
        if not t.numel():
            continue
        z = torch.matmul(x[t], s["w_up"][e].to(torch.float64).T)
        if case["act"] == "squared_relu":
            a = torch.where(z > 0, z * z, torch.zeros_like(z))
        else:
            gate, up = z[:, :case["inter"]], z[:, case["inter"]:]
            gate = torch.minimum(gate, torch.full_like(gate, case["limit"]))
            a = gate * torch.sigmoid(gate) * up.clip(-case["limit"], case["limit"])
        y.index_add_(0, t, torch.matmul(a * weight[t, slot][:, None], s["w_down"][e].to(torch.float64).T))
    return {"y": y, "ids": None, "probs": weight}
