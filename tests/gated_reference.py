"""The gate, its gradient and the 4-bit weights in 64 bits on the CPU, row by row from their
definitions, with bounds as in block_reference (test infrastructure; shares no code with the
kernels)."""
import math

import torch

import block_reference as ref

NAN, INF = float("nan"), float("inf")
# fp64 sums and functions of at most 1024 terms: far below this share of what they add up
WIDE = 2.0 ** -40


def scores_of(row, kind):
    """row: double [experts]. Softmax of a row of -inf is zeros."""
    if kind == "sigmoid":
        return torch.sigmoid(row)
    if bool((row == -INF).all()):
        return torch.zeros_like(row)
    return torch.softmax(row, 0)


def _first(values):
    """Indices in the order of choice: NaN, then descending, equal ones ascending."""
    return sorted(range(len(values)), key=lambda i: (0 if math.isnan(values[i]) else 1,
                                                     0.0 if math.isnan(values[i]) else -values[i], i))


def gate(logits, top_k, scores, bias=None, groups=1, top_groups=None, group_top=1, renormalize=False, scale=1.0):
    """ids (int32) and (probs, bound) of logits (any dtype, on the CPU)."""
    tokens, experts = logits.shape
    size = experts // groups
    top_groups = groups if top_groups is None else top_groups
    ids, probs = [], []
    for row in logits.double():
        s = scores_of(row, scores)
        c = s if bias is None else s + bias.double()
        c = torch.where(row == -INF, torch.full_like(c, -INF), c).tolist()
        kept = range(groups)
        if groups > 1:
            worth = []
            for g in range(groups):
                part = c[g * size:(g + 1) * size]
                worth.append(sum(part[i] for i in _first(part)[:group_top]))
            kept = set(_first(worth)[:top_groups])
        order = [i for i in _first(c) if i // size in kept][:top_k]
        p = s[order]
        if renormalize:
            total = float(p.sum())
            if scores == "softmax" and total == total:
                p = scores_of(row[order], scores)           # the same, but where s runs out of exponents
            else:
                p = torch.zeros_like(p) if total == 0 else p / total
        ids.append(torch.tensor(order, dtype=torch.int32))
        probs.append(p * scale)
    ids = torch.stack(ids) if ids else torch.empty(0, top_k, dtype=torch.int32)
    probs = torch.stack(probs) if probs else torch.empty(0, top_k, dtype=torch.float64)
    return ids, (probs, ref.rounded(probs, probs.abs() * WIDE, torch.float32))


def gate_grads(logits, ids, grad_probs, scores, renormalize, scale, dtype):
    """(grad_logits, bound), slot by slot from the chain rule."""
    out, loss = torch.zeros(logits.shape, dtype=torch.float64), torch.zeros(logits.shape, dtype=torch.float64)
    experts = logits.shape[1]
    for t in range(logits.shape[0]):
        row = logits[t].double()
        s = scores_of(row, scores)
        slots = [(int(e), scale * float(g)) for e, g in zip(ids[t], grad_probs[t]) if 0 <= int(e) < experts]
        if not slots:
            continue
        at = torch.tensor([e for e, _ in slots])
        g = torch.tensor([v for _, v in slots], dtype=torch.float64)
        if scores == "softmax" and renormalize:
            p = scores_of(row[at], "softmax")           # of the chosen ones alone
            d = g - (g * p).sum()
            out[t].index_add_(0, at, p * d)
            loss[t].index_add_(0, at, p * (g.abs() + (g * p).abs().sum()))
        elif scores == "softmax":
            v = g * s[at]
            out[t].index_add_(0, at, v)
            out[t] -= s * v.sum()
            loss[t].index_add_(0, at, v.abs())
            loss[t] += s * v.abs().sum()
        else:
            slope = torch.sigmoid(-row[at])
            p = s[at]
            d = g
            mass = g.abs()
            if renormalize:
                total = p.sum()
                p = torch.zeros_like(p) if float(total) == 0 else p / total
                d = g - (g * p).sum()
                mass = g.abs() + (g * p).abs().sum()
            out[t].index_add_(0, at, p * d * slope)
            loss[t].index_add_(0, at, p * mass * slope)
    return out, ref.rounded(out, loss * WIDE, dtype)


# ---------------------------------------------------------------------------
# Weights in 4 bits
# ---------------------------------------------------------------------------
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def quantize(w):
    """Elements (codes 0 .. 15) and exponents (bytes) of w [..., k], k a multiple of 32."""
    v = w.double().unflatten(-1, (-1, 32))
    top = v.abs().amax(-1)
    bad = ~torch.isfinite(v).all(-1)
    usable = torch.where(bad | (top == 0), torch.ones_like(top), top)
    power = torch.floor(torch.log2(usable / 7))          # about; then exactly
    power = torch.where(usable >= 7 * 2.0 ** power, power + 1, power)
    power = torch.where(usable < 7 * 2.0 ** (power - 1), power - 1, power).clamp(-127, 125)
    byte = torch.where(bad, 255.0, torch.where(top == 0, 127.0, power + 127)).to(torch.uint8)
    a = (v.abs() * 2.0 ** -power[..., None]).nan_to_num(nan=0.0, posinf=0.0)
    levels = torch.tensor(LEVELS, dtype=torch.float64)
    gap = (a[..., None] - levels).abs()                   # the nearest; a tie to the even code
    best = gap.amin(-1, keepdim=True)
    near = gap == best
    even = torch.tensor([i % 2 == 0 for i in range(8)])
    pick = torch.where(near.sum(-1, keepdim=True) > 1, near & even, near)
    code = pick.to(torch.uint8).argmax(-1) + 8 * torch.signbit(v)
    return code.flatten(-2).to(torch.uint8), byte


def values(codes, exponents):
    """The weights in 64 bits: beyond bf16's range infinities, groups of byte 255 NaN."""
    levels = torch.tensor(LEVELS + [-x for x in LEVELS], dtype=torch.float64)
    scale = torch.where(exponents == 255, NAN, 2.0 ** (exponents.double() - 127))
    v = (levels[codes.long()].unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)
    return torch.where(v.abs() > torch.finfo(torch.bfloat16).max, v.sign() * INF, v)


def pairs(codes):
    """Two elements a byte, the first in its lower half."""
    return codes[..., 0::2] | codes[..., 1::2] << 4


def lay_out(codes, exponents):
    """The tiles, element by element: codes uint8 [n/16, k/128, 1024] and scales [.., 64], of one matrix."""
    n, k = codes.shape
    nt, kt = -(-n // 16), -(-k // 128)
    full = torch.zeros(nt * 16, kt * 128, dtype=torch.uint8)
    full[:n, :k] = codes
    byte = torch.full((nt * 16, kt * 4), 127, dtype=torch.uint8)
    byte[:n, :k // 32] = exponents
    # [tile row, r, tile k, j, q, i] -> [tile row, tile k, q, r, j, i]
    c = full.view(nt, 16, kt, 4, 4, 8).permute(0, 2, 4, 1, 3, 5).reshape(nt, kt, 64, 4, 8)
    s = byte.view(nt, 16, kt, 4).permute(0, 2, 1, 3).reshape(nt, kt, 64)
    return pairs(c).reshape(nt, kt, 1024).contiguous(), s.contiguous()


def experts(x, up, down, ids, probs, act, limit, residual, dtype):
    """(y, bound), everything double but ids; up, down: the weights' values. The activation keeps
    its 24 bits through the down product, so its own fp32 rounding is all that it loses."""
    tokens, hidden = x.shape
    n_experts, _, inter = down.shape
    y, dy, mass = (torch.zeros(tokens, hidden, dtype=torch.float64) for _ in range(3))
    for t in range(tokens):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < n_experts:
                continue
            z, dz = ref.product(x[t:t + 1], up[e])
            if act == "swiglu":
                g, u = z[:, :inter].clamp(max=limit), z[:, inter:].clamp(-limit, limit)
                s, ds = ref.activation("silu", g, dz[:, :inter])
                h = s * u
                dh = ds * u.abs() + s.abs() * dz[:, inter:] + ds * dz[:, inter:] + ref.U * h.abs()
            else:
                h, dh = ref.activation("squared_relu", z, dz)
            h, dh = h * probs[t, j], (dh + ref.U * h.abs()) * probs[t, j].abs()
            v, dv = ref.product(h, down[e])
            y[t] += v[0]
            # the three terms' magnitudes add up to at most twice the activation's
            dy[t] += 2 * dv[0] + (dh @ down[e].abs().t())[0]
            mass[t] += v[0].abs()
    dy += (ids.shape[1] + 16) * ref.U * mass
    if residual is not None:
        y = y + residual
        dy = dy + 2 * ref.U * (y.abs() + dy)
    return y, ref.rounded(y, dy, dtype)
