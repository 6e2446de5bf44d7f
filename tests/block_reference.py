"""The block operators in 64 bits (torch on the CPU) with bounds on a 32-bit evaluation's error
(test infrastructure; shares no code with the kernels).

Every reference returns (value, bound): |kernel - value| <= bound elementwise, where the bound
adds, term by term, what the documented arithmetic can lose. u = 2^-24 is half a step of fp32;
a sum of n terms in any order is off by at most (n - 1) u sum |terms| (first order), less for
a tree: the depth stands in for n where the kernel's order is a tree. The last term is the
output's own rounding, half a step of its type (and half its smallest subnormal)."""
import math

import torch

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(value, bound, dtype):
    """bound plus the rounding of the output to dtype."""
    return bound + (value.abs() + bound) * half_step(dtype) + TINY[dtype]


def check(got, value, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    nan = torch.isnan(value)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(value)
    assert torch.equal(torch.where(inf, got, 0.0), torch.where(inf, value, 0.0)), f"{what}: infinities differ"
    fine = ~nan & ~inf
    off = (got - value).abs()[fine]
    lim = bound.expand_as(value)[fine]
    bad = ~(off <= lim)  # a NaN bound fails
    if bool(bad.any()):
        i = int((off / lim.clamp(min=1e-300)).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {off.numel()} past their bound; worst off by "
                             f"{off[i].item():.3e}, bound {lim[i].item():.3e}")


# Depth of the layer norm's row sums: at most 128 elements in a lane (2^20 columns over 1024
# lanes take 1024), 6 wave steps, 16 waves.
def _depth(cols):
    return max(32, math.ceil(cols / 1024)) + 22


def layer_norm(x, weight, bias, eps, dtype):
    """x, weight, bias: double or None. Returns y, mean, rstd, each (value, bound)."""
    cols = x.shape[1]
    w = torch.ones(cols, dtype=torch.float64) if weight is None else weight
    b = torch.zeros(cols, dtype=torch.float64) if bias is None else bias
    d = _depth(cols)
    mean = x.mean(1, keepdim=True)
    dmean = (d + 2) * U * x.abs().mean(1, keepdim=True)
    c = x - mean
    var = (c * c).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    dc = dmean + U * (c.abs() + dmean)
    # var about a mean that is off by dmean is larger by dmean^2; each square is off by 2 |c| dc
    dvar = (2 * c.abs() * dc + dc * dc).mean(1, keepdim=True) + (d + 4) * U * var + 2 * U * eps
    drstd = rstd * (0.5 * dvar / (var + eps).clamp(min=1e-300) + 4 * U)
    n = c * rstd
    dn = dc * rstd + c.abs() * drstd + 2 * U * n.abs()
    y = n * w + b
    dy = dn * w.abs() + 2 * U * (y.abs() + (n * w).abs())
    return ((y, rounded(y, dy, dtype)), (mean[:, 0], dmean[:, 0] + TINY[torch.float32]),
            (rstd[:, 0], drstd[:, 0] + U * rstd[:, 0]))


def layer_norm_grads(gy, x, weight, mean, rstd, dtype, wdtype):
    """mean, rstd: the fp32 values the kernel is given, as double. Returns (value, bound) of
    grad_x, grad_weight, grad_bias."""
    rows, cols = x.shape
    w = torch.ones(cols, dtype=torch.float64) if weight is None else weight
    mu, rs = mean[:, None], rstd[:, None]
    n = (x - mu) * rs
    dn = 3 * U * n.abs()
    d = gy * w
    dd = U * d.abs()
    a = d.mean(1, keepdim=True)
    b = (d * n).mean(1, keepdim=True)
    depth = _depth(cols)
    da = (depth + 3) * U * d.abs().mean(1, keepdim=True)
    db = (depth + 8) * U * (d * n).abs().mean(1, keepdim=True)
    gx = (d - a - n * b) * rs
    dgx = (dd + da + n.abs() * db + dn * b.abs() + 4 * U * (d.abs() + a.abs() + (n * b).abs())) * rs.abs()
    # rows over at most 256 workgroups of up to 16 groups, 16 partial sums a wave, 16 waves;
    # narrow or wide, a lane adds at most ceil(rows / 256) + 1 rows in turn
    turns = math.ceil(rows / 256) + 1 + 16 + 16 + 16
    gw, sw = (gy * n).sum(0), (gy * n).abs().sum(0)
    gb, sb = gy.sum(0), gy.abs().sum(0)
    return ((gx, rounded(gx, dgx, dtype)), (gw, rounded(gw, (turns + 4) * U * sw, wdtype)),
            (gb, rounded(gb, turns * U * sb, wdtype)))


def _logistic_loss(z, w):
    """Bound on the relative error of z / (1 + e^-w) from v_exp_f32 and v_rcp_f32: the exponent
    is rounded twice (|w| u each), the exponential and the reciprocal to 2 u, the rest 4 u."""
    return (2 * w.abs().clamp(max=128) + 8) * U


def activation(name, z, dz):
    """(act(z), bound) for z known to dz."""
    if name in (None, "none"):
        return z, dz
    if name == "silu":
        v = z * torch.sigmoid(z)
        return v, 1.1 * dz + v.abs() * _logistic_loss(z, z)
    if name == "gelu":
        w = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        v = z * torch.sigmoid(w)
        return v, 1.13 * dz + v.abs() * (_logistic_loss(z, w) + 4 * U * w.abs().clamp(max=128))
    a = torch.where(z > 0, z, torch.where(torch.isnan(z), z, torch.zeros_like(z)))
    return a * a, 2 * a * dz + dz * dz + 2 * U * a * a


def product(x, w):
    """x w^T with the loss of an fp32 sum of exact products (matrix cores add several at a time,
    each step rounded or cut off: at most a step of 2 u a term)."""
    return x @ w.t(), 2 * x.shape[1] * U * (x.abs() @ w.abs().t())


def linear_act(x, w, bias, name, residual, dtype):
    z, dz = product(x, w)
    if bias is not None:
        z = z + bias
        dz = dz + U * (z.abs() + dz)
    v, dv = activation(name, z, dz)
    if residual is not None:
        v = v + residual
        dv = dv + U * (v.abs() + dv)
    # past fp16's range the rounding gives infinity
    top = torch.finfo(dtype).max
    return v, rounded(v, dv, dtype), top


def route(x, router, top_k, renormalize):
    """ids and (probs, bound)."""
    logits = x @ router.t()
    ranked, order = torch.sort(logits, dim=1, descending=True, stable=True)
    e = torch.exp(ranked - ranked[:, :1])
    p = e[:, :top_k] / (e[:, :top_k] if renormalize else e).sum(1, keepdim=True)
    # the exponent is rounded once (|l - l_max| u), expf and the division to 2 u, the sum of
    # positive terms over 16 of a lane and 6 steps
    gap = (ranked[:, :1] - ranked)
    loss = (gap[:, :top_k] + gap.mean(1, keepdim=True).clamp(max=88) + 32) * U
    return order[:, :top_k].to(torch.int32), (p, p * loss + 2.0 ** -126)


def experts(x, w_up, w_down, ids, probs, act, limit, residual, dtype):
    """(y, bound), everything double but ids; ids outside the experts contribute nothing."""
    tokens, hidden = x.shape
    n_experts, _, inter = w_down.shape
    y = torch.zeros(tokens, hidden, dtype=torch.float64)
    dy = torch.zeros_like(y)
    mass = torch.zeros_like(y)
    for t in range(tokens):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < n_experts:
                continue
            z, dz = product(x[t:t + 1], w_up[e])
            if act == "swiglu":
                g, up = z[:, :inter], z[:, inter:]
                g = torch.where(g > limit, torch.full_like(g, limit), g)
                up = up.clamp(-limit, limit)
                s, ds = activation("silu", g, dz[:, :inter])
                h = s * up
                dh = ds * up.abs() + s.abs() * dz[:, inter:] + ds * dz[:, inter:] + U * h.abs()
            else:
                h, dh = activation("squared_relu", z, dz)
            p = probs[t, j]
            h, dh = h * p, (dh + U * h.abs()) * p.abs() + h.abs() * p.abs() * 2.0 ** -15  # two bf16 terms: 2^-16, and slack
            v, dv = product(h, w_down[e])
            y[t] += v[0]
            dy[t] += 2 * dv[0] + (dh @ w_down[e].abs().t())[0]
            mass[t] += v[0].abs()
    dy += (ids.shape[1] * 16 + 4) * U * mass
    if residual is not None:
        y = y + residual
        dy = dy + 2 * U * (y.abs() + dy)
    return y, rounded(y, dy, dtype)
