"""The gate and the operators on weights in 4 bits, on the host: every refusal of the C ABI and of
the Python bindings, the sizes of layouts and workspaces, and what is launched at the limits.
Nothing here reaches the HIP runtime; the addresses are never dereferenced."""
import ctypes
import json
import subprocess
import sys

import pytest
import torch

import gated_reference as gated
import memory_bound_elementwise_amd as mbe
from memory_bound_elementwise_amd import build as mbuild
from memory_bound_elementwise_amd.moe_block import load_library
from test_block_launches import STAND_IN

OK, INVALID, ALIGN = 0, 1, 2
BF16, F16, F32 = 0, 1, 2
A = 1 << 20            # an aligned address; tensors lie 2^40 apart
NAN, INF = float("nan"), float("inf")


def at(i):
    return A + (i << 40)


def gate(logits=at(0), dt=F32, bias=at(1), ids=at(2), probs=at(3), tokens=4, experts=48, k=4, scores=1, groups=4, top=2,
         group_top=2, renorm=1, scale=2.5, valid=None):
    return load_library().block_moe_gate_fwd(logits, dt, bias, ids, probs, tokens, experts, k, scores, groups, top,
                                             group_top, renorm, scale, valid, None)


RULES = (dict(experts=0), dict(experts=1025, groups=1, top=1), dict(k=0), dict(k=-1), dict(k=25), dict(k=65, groups=1, top=1,
         experts=128), dict(scores=2), dict(scores=-1), dict(groups=0), dict(groups=5), dict(groups=-4),
         dict(groups=65, experts=130), dict(top=0), dict(top=5), dict(group_top=0), dict(group_top=3),
         dict(groups=48, group_top=2, top=48), dict(scale=NAN), dict(scale=INF), dict(scale=-INF))


def test_gate_refusals():
    assert gate(tokens=0) == OK and gate(tokens=0, logits=None, ids=None, probs=None) == OK
    for bad in RULES + (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(dt=3), dict(dt=-1), dict(logits=None), dict(ids=None),
                        dict(probs=None), dict(ids=at(0)), dict(probs=at(2) + 16), dict(probs=at(1)), dict(ids=at(0) + 700),
                        dict(valid=at(2))):
        assert gate(**bad) == INVALID, bad
    for bad in (dict(logits=A + 4), dict(bias=at(1) + 2), dict(ids=at(2) + 2), dict(probs=at(3) + 1), dict(valid=at(5) + 2)):
        assert gate(**bad) == ALIGN, bad


def gate_bwd(logits=at(0), dt=F32, ids=at(1), g=at(2), out=at(3), tokens=4, experts=48, k=4, scores=0, renorm=0, scale=1.0,
             valid=None):
    return load_library().block_moe_gate_bwd(logits, dt, ids, g, out, tokens, experts, k, scores, renorm, scale, valid, None)


def test_gate_bwd_refusals():
    assert gate_bwd(tokens=0) == OK and gate_bwd(tokens=0, logits=None, out=None) == OK
    for bad in (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(experts=0), dict(experts=1025), dict(k=0), dict(k=65),
                dict(scores=2), dict(scale=NAN), dict(scale=INF), dict(dt=3), dict(logits=None), dict(ids=None), dict(g=None),
                dict(out=None), dict(out=at(0)), dict(out=at(1)), dict(out=at(2) - 32), dict(out=at(9), valid=at(9) + 4)):
        assert gate_bwd(**bad) == INVALID, bad
    for bad in (dict(logits=A + 8), dict(out=at(3) + 4), dict(ids=at(1) + 2), dict(g=at(2) + 2), dict(valid=at(5) + 1)):
        assert gate_bwd(**bad) == ALIGN, bad


def route(x=at(0), w=at(1), rdt=BF16, bias=at(2), ids=at(3), probs=at(4), tokens=4, hidden=64, experts=48, k=4, scores=1,
          groups=4, top=2, group_top=2, renorm=1, scale=2.5, valid=None, ws=at(5), size=1 << 30):
    return load_library().block_moe_route_gated(x, w, rdt, bias, ids, probs, tokens, hidden, experts, k, scores, groups, top,
                                                group_top, renorm, scale, valid, ws, size, None)


def test_route_refusals():
    need = load_library().block_moe_route_workspace(4, 64, 48)
    assert need > 0 and route(tokens=0) == OK
    for bad in RULES + (dict(tokens=-1), dict(tokens=(1 << 19) + 1), dict(hidden=0), dict(hidden=(1 << 20) + 8), dict(rdt=F16),
                        dict(x=None), dict(w=None), dict(ids=None), dict(probs=None), dict(ws=None), dict(size=need - 1),
                        dict(ids=at(0)), dict(probs=at(3)), dict(ws=at(1)), dict(ws=at(2)), dict(valid=at(3))):
        assert route(**bad) == INVALID, bad
    for bad in (dict(hidden=60), dict(x=A + 2), dict(w=at(1) + 8), dict(bias=at(2) + 2), dict(ids=at(3) + 2),
                dict(probs=at(4) + 1), dict(valid=at(6) + 2), dict(ws=at(5) + 8)):
        assert route(**bad) == ALIGN, bad


def quantize(w=at(0), dt=BF16, codes=at(1), scales=at(2), matrices=2, n=40, k=96):
    return load_library().block_fp4_quantize(w, dt, codes, scales, matrices, n, k, None)


def pack(e=at(0), x=at(1), codes=at(2), scales=at(3), matrices=2, n=40, k=96):
    return load_library().block_fp4_pack(e, x, codes, scales, matrices, n, k, None)


def dequantize(codes=at(0), scales=at(1), w=at(2), matrices=2, n=40, k=96):
    return load_library().block_fp4_dequantize(codes, scales, w, matrices, n, k, None)


SIZES = (dict(matrices=-1), dict(matrices=(1 << 16) + 1), dict(n=0), dict(k=0), dict(k=-32), dict(n=(1 << 20) + 1),
         dict(k=(1 << 20) + 32), dict(matrices=1 << 16, n=1 << 20, k=32), dict(matrices=3, n=1 << 20, k=1 << 16))


def test_weights_refusals():
    assert quantize(matrices=0) == OK and pack(matrices=0, e=None) == OK and dequantize(matrices=0, w=None) == OK
    for bad in SIZES:
        assert quantize(**bad) == pack(**bad) == dequantize(**bad) == INVALID, bad
    assert quantize(k=40) == pack(k=100) == dequantize(k=48) == ALIGN
    for bad in (dict(dt=3), dict(dt=-1), dict(w=None), dict(codes=None), dict(scales=None), dict(codes=at(0)),
                dict(codes=at(0) + 2 * 40 * 96 * 2 - 16), dict(scales=at(1) + 1024 * 2 * 3 - 64)):
        assert quantize(**bad) == INVALID, bad
    for bad in (dict(e=None), dict(x=None), dict(codes=None), dict(scales=None), dict(codes=at(1)), dict(scales=at(0))):
        assert pack(**bad) == INVALID, bad
    for bad in (dict(codes=None), dict(scales=None), dict(w=None), dict(w=at(0)), dict(w=at(1) - 64)):
        assert dequantize(**bad) == INVALID, bad
    for i in ("w", "codes", "scales"):
        assert quantize(**{i: at(5) + 4}) == dequantize(**{i: at(5) + 8}) == ALIGN
    for i in ("e", "x", "codes", "scales"):
        assert pack(**{i: at(5) + 4}) == ALIGN


def test_layout_sizes():
    lib = load_library()
    for n, k in ((1, 32), (16, 128), (17, 160), (4096, 7168), (1411, 1408)):
        codes, scales = mbe.fp4_shapes(n, k)
        assert lib.block_fp4_codes_bytes(n, k) == torch.Size(codes).numel()
        assert lib.block_fp4_scales_bytes(n, k) == torch.Size(scales).numel()
        assert lib.block_fp4_codes_bytes(n, k) * 2 >= n * k
    for n, k in ((0, 32), (16, 0), (16, 40), (1 << 21, 32), (16, 1 << 21), (-16, 32)):
        assert lib.block_fp4_codes_bytes(n, k) == lib.block_fp4_scales_bytes(n, k) == 0
    for n, k in ((0, 32), (16, 40), (16, 0)):
        with pytest.raises(ValueError):
            mbe.fp4_shapes(n, k)


def test_layout_of_the_reference():
    """Where single elements lie, as the header states it: byte and half of row, k."""
    n, k = 40, 288
    codes = torch.randint(0, 16, (n, k), generator=torch.Generator().manual_seed(0), dtype=torch.uint8)
    exps = torch.randint(0, 255, (n, k // 32), generator=torch.Generator().manual_seed(1), dtype=torch.uint8)
    c, s = gated.lay_out(codes, exps)
    for row, col in ((0, 0), (5, 7), (17, 130), (39, 287), (16, 96), (33, 33), (15, 127)):
        j, q, i = col % 128 // 32, col % 32 // 8, col % 8
        byte = int(c[row // 16, col // 128, (16 * q + row % 16) * 16 + 4 * j + i // 2])
        assert (byte >> 4 * (i % 2)) & 15 == int(codes[row, col])
        assert int(s[row // 16, col // 128, row % 16 * 4 + j]) == int(exps[row, col // 32])


def linear(x=at(0), codes=at(1), scales=at(2), b=at(3), r=at(4), y=at(5), m=4, n=16, k=64, act=1, ws=at(6), size=1 << 36):
    return load_library().block_linear_act_fp4(x, codes, scales, b, r, y, m, n, k, act, ws, size, None)


def test_linear_refusals():
    assert linear(m=0) == OK and linear(m=0, x=None, codes=None, y=None) == OK
    for bad in (dict(m=-1), dict(n=0), dict(k=0), dict(m=(1 << 24) + 1), dict(n=(1 << 20) + 8), dict(k=(1 << 20) + 32),
                dict(m=1 << 20, n=1 << 17), dict(m=1 << 20, k=1 << 17), dict(n=1 << 19, k=1 << 19), dict(act=4), dict(act=-1),
                dict(x=None), dict(codes=None), dict(scales=None), dict(y=None), dict(y=at(0)), dict(y=at(1)),
                dict(y=at(2) + 32), dict(y=at(3)), dict(y=at(4))):
        assert linear(**bad) == INVALID, bad
    for bad in (dict(n=12), dict(k=40), dict(x=A + 2), dict(codes=at(1) + 8), dict(scales=at(2) + 4), dict(b=at(3) + 2),
                dict(r=at(4) + 4), dict(y=at(5) + 2)):
        assert linear(**bad) == ALIGN, bad
    for m, n, k in ((17, 4096, 7168), (100, 64, 7168), (40, 72, 1 << 20), (16, 16384, 7168), (1, 16392, 7168)):  # split sums
        need = mbe.linear_act_fp4_workspace(m, n, k)
        assert need > 0 and need % (2 * m * n * 4) == 0
        assert linear(m=m, n=n, k=k, size=need - 1) == linear(m=m, n=n, k=k, ws=None) == INVALID
        assert linear(m=m, n=n, k=k, ws=at(1)) == linear(m=m, n=n, k=k, ws=at(2)) == INVALID
        assert linear(m=m, n=n, k=k, ws=at(6) + 4) == ALIGN
    for m, n, k in ((-1, 16, 64), (100, 12, 64), (100, 16, 40), (0, 16, 64), (16, 64, 7168), (4, 16384, 7168), (16, 8192, 7168), (65, 16, 64), (4096, 4096, 4096)):
        assert mbe.linear_act_fp4_workspace(m, n, k) == 0


def experts(x=at(0), uc=at(1), us=at(2), dc=at(3), ds=at(4), ids=at(5), probs=at(6), r=at(7), y=at(8), ydt=BF16, tokens=4,
            hidden=64, inter=32, n=8, k=2, act=4, limit=7.0, valid=None, ws=at(9), size=1 << 36):
    return load_library().block_moe_experts_fp4(x, uc, us, dc, ds, ids, probs, r, y, ydt, tokens, hidden, inter, n, k, act,
                                                limit, valid, ws, size, None)


def test_experts_refusals():
    need = mbe.moe_experts_fp4_workspace(4, 64, 32, 8, 2)
    assert need > 0 and experts(tokens=0) == OK and experts(tokens=0, x=None, uc=None, ws=None, size=0) == OK
    for bad in (dict(tokens=-1), dict(tokens=1025, k=1), dict(tokens=600), dict(hidden=0), dict(inter=0), dict(hidden=1 << 17),
                dict(inter=(1 << 16) + 32), dict(n=0), dict(n=1025), dict(k=0), dict(k=1025), dict(act=1), dict(act=5),
                dict(limit=0.0), dict(limit=-1.0), dict(limit=NAN), dict(ydt=F16), dict(x=None), dict(uc=None), dict(us=None),
                dict(dc=None), dict(ds=None), dict(ids=None), dict(probs=None), dict(y=None), dict(ws=None),
                dict(size=need - 1), dict(y=at(0)), dict(y=at(2)), dict(y=at(4)), dict(y=at(7)), dict(ws=at(1)), dict(ws=at(3)),
                dict(ws=at(8)), dict(valid=at(9))):
        assert experts(**bad) == INVALID, bad
    for bad in (dict(hidden=40), dict(inter=48), dict(x=A + 2), dict(uc=at(1) + 8), dict(us=at(2) + 4), dict(dc=at(3) + 4),
                dict(ds=at(4) + 8), dict(ids=at(5) + 2), dict(probs=at(6) + 2), dict(r=at(7) + 8), dict(y=at(8) + 4),
                dict(valid=at(11) + 2), dict(ws=at(9) + 8)):
        assert experts(**bad) == ALIGN, bad
    for bad in ((-1, 64, 32, 8, 2), (4, 40, 32, 8, 2), (4, 64, 16, 8, 2), (1024, 64, 32, 8, 2)):
        assert mbe.moe_experts_fp4_workspace(*bad) == 0


def test_bindings_refuse_before_any_call():
    """Types, shapes and placement, on tensors of the host."""
    f = torch.zeros
    logits, ids, probs = f(4, 16), f(4, 2, dtype=torch.int32), f(4, 2)
    codes, scales = (f(s, dtype=torch.uint8) for s in mbe.fp4_shapes(16, 64))
    with pytest.raises(ValueError):                          # the host's
        mbe.moe_gate_fwd(logits, ids, probs)
    with pytest.raises(TypeError):
        mbe.moe_gate_fwd(logits.double(), ids, probs)
    with pytest.raises(TypeError):
        mbe.moe_gate_fwd(logits, ids.long(), probs)
    with pytest.raises(TypeError):
        mbe.moe_gate_fwd(logits, ids, probs, bias=f(16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mbe.moe_gate_fwd(logits, ids, f(4, 3))
    with pytest.raises(ValueError):
        mbe.moe_gate_fwd(logits, ids, probs, scores="relu")
    with pytest.raises(ValueError):
        mbe.moe_gate_bwd(logits, ids, probs, f(4, 15))
    with pytest.raises(TypeError):
        mbe.moe_gate_bwd(logits, ids, probs, f(4, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mbe.fp4_quantize(f(16), codes, scales)
    with pytest.raises(TypeError):
        mbe.fp4_quantize(f(16, 64, dtype=torch.int8), codes, scales)
    with pytest.raises(ValueError):
        mbe.fp4_quantize(f(17, 64), codes, scales)
    with pytest.raises(ValueError):
        mbe.fp4_pack(f(16, 32, dtype=torch.uint8), f(16, 3, dtype=torch.uint8), codes, scales)
    with pytest.raises(ValueError):
        mbe.fp4_dequantize(codes, scales, f(2, 16, 64, dtype=torch.bfloat16))
    x = f(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mbe.linear_act_fp4(x, codes, scales, f(2, 24, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mbe.linear_act_fp4(x, codes, scales, f(2, 16, dtype=torch.bfloat16), activation="tanh")
    with pytest.raises(ValueError):
        mbe.moe_experts_fp4(x, codes, scales, codes, scales, ids[:2], probs[:2], x)
    with pytest.raises(ValueError):
        mbe.moe_experts_fp4(x, codes[None], scales[None], codes[None], scales[None], ids[:2], probs[:2], x,
                            activation="gelu")


# ---------------------------------------------------------------------------
# Launches
# ---------------------------------------------------------------------------
CALLER = r"""
import ctypes, json, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
vp, i64, i, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
at = lambda n: vp((1 << 20) + (n << 45))
big = i64(1 << 42)
out = (ctypes.c_uint * 448)()
got = []
for op, *a in json.loads(sys.argv[3]):
    if op == "gate":
        st = lib.block_moe_gate_fwd(at(0), i(a[2]), at(1), at(2), at(3), i64(a[0]), i(a[1]), i(1), i(1), i(1), i(1), i(1),
                                    i(0), f(1.0), None, None)
    elif op == "gate_bwd":
        st = lib.block_moe_gate_bwd(at(0), i(a[2]), at(1), at(2), at(3), i64(a[0]), i(a[1]), i(1), i(0), i(a[3]), f(1.0),
                                    None, None)
    elif op == "route":
        st = lib.block_moe_route_gated(at(0), at(1), i(0), at(2), at(3), at(4), i64(a[0]), i64(a[1]), i(a[2]), i(1), i(1),
                                       i(1), i(1), i(1), i(0), f(1.0), None, at(5), big, None)
    elif op == "quantize":
        st = lib.block_fp4_quantize(at(0), i(2), at(1), at(2), i64(a[0]), i64(a[1]), i64(a[2]), None)
    elif op == "pack":
        st = lib.block_fp4_pack(at(0), at(1), at(2), at(3), i64(a[0]), i64(a[1]), i64(a[2]), None)
    elif op == "dequantize":
        st = lib.block_fp4_dequantize(at(0), at(1), at(2), i64(a[0]), i64(a[1]), i64(a[2]), None)
    elif op == "linear":
        st = lib.block_linear_act_fp4(at(0), at(1), at(2), at(3), at(4), at(5), i64(a[0]), i64(a[1]), i64(a[2]), i(1), at(6),
                                      big, None)
    else:
        st = lib.block_moe_experts_fp4(at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), i(0), i64(a[0]),
                                       i64(a[1]), i64(a[2]), i(a[3]), i(a[4]), i(a[5]), f(7.0), None, at(9), big, None)
    n = fake.launches(out)
    got.append([st, [list(out[7 * k:7 * k + 7]) for k in range(n)]])
print(json.dumps(got))
"""

MOST = 1 << 25          # tiles of 16 x 128
CALLS = (
    [["gate", t, e, dt] for dt in (0, 2) for t, e in ((1, 1), (1 << 24, 1), (1 << 24, 64), (1 << 24, 256), (1 << 24, 1024),
                                                      (1025, 65), (3, 1024))] +
    [["gate_bwd", t, e, 2, r] for r in (0, 1) for t, e in ((1, 1), (1 << 24, 64), (1 << 24, 256), (1 << 24, 1024), (3, 300))] +
    [["route", t, h, e] for t, h, e in ((1, 8, 1), (1 << 19, 8, 64), (1 << 15, 1 << 20, 1024), (4, 1 << 20, 1024))] +
    [[op, *s] for op in ("quantize", "pack", "dequantize")
     for s in ((1, 1, 32), (1, 1 << 20, 32), (1, 16, 1 << 20), (2, 1 << 18, 1 << 16), (1 << 16, 16, 128), (MOST >> 10, 16, 1 << 17))] +
    [["linear", m, n, k] for m, n, k in ((1, 8, 32), (64, 1 << 20, 1 << 16), (65, 8, 1 << 20), (1 << 24, 8, 32),
                                         (16, 1 << 20, 32), (1 << 16, 1 << 20, 32), (17, 4096, 1 << 20))] +
    [["experts", *s, act] for act in (3, 4)
     for s in ((1, 32, 32, 1, 1), (1024, 1 << 16, 1 << 16, 1024, 1), (16, 1 << 16, 1 << 16, 64, 64),
               (1, 1 << 16, 1 << 16, 1024, 64), (64, 7168, 2048, 64, 8), (128, 256, 256, 8, 8), (1024, 64, 64, 1, 1))])


@pytest.fixture(scope="module")
def launched(tmp_path_factory):
    load_library()
    d = tmp_path_factory.mktemp("gate_fp4_launches")
    (d / "stand_in.c").write_text(STAND_IN)
    (d / "caller.py").write_text(CALLER)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", d / "stand_in.so", d / "stand_in.c"], check=True)
    res = subprocess.run([sys.executable, d / "caller.py", d / "stand_in.so", mbuild.lib_path("moe_block"),
                          json.dumps(CALLS)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    return dict(zip(map(tuple, CALLS), json.loads(res.stdout)))


@pytest.mark.parametrize("call", CALLS, ids=lambda c: "-".join(map(str, c)))
def test_every_launch_fits_a_dispatch(launched, call):
    """A dispatch counts its work-items in 32 bits an axis, workgroups have at most 1024 threads, grid
    axes y and z 65535 workgroups."""
    status, shapes = launched[tuple(call)]
    assert status == 0 and 1 <= len(shapes) <= 4
    for gx, gy, gz, bx, by, bz, lds in shapes:
        assert min(gx, gy, gz, bx) >= 1 and by == bz == 1 and bx <= 1024 and bx % 64 == 0
        assert gx * bx <= 0xffffffff and gy <= 65535 and gz <= 65535
        assert lds <= 128 * 1024
