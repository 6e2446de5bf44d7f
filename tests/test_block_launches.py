"""What libmoe_block.so launches for the largest and the smallest sizes its header accepts, on the
host: a stand-in for hipLaunchKernel notes each launch's shape and starts nothing."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

from memory_bound_elementwise_amd import build as mbuild

STAND_IN = r"""
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3_t;
static unsigned noted[64][7];
static int count;
int hipLaunchKernel(const void *f, dim3_t grid, dim3_t block, void **args, size_t lds, void *stream)
{
    (void)f; (void)args; (void)stream;
    if (count < 64) {
        unsigned *n = noted[count++];
        n[0] = grid.x; n[1] = grid.y; n[2] = grid.z; n[3] = block.x; n[4] = block.y; n[5] = block.z; n[6] = (unsigned)lds;
    }
    return 0;
}
int launches(unsigned *out)
{
    int n = count;
    for (int i = 0; i < n * 7; ++i) out[i] = noted[i / 7][i % 7];
    count = 0;
    return n;
}
"""

CALLER = r"""
import ctypes, json, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
vp, i64, i, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
at = lambda n: vp((1 << 20) + (n << 45))
big = i64(1 << 41)
out = (ctypes.c_uint * 448)()
got = []
for call in json.loads(sys.argv[3]):
    op, a = call[0], call[1:]
    if op == "norm_fwd":
        st = lib.block_layer_norm_fwd(at(0), at(1), at(2), at(3), at(4), at(5), i64(a[0]), i64(a[1]), f(1e-5), i(a[2]),
                                      i(2), None)
    elif op == "norm_bwd":
        st = lib.block_layer_norm_bwd(at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), i64(a[0]), i64(a[1]), i(a[2]),
                                      i(2), at(8), big, None)
    elif op == "linear":
        st = lib.block_linear_act(at(0), at(1), at(2), at(3), at(4), i64(a[0]), i64(a[1]), i64(a[2]), i(1), i(0), at(5),
                                  big, None)
    elif op == "route":
        st = lib.block_moe_route(at(0), at(1), i(0), at(2), at(3), i64(a[0]), i64(a[1]), i(a[2]), i(1), i(0), None, at(4),
                                 big, None)
    else:
        st = lib.block_moe_layer(at(0), at(1), i(0), at(2), at(3), at(4), at(5), i(0), at(6), at(7), i64(a[0]), i64(a[1]),
                                 i64(a[2]), i(a[3]), i(a[4]), i(0), i(a[5]), f(7.0), None, at(8), big, None)
    n = fake.launches(out)
    got.append([st, [list(out[7 * k:7 * k + 7]) for k in range(n)]])
print(json.dumps(got))
"""

BF16, F32 = 0, 2
SWIGLU, SQUARED_RELU = 4, 3
CALLS = (
    [["norm_" + d, rows, cols, dt] for d in ("fwd", "bwd") for dt in (BF16, F32)
     for rows, cols in ((1, 1), (1, 1 << 20), (1 << 19, 1 << 20), (1 << 22, 16392), (1 << 22, 65537), (1 << 36, 8),
                        (1 << 38, 1), (1 << 26, 7168), (1 << 25, 16384))] +
    [["linear", m, n, k] for m, n, k in ((1, 8, 8), (32, 1 << 20, 1 << 16), (33, 8, 1 << 20), (1 << 24, 8, 8),
                                         (1 << 24, 4096, 4096), (1 << 16, 1 << 20, 8), (257, 1 << 20, 1 << 16),
                                         (4096, 4096, 1 << 20))] +
    [["route", t, h, e] for t, h, e in ((1, 8, 1), (1 << 19, 8, 64), (1 << 15, 1 << 20, 1024), (4, 1 << 20, 1024),
                                        (1 << 19, 1 << 10, 8))] +
    [["layer", t, h, i, e, k, act] for act in (SWIGLU, SQUARED_RELU)
     for t, h, i, e, k in ((1, 8, 8, 1, 1), (1024, 1 << 16, 1 << 16, 1024, 1), (16, 1 << 16, 1 << 16, 64, 64),
                           (1, 1 << 16, 1 << 16, 1024, 64), (64, 7168, 2048, 64, 8), (65, 7168, 2048, 64, 8),
                           (128, 1 << 16, 1 << 16, 8, 8), (128, 256, 256, 1024, 1), (4, 8, 8, 64, 64),
                           (64, 1 << 16, 1 << 16, 16, 16), (127, 64, 64, 2, 1))])


@pytest.fixture(scope="module")
def launched(tmp_path_factory):
    if not os.path.exists(mbuild.lib_path("moe_block")):
        mbuild.build_lib("moe_block")
    d = tmp_path_factory.mktemp("launches")
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
    axes y and z 65535 workgroups, and a workgroup 160 KB of shared memory."""
    status, shapes = launched[tuple(call)]
    assert status == 0 and 1 <= len(shapes) <= 5
    for gx, gy, gz, bx, by, bz, lds in shapes:
        assert min(gx, gy, gz, bx) >= 1 and by == bz == 1 and bx <= 1024 and bx % 64 == 0
        assert gx * bx <= 0xffffffff and gy <= 65535 and gz <= 65535
        assert lds <= 64 * 1024
