"""The gate's exponential, compiled for the host: its error against long double, its ends, and no undefined
step on the way (a conversion of NaN among them)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "memory_bound_elementwise_amd", "csrc")

DRIVE = r"""
#include <cmath>
#include <cstdio>
#include <cstdlib>
#define __device__
#define __forceinline__ inline
#include "gate_math.h"
int main()
{
    double worst = 0;
    for (int i = 0; i < 2000000; ++i) {
        const double v = -708.0 * std::pow(i / 2000000.0, 3);
        const long double exact = expl((long double)v);
        const double step = std::nextafter((double)exact, 2.0) - (double)exact;
        const double off = std::fabs((double)(((long double)block::exp_below(v) - exact) / step));
        worst = off > worst ? off : worst;
    }
    std::printf("worst %.3f\n", worst);
    for (double v = -708; v > -760; v -= 0.01) {  // subnormal numbers, then zeros
        const double off = std::fabs((double)((long double)block::exp_below(v) - expl((long double)v)));
        if (off > 0x1p-1074)
            return std::printf("off %g at %g\n", off, v), 1;
    }
    const double inf = HUGE_VAL;
    if (block::exp_below(0.0) != 1.0 || block::exp_below(-0.0) != 1.0 || block::exp_below(-inf) != 0.0 ||
        block::exp_below(-1e300) != 0.0 || block::exp_below(-746.0) != 0.0)
        return std::printf("ends\n"), 1;
    if (!std::isnan(block::exp_below(std::nan(""))) || !std::isnan(block::exp_below(-std::nan(""))))
        return std::printf("NaN\n"), 1;
    std::printf("ok\n");
    return worst < 1.0 ? 0 : 1;
}
"""


@pytest.mark.skipif(bool(os.environ.get("LD_PRELOAD")) or os.path.exists("/etc/ld.so.preload"),
                    reason="a preloaded library would come before the sanitizer runtime")
def test_exponential(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    (tmp_path / "drive.cpp").write_text(DRIVE)
    cmd = [gxx, "-std=c++17", "-O2", "-ffp-contract=off", "-Wno-unknown-pragmas", f"-I{CSRC}",
           "-fsanitize=undefined,float-cast-overflow", "-fno-sanitize-recover=all", "-o", str(tmp_path / "drive"),
           str(tmp_path / "drive.cpp"), "-lm"]
    built = subprocess.run(cmd, capture_output=True, text=True)
    assert built.returncode == 0, built.stderr[-3000:]
    ran = subprocess.run([str(tmp_path / "drive")], capture_output=True, text=True, timeout=120)
    assert ran.returncode == 0 and "ok" in ran.stdout, ran.stdout + ran.stderr[-2000:]
