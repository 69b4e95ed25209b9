"""The parts an expert's rows are split into by the weight gradient (csrc/rgg_wgrad_parts.h, plain host code): they
follow each other, cover every row once and start on whole stages, up to the largest expert the library takes."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ragged_grouped_gemm_02_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "rgg_wgrad_parts.h"
using namespace rgg;
int main() {
    const int32_t top = 2147483647;
    const int32_t sizes[] = {0, 1, 63, 64, 65, 4095, 4096, 4097, 15000, 1 << 20, top - 4096, top - 64, top - 32, top - 31,
                             top - 30, top - 15, top - 1, top};
    for (int32_t m : sizes)
        for (int32_t split = 2; split <= 32; split *= 2) {
            int64_t next = 0, share = 0;
            for (int32_t part = 0; part < split; ++part) {
                const WgradPart p = wgrad_part(m, split, part);
                if (part == 0) share = p.rows;
                const bool short_ok = p.rows == share || next + p.rows == m;
                if (p.rows < 0 || p.first != next || !short_ok || (p.rows > 0 && p.first % kWgradRows != 0)) {
                    std::printf("part %d of %d of %d rows: first %d, %d rows, expected first %lld\n", part, split, m,
                                p.first, p.rows, static_cast<long long>(next));
                    return 1;
                }
                next += p.rows;
            }
            if (next != m) return 2;
        }
    std::printf("ok\n");
    return 0;
}
"""


def test_parts(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "parts.cc").write_text(PROGRAM)
    r = subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "parts.cc"), "-o",
                        str(tmp_path / "parts")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(tmp_path / "parts")], capture_output=True, text=True, timeout=30)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
