"""The division by a number of query heads as a product, for every number that a call may have: compiled from its header on
the host, against the division itself."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "up_proj_gemm_gb300", "csrc")
PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "checks.h"
int main() {
    const int64_t top = 2147483647;
    int64_t ds[400], n = 0;
    for (int64_t d = 1; d <= 130; ++d) ds[n++] = d;
    for (int b = 8; b < 31; ++b)
        for (int64_t o = -1; o <= 1; ++o) ds[n++] = ((int64_t)1 << b) + o;
    for (int64_t d = top; d > top - 5; --d) ds[n++] = d;
    for (int64_t d = 1000003; d < top; d = d * 3 + 1) ds[n++] = d;
    for (int64_t i = 0; i < n; ++i) {
        const int64_t d = ds[i];
        const mlaq::Divisor v = mlaq::divisor((int32_t)d);
        uint64_t x = 12345;
        for (int k = 0; k < 4000; ++k) {
            x = x * 6364136223846793005ull + 1442695040888963407ull;
            const int64_t m = (int64_t)(x >> 33), q = m / d * d;  // a number, and those around a multiple
            for (const int64_t a : {m, q, q - 1, q + d - 1, top})
                if (a >= 0 && a <= top && (int64_t)((uint64_t)(uint32_t)a * v.mul >> v.shift) != a / d)
                    return std::printf("%lld / %lld\n", (long long)a, (long long)d), 1;
        }
    }
    return std::puts("ok"), 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no compiler")
def test_every_divisor(tmp_path):
    source, program = tmp_path / "division.cpp", tmp_path / "division"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", CSRC,
                    str(source), "-o", str(program)], check=True, timeout=120)
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
