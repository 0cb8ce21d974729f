"""The bias-correction power on the host: the bits of t multiplications, and an end
for every counter (a restored step counter has no upper limit)."""
import shutil
import subprocess

import pytest

from zero_dp_sharded_amd import build as B

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include "beta_pow.h"
static double plain(double beta, int64_t t)
{
    const double b = (double)(float)beta;
    volatile double p = 1.0;
    for (int64_t k = 0; k < t; ++k) p = p * b;
    return p;
}
int main()
{
    const double betas[] = {0.0, 0.1, 0.5, 0.50001, 0.9, 0.95, 0.99, 0.999, 0.9999};
    const int64_t ts[] = {0, 1, 2, 3, 10, 999, 1074, 1075, 1076, 7000, 7100, 100000, 800000};
    for (double b : betas)
        for (int64_t t : ts) {
            const double x = beta_pow(b, t), y = plain(b, t);
            if (std::memcmp(&x, &y, sizeof x)) { std::printf("beta %g t %lld: %a, not %a\n", b, (long long)t, x, y); return 1; }
        }
    // after the last change: the product for ever
    for (double b : betas)
        for (int64_t t : {int64_t(1) << 40, INT64_MAX})
            if (beta_pow(b, t) != beta_pow(b, int64_t(1) << 24)) { std::printf("beta %g\n", b); return 1; }
    std::printf("ok\n");
    return 0;
}
"""


def test_the_same_bits_and_an_end(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "p.cpp", tmp_path / "p"
    src.write_text(PROGRAM)
    r = subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", f"-I{B.CSRC}", str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    # (t multiplications of 2^40 would take an hour)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout
