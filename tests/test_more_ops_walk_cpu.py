"""The sizes of the GPU tests of low tiles that walk, by the library's own plan: more tiles of 64 rows than workgroups
stand in the CUs, and one such workgroup to a CU."""
import os
import subprocess

import pytest

from conftest import ROOT
from test_gpu_ops_product_walk import SIZES
from zero_dp_sharded_amd import build as B

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ops_internal.h"
int main(int c, char** v)
{
    std::printf("%d %d %d\n", zo::product_tiles_in_cu(false, 2), zo::product_tiles_in_cu(false, 4), zo::product_tiles_in_cu(false, 8));
    for (int k = 1; k + 2 < c; k += 3) {
        const int64_t m = atoll(v[k]), n = atoll(v[k + 1]);
        const zo::ProductPlan p = zo::product_plan(m, n, atoll(v[k + 2]), 2);
        std::printf("%d %lld %d\n", p.ni, (long long)(zo::product_tiles_in_cu(false, 2) * 256), (int)((m + 63) / 64 * ((n + 255) / 256) * p.splits));
    }
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    at = tmp_path_factory.mktemp("walk")
    src, exe = at / "walk.cpp", at / "walk"
    src.write_text(PROGRAM)
    lib = os.path.join(ROOT, "zero_dp_sharded_amd")
    r = subprocess.run([B.HIPCC, "-O1", "-std=c++17", "-x", "hip", "--offload-host-only", f"-I{B.CSRC}", str(src), "-o", str(exe),
                        f"-L{lib}", "-lzeroops", f"-Wl,-rpath,{lib}"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([str(exe)] + [str(x) for size in SIZES for x in size], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    return [tuple(int(x) for x in line.split()) for line in out.stdout.splitlines()]


def test_a_tile_of_8_bits_has_a_cu_to_itself(lines):
    assert lines[0] == (1, 1, 1)


def test_the_sizes_walk(lines):
    assert len(lines) == 1 + len(SIZES)
    for ni, stand, tiles in lines[1:]:
        assert ni == 2 and tiles > stand
