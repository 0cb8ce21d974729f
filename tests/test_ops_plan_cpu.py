"""The tiles and parts that the vocabulary loss takes, by the library's own plan, for the
sizes that the GPU tests of large tiles have: each reaches what it is there for."""
import os
import subprocess

import pytest

from conftest import ROOT
from test_gpu_ops_loss_many import CASES
from zero_dp_sharded_amd import build as B

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ops_internal.h"
static long long tiles(int64_t rows, int64_t columns, zo::TileChoice t)
{
    return ((rows + 32 * t.ni - 1) / (32 * t.ni)) * ((columns + 64 * t.nj - 1) / (64 * t.nj));
}
int main(int c, char** v)
{
    for (int k = 1; k + 3 < c; k += 4) {
        const int64_t most = atoll(v[k + 3]);
        const zo::LossPlan p = zo::loss_plan(atoll(v[k]), atoll(v[k + 1]), atoll(v[k + 2]), most ? most : 8192, true);
        std::printf("%d %d %lld %d %d %d %d %d %d %lld %d\n", p.logits_tile.ni, p.logits_tile.nj, tiles(p.chunk, p.vocab, p.logits_tile),
                    p.hidden_tile.ni, p.hidden_tile.nj, p.hidden_splits, p.weight_tile.ni, p.weight_tile.nj, p.weight_splits,
                    (long long)(p.chunk * p.vocab_ld * 2), (int)p.pairs);
    }
}
"""
WORKGROUPS = {8: 256, 2: 512}           # of the logits, by the tile's rows
LAST_CACHE = 256 << 20


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    src, exe = at / "plan.cpp", at / "plan"
    src.write_text(PROGRAM)
    lib = os.path.join(ROOT, "zero_dp_sharded_amd")
    r = subprocess.run([B.HIPCC, "-O1", "-std=c++17", "-x", "hip", "--offload-host-only", f"-I{B.CSRC}", str(src), "-o", str(exe),
                        f"-L{lib}", "-lzeroops", f"-Wl,-rpath,{lib}"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([str(exe)] + [str(x) for size in CASES for x in size], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    return {size: [int(x) for x in line.split()] for size, line in zip(CASES, out.stdout.splitlines())}


@pytest.mark.parametrize("size", CASES)
def test_the_plan_of_a_size(plans, size):
    li, lj, tiles, hi, hj, hs, wi, wj, ws, held, _ = plans[size]
    got = ((li, lj), tiles > WORKGROUPS[li], (hi, hj), hs > 1, (wi, wj), ws > 1, held > LAST_CACHE)
    assert got == CASES[size]


def test_every_form_is_among_them(plans):
    for product in ("logits", "hidden", "weight"):
        at = {"logits": 0, "hidden": 2, "weight": 4}[product]
        assert {c[at] for c in CASES.values()} == {(8, 4), (8, 5), (2, 4)}
    for kind in ((8, 4), (8, 5)):
        assert any(c[0] == kind and c[1] for c in CASES.values())               # a walk over tiles
        assert any(c[0] == kind and c[6] for c in CASES.values())               # past the last cache
        assert {c[3] for c in CASES.values() if c[2] == kind} >= {True}         # parts
        assert {c[5] for c in CASES.values() if c[4] == kind} == {True, False}
    assert any(c[2] == (8, 5) and not c[3] for c in CASES.values())
    assert plans[(20, 140003, 24, 0)][-1] == 1 and plans[(100, 70001, 40, 0)][-1] == 0
