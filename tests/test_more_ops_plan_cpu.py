"""The forms that the scaled product and the log probabilities take, by the library's own plan, for the sizes of
the GPU tests: every form is among them."""
import os
import re
import subprocess

import pytest

from conftest import ROOT
from zero_dp_sharded_amd import build as B

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ops_internal.h"
int main(int c, char** v)
{
    for (int k = 1; k + 3 < c; k += 4) {
        const int64_t x = atoll(v[k + 1]), y = atoll(v[k + 2]), z = atoll(v[k + 3]);
        if (v[k][0] == 'l') {
            const zo::LogprobPlan p = zo::logprob_plan(x, y, z, 8192, 0), top = zo::logprob_plan(x, y, z, 8192, y < 20 ? 1 : 20);
            std::printf("%d %d %d %d %d\n", p.tile.ni, p.tile.nj, top.tile.ni, top.tile.nj, (int)(p.pieces > 1024));
        } else {
            const zo::ProductPlan p = zo::product_plan(x, y, z, v[k][0] == 'f' ? 3 : 2);
            std::printf("%d %d %d\n", p.ni, p.splits, (int)p.exact);
        }
    }
}
"""


def listed(file):
    """The sizes that a file's lists name: three numbers, or four of which the first three are."""
    text = open(os.path.join(ROOT, "tests", file)).read()
    found = []
    for m in re.finditer(r"^(?:SIZES = |@pytest\.mark\.parametrize\(\"(?:m,n,k|n,v,d|n,v,d,top)\", )\[(.*?)\]\)?$", text, re.M | re.S):
        found += [tuple(int(x) for x in t.split(",")[:3]) for t in re.findall(r"\(([\d, ]+)\)", m.group(1))]
    return sorted(set(found))


PRODUCTS, SCORES = listed("test_gpu_ops_product.py"), listed("test_gpu_ops_logprobs.py")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    src, exe = at / "plan.cpp", at / "plan"
    src.write_text(PROGRAM)
    lib = os.path.join(ROOT, "zero_dp_sharded_amd")
    r = subprocess.run([B.HIPCC, "-O1", "-std=c++17", "-x", "hip", "--offload-host-only", f"-I{B.CSRC}", str(src), "-o", str(exe),
                        f"-L{lib}", "-lzeroops", f"-Wl,-rpath,{lib}"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    calls = [("f", *s) for s in PRODUCTS] + [("b", *s) for s in PRODUCTS] + [("l", *s) for s in SCORES]
    out = subprocess.run([str(exe)] + [str(x) for call in calls for x in call], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    return {call: tuple(int(x) for x in line.split()) for call, line in zip(calls, out.stdout.splitlines())}


def test_every_form_of_the_product_is_among_the_tests_sizes(plans):
    two = {plans[("b", *s)] for s in PRODUCTS}
    four = {plans[("f", *s)] for s in PRODUCTS}
    assert {ni for ni, _, exact in two if not exact} == {0, 2, 4, 8}
    assert {ni for ni, _, exact in four if ni} == {2, 6, 8} and all(exact for ni, _, exact in four if ni) and 0 in {ni for ni, _, _ in four}
    for forms, tiles in ((two, (2, 4, 8)), (four, (2, 6, 8))):
        for ni in tiles:
            parts = {splits > 1 for n, splits, _ in forms if n == ni}
            assert False in parts, ni
        assert any(splits > 1 for n, splits, _ in forms if n)


def test_every_form_of_the_log_probabilities_is_among_the_tests_sizes(plans):
    forms = [plans[("l", *s)] for s in SCORES]
    assert {(ni, nj) for ni, nj, *_ in forms} == {(2, 4), (8, 4), (8, 5)}
    assert {(ni, nj) for _, _, ni, nj, _ in forms} == {(2, 4), (8, 4)}
    assert {many for *_, many in forms} == {0, 1}
