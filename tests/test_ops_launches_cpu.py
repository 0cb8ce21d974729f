"""How the operators cut work that one launch cannot hold (HIP counts a launch's
work-items in 32 bits), on the host: in_launches of ops_common.h covers every
workgroup once, in order, and no launch passes the limit, at the largest sizes that the C
ABI takes and under the small limit of the build that the GPU tests run."""
import os
import subprocess

import pytest

from conftest import ROOT
from zero_dp_sharded_amd import build as B

PROGRAM = r"""
#include <cstdio>
#include "ops_common.h"
int main()
{
    const int64_t groups[] = {0, 1, 2, 7, 8, 9, 1000, (int64_t(1) << 21) - 1, int64_t(1) << 21, (int64_t(1) << 21) + 1,
                              int64_t(1) << 23, (int64_t(1) << 25) + 3, (int64_t(1) << 31) - 1,   // rows
                              int64_t(1) << 30};                                                  // 2^40 moments by 1024
    const int lanes[] = {64, 256, 1024};
    for (int64_t g : groups)
        for (int l : lanes) {
            if (g / (zo::kMaxLaunchItems / l) > 4000000) continue;
            int64_t next = 0, launches = 0;
            bool fine = true;
            zo::in_launches(g, l, [&](int64_t first, int64_t count) {
                fine = fine && first == next && count > 0 && count * l <= zo::kMaxLaunchItems && count <= 0x7fffffff;
                next += count;
                ++launches;
            });
            if (!fine || next != g) { std::printf("wrong at %lld x %d\n", (long long)g, l); return 1; }
            if ((g * l > zo::kMaxLaunchItems) != (launches > 1)) { std::printf("launches at %lld x %d\n", (long long)g, l); return 1; }
        }
    std::printf("ok %lld\n", (long long)zo::kMaxLaunchItems);
    return 0;
}
"""


@pytest.mark.parametrize("limit", [None, B.OPS_SPLIT_LAUNCH_DEFINES["ZO_MAX_LAUNCH_ITEMS"]])
def test_every_workgroup_once_and_no_launch_past_the_limit(tmp_path, limit):
    src, exe = tmp_path / "launches.cpp", tmp_path / "launches"
    src.write_text(PROGRAM)
    define = [] if limit is None else [f"-DZO_MAX_LAUNCH_ITEMS={limit}"]
    r = subprocess.run([B.HIPCC, "-O1", "-std=c++17", "-x", "hip", "--offload-host-only", *define, f"-I{B.CSRC}", str(src), "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
    assert out.stdout.strip() == f"ok {2 ** 31 if limit is None else limit}"


def test_launches_over_rows_or_elements_go_through_it():
    """Kernel launches whose grid grows with rows or elements without a bound."""
    grows = {"ops_norm.hip": ("forward_kernel", "forward_long_kernel", "backward_long_kernel"),
             "ops_adamw.hip": ("update_kernel", "pack_kernel", "unpack_kernel"), "ops_loss.hip": ("repack_kernel",)}
    for name, kernels in grows.items():
        text = open(os.path.join(ROOT, "zero_dp_sharded_amd", "csrc", name), encoding="utf-8").read()
        for line in text.splitlines():
            if "<<<" in line and any(k + "<" in line for k in kernels):
                assert "count" in line, (name, line)
