"""The operators' consecutive launches.  Work of more than 2^31 work-items (33M rows of up
to 512 elements, 2M of more than 8192, 8.6e9 elements) goes in consecutive launches;
__graft_entry__.build() also builds the library with every launch split after 2048
work-items (zero_dp_sharded_amd/variants/split_launch/libzeroops.so), and the operators'
tests run against that build in a child process through ZERO_OPS_LIB."""
import os
import re
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

SPLIT_LIB = os.path.join(ROOT, "zero_dp_sharded_amd", "variants", "split_launch", "libzeroops.so")
FILES = ["test_gpu_ops_norm.py", "test_gpu_ops_norm_values.py", "test_gpu_ops_norm_many.py", "test_gpu_ops_adamw.py",
         "test_gpu_ops_adamw_values.py", "test_gpu_ops_adamw_many.py", "test_gpu_ops_moments.py", "test_gpu_ops_loss.py"]


def _child(args, timeout):
    if not os.path.exists(SPLIT_LIB):
        pytest.fail(f"{SPLIT_LIB} is missing: run __graft_entry__.build()")
    env = dict(os.environ, ZERO_OPS_LIB=SPLIT_LIB, PYTHONPATH=os.pathsep.join([ROOT, os.environ.get("PYTHONPATH", "")]))
    return subprocess.run([sys.executable, *args], cwd=ROOT, env=env, capture_output=True, text=True, timeout=timeout)


def test_the_operators_hold_over_consecutive_launches():
    r = _child(["-u", "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu", *[os.path.join("tests", f) for f in FILES]], 300)
    tail = r.stdout[-3000:] + r.stderr[-2000:]
    print(tail)
    assert r.returncode == 0, tail
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) > 130 and " failed" not in r.stdout, tail


def test_the_child_loads_the_split_build():
    r = _child(["-c", "import zero_dp_sharded_amd as zs; zs.zero_ops_abi_version(); print('library', zs.ops.LIB_PATH)"], 120)
    assert r.returncode == 0 and f"library {SPLIT_LIB}" in r.stdout, r.stdout + r.stderr


def test_more_rows_than_a_launch_holds():
    """More than 2^26 rows of 8: a wave a row would be 2^32 work-items.  16384 blocks of the
    same 4099 rows, so every block must come out as the rows alone do (in place)."""
    import torch
    import zero_dp_sharded_amd as zs
    blocks, period, width = 16384, 4099, 8
    rows = blocks * period
    assert rows > 1 << 26
    g = torch.Generator(device="cuda").manual_seed(1)
    few = torch.randn(period, width, generator=g, device="cuda").half()
    w = torch.randn(width, generator=g, device="cuda").half()
    want, mean0, rstd0 = torch.empty_like(few), torch.empty(period, device="cuda"), torch.empty(period, device="cuda")
    zs.zero_layernorm_forward(few, w, w, want, mean0, rstd0)
    x = few.expand(blocks, period, width).contiguous()
    flat = x.view(rows, width)
    mean, rstd = torch.full((rows,), float("nan"), device="cuda"), torch.full((rows,), float("nan"), device="cuda")
    zs.zero_layernorm_forward(flat, w, w, flat, mean, rstd)
    for k in range(0, blocks, 1024):
        part = slice(k, k + 1024)
        assert (x[part] == want).all() and (mean.view(blocks, period)[part] == mean0).all()
        assert (rstd.view(blocks, period)[part] == rstd0).all()
