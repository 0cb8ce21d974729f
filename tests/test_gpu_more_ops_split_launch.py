"""The norms, products and log probabilities in consecutive launches (those of more than 2^31
work-items are split; in the build that is loaded here those of more than 2048): their tests in a
child process, through ZERO_OPS_LIB."""
import os
import re

import pytest

from test_gpu_ops_split_launch import _child

pytestmark = pytest.mark.gpu

FILES = ["test_gpu_ops_rms.py", "test_gpu_ops_pack.py", "test_gpu_ops_product.py", "test_gpu_ops_logprobs.py"]


def test_the_operators_hold_over_consecutive_launches():
    # (without the largest: as many small launches as they would take say nothing more)
    r = _child(["-u", "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu", "-k", "not test_many and not test_large_tiles",
                *[os.path.join("tests", f) for f in FILES]], 100)
    tail = r.stdout[-3000:] + r.stderr[-2000:]
    print(tail)
    assert r.returncode == 0, tail
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) > 300 and " failed" not in r.stdout, tail
