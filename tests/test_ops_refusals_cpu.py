"""Refusals of the training operators that need no GPU, beyond test_ops_cpu.py."""
import pytest

import zero_dp_sharded_amd as zs
from test_ops_cpu import loss


@pytest.mark.parametrize("scale", [1e39, -1e39, 1.7e308, 3.4028236e38])
def test_a_gradient_scale_that_is_infinite_in_fp32(scale):
    """Gradients that are zeros (no tokens, or none that counts) would be 0 times infinity."""
    for kw in (dict(), dict(tokens=0)):
        s, msg = loss(grad_scale=scale, **kw)
        assert s == zs.ZERO_ERR_INVALID_ARG and "grad_scale" in msg, (s, msg)


def test_the_largest_gradient_scale_is_taken():
    s, msg = loss(grad_scale=3.4028234e38)              # (the call goes on to the device, which is not here)
    assert "grad_scale" not in msg
