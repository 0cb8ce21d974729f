"""Packing and unpacking of 8-bit moments: what existing tests of the codes leave out."""
import pytest
import torch

import zero_dp_sharded_amd as zs
from test_gpu_ops_adamw import DEV, unpack

pytestmark = pytest.mark.gpu


def pack(x, signed):
    n = x.numel()
    codes, exps = torch.full((n,), 85, dtype=torch.uint8, device=DEV), torch.full((-(-n // 256),), 3, dtype=torch.int8, device=DEV)
    zs.zero_moments_pack(x, codes, exps, signed=signed)
    return codes, exps


def test_negative_values_of_a_moment_without_sign_count_as_zeros():
    """They do not set their block's exponent either: the others keep their places."""
    n = 1500
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(n, generator=g, device=DEV).square() * 1e-8
    x[::7] = 0.0
    want = pack(x, False)
    for value in (-1e6, -3e38, -1e-30, float("-inf")):
        y = x.clone()
        y[::7] = value
        got = pack(y, False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), value
    # a block of nothing else is zeros
    c, e = pack(torch.full((300,), -5.0, device=DEV), False)
    assert not c.any() and (e == -100).all() and not unpack(c, e, False).any()
    # NaN is no negative value
    x[300] = float("nan")
    c, e = pack(x, False)
    y = unpack(c, e, False)
    assert torch.isnan(y[256:512]).all() and torch.isfinite(y[:256]).all() and torch.isfinite(y[512:]).all()
