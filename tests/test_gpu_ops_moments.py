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


@pytest.mark.parametrize("spread", [4, 10, 14])
def test_gradients_that_differ_within_a_block_move_as_adam_does(spread):
    """Blocks whose gradients are constant, one element's 2^spread times the others': Adam
    moves every element by lr a step.  With 8-bit moments none may move by more than twice
    that, in any of 1500 steps (the times of decay of exp_avg_sq are 1000), and all of them by
    that in the mean, within a tenth: v's relative spread about its value, from roundings up or
    down by at most an eighth at a rate of a thousandth, is at most 1 / 4, and the mean of
    1 / sqrt(v) is off by at most 3 / 8 of its square."""
    n, steps = 256 * 16, 1500
    grad = torch.full((n,), 2.0 ** -spread, device=DEV)
    grad[::256] = 1.0
    master = torch.zeros(n, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    em, ev = (torch.zeros(n // 256, dtype=torch.int8, device=DEV) for _ in range(2))
    hp = zs.AdamHParams(lr=1.0, beta1=0.9, beta2=0.999, eps=1e-30, weight_decay=0.0)
    h = zs.zero_adamw_init([zs.AdamWTensor(grad, master, None, m, v, em, ev)], hp=hp, ls=zs.LossScaleCfg(init_scale=1.0, dynamic=0),
                           state_bits=8, checked=False, seed=5)
    largest = torch.zeros((), device=DEV)
    try:
        for _ in range(steps):
            before = master.clone()
            zs.zero_adamw_step(h)
            largest = torch.maximum(largest, (before - master).abs().max())
    finally:
        zs.zero_adamw_destroy(h)
    rest = torch.arange(n, device=DEV) % 256 != 0
    assert largest.item() <= 2.0 + 1e-3
    assert abs(master[rest].double().mean().item() / -steps - 1.0) <= 0.1
