"""The RMS norm's eps enters the sums in 64 bits as it is given: rstd is off by its own rounding to fp32 alone
(2^-24 of itself, and a few roundings of 64 bits), also for an eps that fp32 does not hold."""
import pytest
import torch

import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("width", [40, 1600, 5120, 20000])
def test_rstd_is_rounded_once(width):
    g = torch.Generator().manual_seed(width)
    x = torch.zeros(2, width, device=DEV)
    x[1] = 2.0 ** -12 * torch.randn(width, device=DEV)
    mean = x.double().square().mean(1)
    y, rstd = torch.empty_like(x), torch.empty(2, device=DEV)
    for eps in (10.0 ** (-12 + 14 * torch.rand(60, generator=g, dtype=torch.float64))).tolist() + [1e-5, 1e-6, 1e-8, 0.1]:
        zs.zero_rmsnorm_forward(x, None, None, None, y, rstd, eps=eps)
        want = 1 / torch.sqrt(mean + eps)
        assert ((rstd.double() - want).abs() <= want * (2.0 ** -24 + 2.0 ** -48)).all(), eps


@pytest.mark.parametrize("width", [40, 1600, 5120, 20000])
@pytest.mark.parametrize("eps", [1e-46, 1e-60])
def test_an_eps_below_fp32(width, eps):
    """A row of zeros has the norm 0, not 0 times infinity."""
    x = torch.zeros(3, width, dtype=torch.bfloat16, device=DEV)
    x[1] = 1.0
    y, rstd = torch.empty_like(x), torch.empty(3, device=DEV)
    codes = torch.empty(3, width, dtype=torch.uint8, device=DEV)
    exps = torch.empty(3, -(-width // 128), dtype=torch.uint8, device=DEV)
    zs.zero_rmsnorm_forward(x, None, None, None, y, rstd, codes.view(torch.float8_e4m3fn), exps, eps=eps)
    assert y[0].eq(0).all() and y[1].eq(1).all() and y[2].eq(0).all()
    assert codes[0].eq(0).all() and exps[0].eq(27).all()
    assert abs(rstd[0].item() * eps ** 0.5 - 1) <= 2.0 ** -23 and rstd[1].item() == 1
