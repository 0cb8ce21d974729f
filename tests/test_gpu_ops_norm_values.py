"""Layer norm at values where a step between inputs and results leaves fp32's range,
and at sizes where a workgroup walks many rows, against the definition in 64 bits."""
import pytest
import torch

import zero_dp_sharded_amd as zs
from test_gpu_ops_norm import DEV, E, TYPES, half_step

pytestmark = pytest.mark.gpu


def backward(dy, x, w, mean, rstd):
    dx, dw, db = torch.full_like(x, 7.0), torch.full_like(w, 7.0), torch.full_like(w, 7.0)
    space = torch.empty(zs.zero_layernorm_workspace(*x.shape), dtype=torch.uint8, device=DEV)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, space)
    return dx, dw, db


@pytest.mark.parametrize("width,kind", [(1, "fp32"), (63, "bf16"), (65, "fp32"), (513, "bf16"), (1600, "bf16"), (1601, "fp32"),
                                        (2049, "bf16"), (4097, "fp32"), (8200, "bf16"), (9001, "fp32"), (16389, "bf16"), (16391, "fp32")])
def test_constant_rows_of_large_values(width, kind):
    """Rows without variance: xhat is 0 and dx = rstd (g - mean(g)), however large the
    values; rstd is 1 / sqrt(eps) and rstd times the mean passes fp32's range.

    Off by a rounding to the type and, in fp32, the row's sum (at most 128 terms in a
    chain) and a few operations: E of the absolute sum, as in the norm's other tests."""
    t = TYPES[kind]
    rows = 5
    g = torch.Generator(device=DEV).manual_seed(width)
    value = torch.tensor([1e37, -3e38, 2.0, 1e30, 0.0], device=DEV).to(t)
    x = value[:, None].expand(rows, width).contiguous()
    dy = torch.randn(rows, width, generator=g, device=DEV).to(t)
    w = (1 + 0.3 * torch.randn(width, generator=g, device=DEV)).to(t)
    mean, rstd = value.float(), torch.full((rows,), 1e-5, device=DEV).rsqrt()
    dx, dw, db = backward(dy, x, w, mean, rstd)
    gw = dy.double() * w.double()
    r = rstd.double()[:, None]
    want = r * (gw - gw.mean(1, keepdim=True))
    size = r * (gw.abs() + gw.abs().mean(1, keepdim=True))
    assert torch.isfinite(dx).all()
    assert ((dx.double() - want).abs() <= half_step(t) * want.abs() + E * (1 + half_step(t)) * size + torch.finfo(t).tiny).all()
    assert not dw.any()
    assert ((db.double() - dy.double().sum(0)).abs() <= half_step(t) * dy.double().sum(0).abs() + 2 * E * dy.double().abs().sum(0)).all()
