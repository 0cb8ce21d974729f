"""Layer norm over many rows, against its definition in 64 bits: every form of the
backward kernel with several rows for a wave or workgroup and a rest (the row that is read
ahead, the sums that go from row to row), the slabs of very long rows, and results of
more than the caches' 32 MiB, which are written past them.

Tolerances as in test_gpu_ops_norm.py.  The columns' sums here have chains of at most 13
rows a wave, 16 waves, and 32 partials in two steps: below the 128 that E covers."""
import pytest
import torch

import zero_dp_sharded_amd as zs
from test_gpu_ops_norm import DEV, E, TYPES, half_step, make, reference

pytestmark = pytest.mark.gpu

# rows and widths by the backward kernel's forms: (waves a row, workgroups) with 2-byte rows
# and with fp32 ones
CASES = [(10007, 500, "fp16", "fp16"), (12301, 509, "bf16", "fp32"), (9001, 300, "fp32", "fp32"),       # 1, 16 rows x 256
         (5003, 1000, "bf16", "bf16"), (6001, 777, "fp32", "fp32"),                                    # 1, 8 rows x 256
         (4999, 1601, "fp16", "fp16"), (1301, 1601, "fp32", "fp32"),                                   # 1, 8 x 256; 4, 512
         (1201, 4000, "bf16", "fp32"), (1100, 3001, "fp32", "fp32"),                                   # 4, 512
         (1100, 8001, "bf16", "bf16"), (1030, 5121, "fp32", "fp32"),                                   # 4, 512
         (700, 16001, "fp16", "fp16"), (600, 9000, "fp32", "fp32"),                                    # 8, 256
         (201, 16401, "bf16", "bf16"), (129, 17003, "fp32", "fp32"),                                   # long rows, slabs
         # results of more than 32 MiB
         (40003, 450, "bf16", "bf16"), (20011, 900, "fp16", "fp32"), (16411, 1100, "bf16", "bf16"), (8195, 2100, "fp32", "fp32"),
         (4111, 4100, "bf16", "fp32"), (2203, 7999, "fp16", "fp16"), (1103, 16000, "bf16", "bf16"), (1031, 16500, "fp16", "fp16"),
         (530, 16500, "fp32", "fp32")]


@pytest.mark.parametrize("rows,width,kind,affine", CASES)
def test_both_ways(rows, width, kind, affine):
    t, a = TYPES[kind], TYPES[affine]
    x, dy, w, b = make(rows, width, t, a, seed=rows + width)
    y = torch.full((rows, width), 7.0, dtype=t, device=DEV)
    mean, rstd = (torch.full((rows,), float("nan"), device=DEV) for _ in range(2))
    zs.zero_layernorm_forward(x, w, b, y, mean, rstd, eps=1e-5)
    ry, rm, rr, size = reference(x, w, b, 1e-5)
    assert ((y.double() - ry).abs() <= half_step(t) * ry.abs() + (E + half_step(t) * E) * size + torch.finfo(t).tiny).all()
    assert ((mean.double() - rm).abs() <= E * x.double().abs().mean(1)).all()
    assert ((rstd.double() - rr).abs() <= E * rr * (1 + (x.double().abs().mean(1) * rr))).all()
    del ry, size

    dx, dw, db = torch.full((rows, width), 7.0, dtype=t, device=DEV), torch.full_like(w, 7.0), torch.full_like(w, 7.0)
    space = torch.full((zs.zero_layernorm_workspace(rows, width),), 255, dtype=torch.uint8, device=DEV)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, space)
    X, G, W, m, r = x.double(), dy.double(), w.double(), mean.double()[:, None], rstd.double()[:, None]
    xhat, g = (X - m) * r, G * W
    want = r * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    A = (X.abs() + m.abs()) * r
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + A * (g.abs() * A).mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= half_step(t) * want.abs() + (E + half_step(t) * E) * size + torch.finfo(t).tiny).all()
    for got, ref, abs_sum in ((dw, (G * xhat).sum(0), (G.abs() * A).sum(0)), (db, G.sum(0), G.abs().sum(0))):
        assert ((got.double() - ref).abs() <= half_step(a) * ref.abs() + E * (1 + half_step(a)) * abs_sum + torch.finfo(a).tiny).all()


def test_rows_apart_in_both_directions():
    """Strided rows, several to a workgroup, past the caches: what lies between stays."""
    rows, width = 9001, 2000
    x, dy, w, b = make(rows, width, torch.bfloat16, torch.bfloat16, seed=1, pad=5)
    wide = torch.full((rows, 2 * width + 7), 3.0, dtype=torch.bfloat16, device=DEV)
    y, dx = wide[:, 1:width + 1], wide[:, width + 4:2 * width + 4]
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    zs.zero_layernorm_forward(x, w, b, y, mean, rstd)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx)
    y1, dx1 = (torch.empty(rows, width, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    zs.zero_layernorm_forward(x.contiguous(), w, b, y1)
    zs.zero_layernorm_backward(dy.contiguous(), x.contiguous(), w, mean, rstd, dx1)
    assert torch.equal(y, y1) and torch.equal(dx, dx1)
    assert (wide[:, 0] == 3).all() and (wide[:, width + 1:width + 4] == 3).all() and (wide[:, 2 * width + 4:] == 3).all()
