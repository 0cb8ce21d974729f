"""Codes of the RMS norm are rounded once, from 64 bits, and rstd; y is rounded to fp32, and that to its type: bit
for bit the definition's.

The definition's own sums in 64 bits are off by a few 2^-53: one of 2^40 results lies so near a middle that
this would show."""
import pytest
import torch

import ops_scaled_common as sc
import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.mark.parametrize("rows,width,kind,affine", [(8192, 5120, "bf16", "fp32"), (8192, 1600, "bf16", "bf16"), (4099, 1601, "fp16", "fp16"),
                                                    (4099, 515, "fp32", "fp32"), (2000, 8200, "fp16", "fp32"), (300, 20001, "bf16", "fp32"),
                                                    (300, 20001, "fp32", "fp32")])
@pytest.mark.parametrize("weighted", [True, False])
def test_bit_for_bit(rows, width, kind, affine, weighted):
    g = torch.Generator(device=DEV).manual_seed(rows + width)
    t = TYPES[kind]
    h = (torch.randn(rows, width, generator=g, device=DEV) * torch.exp(torch.randn(rows, 1, generator=g, device=DEV))).to(t)
    h[5] = 0
    w = (1 + 0.3 * torch.randn(width, generator=g, device=DEV)).to(TYPES[affine]) if weighted else None
    y, rstd = torch.empty_like(h), torch.empty(rows, device=DEV)
    codes = torch.empty(rows, width, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    exps = torch.empty(rows, -(-width // 128), dtype=torch.uint8, device=DEV)
    zs.zero_rmsnorm_forward(h, None, w, None, y, rstd, codes, exps, eps=1e-6)
    for r in range(0, rows, 2048):
        p = slice(r, r + 2048)
        x = h[p].double()
        rs = 1 / torch.sqrt(x.square().sum(1, keepdim=True) / width + 1e-6)
        want = x * (rs * w.double() if weighted else rs)
        assert torch.equal(rstd[p], rs[:, 0].float())
        assert torch.equal(y[p], want.float().to(t))
        _, big = sc.blocks_of(want, False)
        E = sc.scale_byte(big)
        assert torch.equal(exps[p].long(), E)
        assert torch.equal(codes[p].view(torch.uint8).long(), sc.codes(want / torch.exp2(sc.spread(E.double(), *want.shape, False) - 127)))
