"""The 8-bit product by tiles of 64 rows, more of them than stand in the CUs at once: each workgroup walks several.
Tolerances are those of the product's tests."""
import pytest
import torch

import ops_scaled_common as sc
import zero_dp_sharded_amd as zs
from test_gpu_ops_product import check, packed, space

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIZES = [(40, 102400, 300), (33, 102400, 1025), (64, 25600, 20480), (192, 102400, 128), (300, 25600, 513)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
def test_against_the_definition(m, n, k, square, kind):
    a, ae = packed(m, k, False, 3, -k % 4)
    b, be = packed(n, k, square, 4, -k % 4)
    bias = torch.randn(n, device=DEV).to(kind)
    out = torch.full((m, n), float("nan"), dtype=kind, device=DEV)
    zs.zero_scaled_product(a, ae, b, be, out, bias, space(m, n, k))
    A = sc.values(a, ae, False)
    for c in range(0, n, 12800):
        p = slice(c, c + 12800)
        B = sc.values(b[p], be[c // 128:c // 128 + 100] if square else be[p], square)
        size = A.abs() @ B.abs().t() + bias[p].double().abs()
        check(out[:, p], A @ B.t() + bias[p].double(), size * ((k + 2) * 2.0 ** -23 + 2.0 ** -10))
