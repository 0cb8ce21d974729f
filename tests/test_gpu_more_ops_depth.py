"""The scaled product at the largest depth and at row strides beyond what the tiles load: numbers of -1, 0 and 1 with
scales of 1 and 2, whose sums fp32 holds exactly in any order, and results that are equal to the definition's."""
import pytest
import torch

import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ONE = torch.tensor([0xb8, 0x00, 0x38], dtype=torch.uint8)          # -1, 0, 1 in e4m3


def make(rows, k, square, seed, stride=None):
    """Codes, exponents and the values that they stand for, in int8."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randint(0, 3, (rows, k), generator=g, device=DEV, dtype=torch.uint8)
    codes = torch.full((rows, stride or k), 0x7f, dtype=torch.uint8, device=DEV)[:, :k]
    for r in range(0, rows, 64):
        codes[r:r + 64] = ONE.to(DEV)[x[r:r + 64].int()]
    blocks, down = -(-k // 128), -(-rows // 128) if square else rows
    exps = torch.full((down, blocks), 127, dtype=torch.uint8, device=DEV)
    exps[:, 1::7] = 128
    return codes.view(torch.float8_e4m3fn), exps, x


def product(a, ae, x, b, be, y, kind, square):
    m, n, k = x.shape[0], y.shape[0], x.shape[1]
    out = torch.full((m, n), float("nan"), dtype=TYPES[kind], device=DEV)
    zs.zero_scaled_product(a, ae, b, be, out, None, torch.empty(zs.zero_scaled_product_workspace(m, n, k), dtype=torch.uint8, device=DEV))
    want = torch.zeros(m, n, dtype=torch.float64, device=DEV)
    for c in range(0, k, 1 << 16):
        at, end = slice(c, c + (1 << 16)), min(k, c + (1 << 16))
        two = 1.0 + ((torch.arange(c, end, device=DEV) // 128) % 7 == 1).double()
        want += ((x[:, at].double() - 1) * two) @ ((y[:, at].double() - 1) * two).t()
    assert want.abs().max() < 1 << 24 and want.any()
    assert torch.equal(out, want.to(TYPES[kind]))


@pytest.mark.parametrize("m,n", [(4, 40), (40, 1100), (260, 300)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("k", [1 << 22, (1 << 22) - 5])
def test_the_largest_depth(m, n, kind, square, k):
    print(m, n, kind, square, k, flush=True)
    a, b = make(m, k, False, 1), make(n, k, square, 2)
    product(*a, *b, kind, square)


@pytest.mark.parametrize("m,n", [(20, 70), (40, 300)])
@pytest.mark.parametrize("kind", ["fp16", "fp32"])
@pytest.mark.parametrize("stride", [1 << 22, (1 << 22) + 4])
def test_rows_far_apart(m, n, kind, stride):
    a, b = make(m, 1000, False, 3, stride), make(n, 1000, True, 4, stride)
    product(*a, *b, kind, True)
