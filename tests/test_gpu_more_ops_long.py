"""Arrays of more than 2^32 elements: the last rows of each are what the same rows alone give."""
import pytest
import torch

import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def repeated(period, rows, width, seed):
    """[rows, width] in bf16 of the same `period` rows, and those."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    few = torch.randn(period, width, generator=g, device=DEV).bfloat16()
    return few.repeat(-(-rows // period), 1)[:rows], few


def test_norm_and_packing():
    width, period = 2056, 1000
    rows = (1 << 21) + 3000
    x, few = repeated(period, rows, width, 1)
    assert x.numel() > 1 << 32
    w = torch.randn(width, device=DEV)
    blocks = -(-width // 128)

    def norm(x):
        n = x.shape[0]
        y, rstd = torch.empty_like(x), torch.empty(n, device=DEV)
        codes, exps = torch.empty(n, width, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn), torch.empty(n, blocks, dtype=torch.uint8, device=DEV)
        zs.zero_rmsnorm_forward(x, None, w, None, y, rstd, codes, exps)
        return y, rstd, codes.view(torch.uint8), exps

    got, want = norm(x), norm(few)
    for a, b in zip(got, want):
        for at in (0, period * 1044, period * 2089, period * 2099):      # (on both sides of 2^31 and of 2^32 elements)
            assert torch.equal(a[at:at + period], b)
    y, rstd, codes, exps = got
    dx, dfew = torch.empty_like(x), torch.empty_like(few)
    zs.zero_rmsnorm_backward(y, x, w, rstd, dx)
    zs.zero_rmsnorm_backward(want[0], few, w, want[1], dfew)
    assert torch.equal(dx[period * 2099:period * 2100], dfew) and torch.equal(dx[:period], dfew)
    out = dx
    zs.zero_scaled_unpack(codes.view(torch.float8_e4m3fn), exps, out)
    few_out = torch.empty_like(few)
    zs.zero_scaled_unpack(want[2].view(torch.float8_e4m3fn), want[3], few_out)
    assert torch.equal(out[period * 2099:period * 2100], few_out)
    del y, got, out, dx
    codes_t = torch.empty(width, rows, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    exps_t = torch.empty(width, -(-rows // 128), dtype=torch.uint8, device=DEV)
    zs.zero_scaled_pack(x, codes.view(torch.float8_e4m3fn), exps, codes_t, exps_t)
    # (the last 1000 columns of the transpose: rows from a multiple of 128 on, alone)
    from_row = (rows - 1000) // 128 * 128
    part = x[from_row:].contiguous()
    n = part.shape[0]
    pt, pe = torch.empty(width, n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn), torch.empty(width, -(-n // 128), dtype=torch.uint8, device=DEV)
    zs.zero_scaled_pack(part, None, None, pt, pe)
    assert torch.equal(codes_t.view(torch.uint8)[:, from_row:], pt.view(torch.uint8))
    assert torch.equal(exps_t[:, from_row // 128:], pe)


@pytest.mark.parametrize("m,n", [(66_000, 66_000), (20, 215_000_000)])
def test_product(m, n):
    k = 40
    g = torch.Generator(device=DEV).manual_seed(2)
    code = lambda rows: torch.randint(0, 0x70, (rows, k), generator=g, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn)
    a, b = code(m), code(n)
    ae = torch.full((m, 1), 126, dtype=torch.uint8, device=DEV)
    be = torch.randint(120, 130, (n, 1), generator=g, device=DEV, dtype=torch.uint8)
    out = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    assert out.numel() >= (1 << 32) - (1 << 24)
    ws = torch.empty(zs.zero_scaled_product_workspace(m, n, k, torch.bfloat16), dtype=torch.uint8, device=DEV)
    zs.zero_scaled_product(a, ae, b, be, out, None, ws)
    # the corner behind all others, by sums in 64 bits (40 positive products: no more than their rounding and the
    # alignment of 8 to the largest, 2^-10 of it at most)
    rows, columns = slice(m - 20, m), slice(n - 300, n)
    values = lambda c, e: c.float().double() * torch.exp2(e.double() - 127)
    want = values(a[rows], ae[rows]) @ values(b[columns], be[columns]).t()
    assert ((out[rows, columns].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -10 + 40 * 2.0 ** -23) * want).all()


def test_log_probabilities():
    width, period, v = 2056, 1000, 100
    rows = (1 << 21) + 3000
    h, few = repeated(period, rows, width, 3)
    w = (torch.randn(v, width, device=DEV) * width ** -0.5).bfloat16()
    ids = (torch.arange(rows, device=DEV) % period) % v

    def run(h, ids, most):
        n = h.shape[0]
        logp, lse, ent = (torch.empty(n, device=DEV) for _ in range(3))
        top_ids, top_logp = torch.empty(n, 3, dtype=torch.int64, device=DEV), torch.empty(n, 3, device=DEV)
        ws = torch.empty(zs.zero_token_logprobs_workspace(n, v, width, top=3, max_tokens=most), dtype=torch.uint8, device=DEV)
        zs.zero_token_logprobs(h, w, ids, logp, lse, ent, top_ids, top_logp, ws, max_tokens=most)
        return logp, lse, ent, top_ids, top_logp

    got, want = run(h, ids, 65535), run(few, ids[:period], 0)
    for a, b in zip(got, want):
        for at in (0, period * 1044, period * 2089, period * 2099):
            assert torch.equal(a[at:at + period], b)
