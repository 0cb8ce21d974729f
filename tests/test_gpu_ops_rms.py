"""RMS norm with the residual's addition on the GPU against its definition in 64 bits, and
its gradient against differences.

Tolerances.  A result is rounded once: half a step, eps/2 of its type times its size.
Before that, fp32 sums of at most 128 terms one after the other, each off by at most 2^-24
of the terms' absolute sum, and a few roundings a product: 160 * 2^-24 of the expression
with every term's absolute value.  A result in 8 bits is off by half a step of e4m3, 2^-4
of itself or (below its normal range) 2^-10 of the scale, whichever is larger."""
import pytest
import torch

import ops_scaled_common as sc
import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
E = 160 * 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def make(rows, width, t, a, seed=0, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    out = []
    for k in range(4):
        x = torch.empty(rows, width + pad * (k + 1), dtype=t, device=DEV)[:, :width]
        x.copy_(r(rows, width) * torch.exp(0.5 * r(rows, 1)))
        out.append(x)
    return out + [(1 + 0.3 * r(width)).to(a)]


def room(rows, width, pad=0):
    codes = torch.full((rows, width + pad), 0x55, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)[:, :width]
    exps = torch.full((rows, -(-width // 128) + pad), 0x55, dtype=torch.uint8, device=DEV)[:, :-(-width // 128)]
    return codes, exps


def reference(h, w, eps):
    h = h.double()
    rstd = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return h * rstd * (1.0 if w is None else w.double()), rstd[:, 0]


def check_codes(codes, exps, y):
    size = y.abs()
    _, big = sc.blocks_of(y, False)
    low, high = sc.scale_byte(big * (1 - 2 * E)), sc.scale_byte(big * (1 + 2 * E))
    assert ((exps.long() >= low) & (exps.long() <= high)).all()
    got = sc.values(codes, exps, False)
    scale = sc.spread(torch.exp2(exps.double() - 127), *y.shape, False)
    step = torch.maximum(size * 2.0 ** -4, scale * 2.0 ** -10)
    assert ((got - y).abs() <= step * (1 + 2.0 ** -20) + 2 * E * size).all()


CASES = [(1, 1, "fp32", "fp32"), (3, 2, "fp16", "fp16"), (5, 63, "bf16", "fp32"), (70, 64, "bf16", "bf16"), (2, 127, "fp32", "fp32"),
         (9, 129, "fp16", "fp32"), (1025, 512, "fp16", "fp16"), (33, 513, "fp32", "fp32"), (12, 1600, "bf16", "bf16"),
         (7, 2047, "bf16", "fp32"), (6, 2049, "fp16", "fp16"), (300, 4096, "bf16", "bf16"), (5, 5120, "fp32", "fp32"),
         (4, 8193, "bf16", "bf16"), (3, 16384, "fp16", "fp32"), (2, 16389, "bf16", "fp32"), (2, 40001, "fp32", "fp32")]


@pytest.mark.parametrize("rows,width,kind,affine", CASES)
def test_forward(rows, width, kind, affine):
    t = TYPES[kind]
    x, residual, _, _, w = make(rows, width, t, TYPES[affine], seed=width, pad=3)
    h, y, rstd = torch.full_like(x, 7.0), torch.full((rows, width), 7.0, dtype=t, device=DEV), torch.empty(rows, device=DEV)
    codes, exps = room(rows, width, 5)
    zs.zero_rmsnorm_forward(x, residual, w, h, y, rstd, codes, exps, eps=1e-6)
    total = x.double() + residual.double()
    # (the sum is rounded to fp32, then to the type)
    assert ((h.double() - total).abs() <= (half_step(t) + 2.0 ** -24) * total.abs() + torch.finfo(t).tiny).all()
    want, rr = reference(h, w, 1e-6)
    assert ((rstd.double() - rr).abs() <= E * rr).all()
    assert ((y.double() - want).abs() <= (half_step(t) + E * (1 + half_step(t))) * want.abs() + torch.finfo(t).tiny).all()
    check_codes(codes, exps, want)
    # each output alone has the same bits
    only, c2, e2 = torch.empty_like(y), *room(rows, width)
    zs.zero_rmsnorm_forward(x, residual, w, h.clone(), only)
    zs.zero_rmsnorm_forward(x, residual, w, h.clone(), None, None, c2, e2)
    assert torch.equal(only, y) and torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(e2, exps)
    # without a residual: the norm of h itself
    zs.zero_rmsnorm_forward(h, None, w, None, only)
    assert torch.equal(only, y)


@pytest.mark.parametrize("rows,width,kind,affine", CASES)
def test_backward(rows, width, kind, affine):
    t, a = TYPES[kind], TYPES[affine]
    h, dy, dh, _, w = make(rows, width, t, a, seed=width + 1, pad=1)
    rstd = reference(h, None, 1e-6)[1].float()
    dx, dw = torch.empty(rows, width, dtype=t, device=DEV), torch.empty_like(w)
    space = torch.empty(zs.zero_rmsnorm_workspace(rows, width), dtype=torch.uint8, device=DEV)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dh, dw, space)
    H, G, W, r, D = h.double(), dy.double(), w.double(), rstd.double()[:, None], dh.double()
    xhat, g = H * r, G * W
    want = r * (g - xhat * (g * xhat).mean(1, keepdim=True)) + D
    size = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True)) + D.abs()
    low = torch.finfo(t).tiny
    assert ((dx.double() - want).abs() <= half_step(t) * want.abs() + E * (1 + half_step(t)) * size + low).all()
    ref, abs_sum = (G * xhat).sum(0), (G * xhat).abs().sum(0)
    assert ((dw.double() - ref).abs() <= half_step(a) * ref.abs() + E * (1 + half_step(a)) * abs_sum + torch.finfo(a).tiny).all()
    # in place of dh, and without dh and dw
    again = dh.clone()
    zs.zero_rmsnorm_backward(dy, h, w, rstd, again, again)
    assert torch.equal(again, dx)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, again)
    zero = torch.empty_like(dx)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, zero, torch.zeros_like(dh))
    assert torch.equal(again, zero)


def test_gradient_against_differences():
    """d/dz of sum(dy * y) + sum(dh * h) by central differences in 64 bits, for x and weight."""
    rows, width = 5, 37
    x, residual, dy, dh, w = make(rows, width, torch.float32, torch.float32, seed=3)
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=DEV)
    zs.zero_rmsnorm_forward(x, residual, w, h, y, rstd)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    space = torch.empty(zs.zero_rmsnorm_workspace(rows, width), dtype=torch.uint8, device=DEV)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dh, dw, space)

    def value(x, w):
        h = x + residual.double()
        return (dy.double() * h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * w).sum() + (dh.double() * h).sum()

    at, step = [x.double(), w.double()], 1e-6
    for k, got in enumerate((dx, dw)):
        for j in range(0, got.numel(), 7):
            ends = []
            for sign in (1, -1):
                moved = [z.clone() for z in at]
                moved[k].view(-1)[j] += sign * step
                ends.append(value(*moved))
            d = ((ends[0] - ends[1]) / (2 * step)).item()
            assert abs(got.view(-1)[j].item() - d) <= 2e-5 * max(1.0, abs(d)), (k, j)


def test_in_place_and_around():
    x, residual, _, _, w = make(50, 130, torch.bfloat16, torch.bfloat16, seed=5, pad=3)
    want_h, want = torch.empty_like(x), torch.empty(50, 130, dtype=torch.bfloat16, device=DEV)
    zs.zero_rmsnorm_forward(x, residual, w, want_h, want)
    buf = torch.zeros(50, 262, dtype=torch.bfloat16, device=DEV)
    r2 = residual.clone()
    zs.zero_rmsnorm_forward(x, r2, w, r2, buf[:, 1:131])         # the residual becomes the sum
    assert torch.equal(r2, want_h) and torch.equal(buf[:, 1:131], want) and not buf[:, 0].any() and not buf[:, 131:].any()
    x2, x3 = x.clone(), x.clone()
    zs.zero_rmsnorm_forward(x2, residual, w, x2, want)           # x becomes the sum
    assert torch.equal(x2, want_h)
    zs.zero_rmsnorm_forward(x3, None, None, None, x3)            # the norm in place of x
    zs.zero_rmsnorm_forward(x, None, torch.ones_like(w), None, want)
    assert torch.equal(x3, want)
    # codes within wider arrays: nothing else is written
    wide_c, wide_e = torch.full((50, 200), 7, dtype=torch.uint8, device=DEV), torch.full((50, 5), 7, dtype=torch.uint8, device=DEV)
    zs.zero_rmsnorm_forward(x, None, w, None, None, None, wide_c.view(torch.float8_e4m3fn)[:, 3:133], wide_e[:, 1:3])
    assert (wide_c[:, :3] == 7).all() and (wide_c[:, 133:] == 7).all() and (wide_e[:, 0] == 7).all() and (wide_e[:, 3:] == 7).all()
    y, _ = reference(x, w, 1e-6)
    check_codes(wide_c.view(torch.float8_e4m3fn)[:, 3:133], wide_e[:, 1:3], y)


def test_no_rows_zeros_and_what_is_not_finite():
    w = torch.ones(40, device=DEV)
    x, e = torch.empty(0, 40, device=DEV), torch.empty(0, device=DEV)
    zs.zero_rmsnorm_forward(x, None, w, None, x.clone(), e)
    dw = torch.full_like(w, 3.0)
    space = torch.empty(zs.zero_rmsnorm_workspace(0, 40), dtype=torch.uint8, device=DEV)
    zs.zero_rmsnorm_backward(x, x.clone(), w, e, x.clone(), None, dw, space)
    assert not dw.any()
    x = torch.randn(9, 1000, device=DEV)
    x[2] = 0
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    c0, e0 = room(9, 1000)
    c1, e1 = room(9, 1000)
    w = torch.ones(1000, device=DEV)
    zs.zero_rmsnorm_forward(x, None, w, None, y0, None, c0, e0)
    assert not y0[2].any() and not c0.view(torch.uint8)[2].any() and (e0[2] == 27).all()
    x[4, 17] = float("inf")
    x[6, 999] = float("nan")
    zs.zero_rmsnorm_forward(x, None, w, None, y1, None, c1, e1)
    rest = [0, 1, 2, 3, 5, 7, 8]
    same = lambda a, b: torch.equal(a.view(torch.uint8)[rest], b.view(torch.uint8)[rest])
    assert torch.equal(y0[rest], y1[rest]) and same(c0, c1) and same(e0, e1)
    assert torch.isnan(y1[6]).all() and torch.isnan(y1[4, 17])
    assert (c1.view(torch.uint8)[6] & 127 == 127).all() and c1.view(torch.uint8)[4, 17] & 127 == 127


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("width", [40, 1601, 5000, 20000])
def test_values_whose_squares_pass_fp32(kind, width):
    t = TYPES[kind]
    x, _, dy, dh, w = make(4, width, t, torch.float32, seed=9)
    x[0] *= 2.0 ** 70
    x[1] *= 2.0 ** 120
    x[2] *= 2.0 ** -60           # (eps rules)
    y, rstd = torch.empty_like(x), torch.empty(4, device=DEV)
    zs.zero_rmsnorm_forward(x, None, w, None, y, rstd)
    want, rr = reference(x, w, 1e-6)
    assert ((rstd.double() - rr).abs() <= E * rr).all()
    assert ((y.double() - want).abs() <= (half_step(t) + 2 * E) * want.abs() + torch.finfo(t).tiny).all()
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    space = torch.empty(zs.zero_rmsnorm_workspace(4, width), dtype=torch.uint8, device=DEV)
    zs.zero_rmsnorm_backward(dy, x, w, rstd, dx, dh, dw, space)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_same_bits_other_streams_and_graphs():
    x, residual, dy, dh, w = make(3000, 777, torch.float16, torch.float32, seed=4)
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(3000, device=DEV)
    codes, exps = room(3000, 777)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    space = torch.empty(zs.zero_rmsnorm_workspace(3000, 777), dtype=torch.uint8, device=DEV)
    outs = (h, y, rstd, codes.view(torch.uint8), exps, dx, dw)

    def both(stream=None):
        zs.zero_rmsnorm_forward(x, residual, w, h, y, rstd, codes, exps, stream=stream)
        zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dh, dw, space, stream=stream)

    both()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    s = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, outs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for k in range(4):
        for t in outs:
            t.zero_()
        x.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        both()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, outs)), k


@pytest.mark.parametrize("rows,width,kind", [(16384, 1600, "bf16"), (4099, 5121, "fp16"), (700, 30000, "fp32")])
def test_many_rows(rows, width, kind):
    """Rows that a workgroup walks, and results past the caches."""
    t = TYPES[kind]
    h, dy, dh, x, w = make(rows, width, t, torch.float32, seed=rows)
    y, s, rstd = torch.empty_like(h), torch.empty_like(h), torch.empty(rows, device=DEV)
    zs.zero_rmsnorm_forward(x, dh, w, s, y, rstd)
    want, _ = reference(s, w, 1e-6)
    assert ((y.double() - want).abs() <= (half_step(t) + 2 * E) * want.abs() + torch.finfo(t).tiny).all()
    del want
    dx, dw = torch.empty_like(h), torch.empty_like(w)
    space = torch.empty(zs.zero_rmsnorm_workspace(rows, width), dtype=torch.uint8, device=DEV)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dh, dw, space)
    r, W = rstd.double()[:, None], w.double()
    ref, abs_sum = torch.zeros(width, dtype=torch.float64, device=DEV), torch.zeros(width, dtype=torch.float64, device=DEV)
    for a in range(0, rows, 2048):
        p = slice(a, a + 2048)
        xhat, g = h[p].double() * r[p], dy[p].double() * W
        z = r[p] * (g - xhat * (g * xhat).mean(1, keepdim=True)) + dh[p].double()
        size = r[p] * (g.abs() + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True)) + dh[p].double().abs()
        assert ((dx[p].double() - z).abs() <= half_step(t) * z.abs() + 2 * E * size + torch.finfo(t).tiny).all()
        ref += (dy[p].double() * xhat).sum(0)
        abs_sum += (dy[p].double() * xhat).abs().sum(0)
    assert ((dw.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 2 * E * abs_sum).all()
