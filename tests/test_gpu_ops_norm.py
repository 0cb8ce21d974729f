"""Layer norm on the GPU against its definition in 64 bits, and its gradient
against differences of the loss.

Tolerances.  A result is rounded once: half a step, eps/2 of its type times its
size.  Before that, fp32 sums of at most 128 terms one after the other (a lane's
share, then the wave's and the waves' tree), each off by at most 2^-24 of the terms'
absolute sum, and a few roundings a product: 160 * 2^-24 times the expression with
every term's absolute value covers them (the statistics' errors enter the results
through the same absolute sums)."""
import pytest
import torch

import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
E = 160 * 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def make(rows, width, t, a, seed=0, pad=0, mean=0.3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x = torch.empty(rows, width + pad, dtype=t, device=DEV)[:, :width]
    x.copy_(r(rows, width) * torch.exp(0.5 * r(rows, 1)) + mean * r(rows, 1))
    dy = torch.empty(rows, width + 2 * pad, dtype=t, device=DEV)[:, :width]
    dy.copy_(r(rows, width))
    return x, dy, (1 + 0.3 * r(width)).to(a), (0.2 * r(width)).to(a)


def reference(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + eps)
    one = torch.ones(x.shape[1], dtype=torch.float64, device=x.device)
    w = one if w is None else w.double()
    b = 0 * one if b is None else b.double()
    y = (x - mean) * rstd * w + b
    # with absolute values: what the error is a share of
    size = (x.abs() + x.abs().mean(1, keepdim=True)) * rstd
    return y, mean[:, 0], rstd[:, 0], 2 * size * w.abs() + b.abs()


CASES = [(1, 1, "fp32", "fp32"), (3, 2, "fp16", "fp16"), (5, 63, "bf16", "fp32"), (70, 64, "bf16", "bf16"),
         (9, 511, "fp16", "fp32"), (1025, 512, "fp16", "fp16"), (33, 513, "fp32", "fp32"), (12, 1600, "bf16", "bf16"),
         (7, 2047, "bf16", "fp32"), (6, 2049, "fp16", "fp16"), (300, 4096, "bf16", "bf16"), (5, 5120, "fp32", "fp32"),
         (4, 8193, "bf16", "bf16"), (3, 16384, "fp16", "fp32"), (2, 16389, "bf16", "fp32"), (2, 40001, "fp32", "fp32")]


@pytest.mark.parametrize("rows,width,kind,affine", CASES)
def test_forward(rows, width, kind, affine):
    t, a = TYPES[kind], TYPES[affine]
    x, _, w, b = make(rows, width, t, a, seed=width)
    y = torch.full((rows, width), 7.0, dtype=t, device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    zs.zero_layernorm_forward(x, w, b, y, mean, rstd, eps=1e-5)
    ry, rm, rr, size = reference(x, w, b, 1e-5)
    assert ((y.double() - ry).abs() <= half_step(t) * ry.abs() + (E + half_step(t) * E) * size + torch.finfo(t).tiny).all()
    assert ((mean.double() - rm).abs() <= E * x.double().abs().mean(1)).all()
    assert ((rstd.double() - rr).abs() <= E * rr * (1 + (x.double().abs().mean(1) * rr))).all()


@pytest.mark.parametrize("rows,width,kind,affine", CASES)
def test_backward(rows, width, kind, affine):
    t, a = TYPES[kind], TYPES[affine]
    x, dy, w, _ = make(rows, width, t, a, seed=width + 1)
    _, m64, r64, _ = reference(x, w, None, 1e-5)
    mean, rstd = m64.float(), r64.float()
    dx, dw, db = torch.empty(rows, width, dtype=t, device=DEV), torch.empty_like(w), torch.empty_like(w)
    space = torch.empty(zs.zero_layernorm_workspace(rows, width), dtype=torch.uint8, device=DEV)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, space)
    # the gradient at the statistics that were given
    X, G, W, m, r = x.double(), dy.double(), w.double(), mean.double()[:, None], rstd.double()[:, None]
    xhat, g = (X - m) * r, G * W
    want = r * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    A = (X.abs() + m.abs()) * r
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + A * (g.abs() * A).mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= half_step(t) * want.abs() + (E + half_step(t) * E) * size + torch.finfo(t).tiny).all()
    for got, ref, abs_sum in ((dw, (G * xhat).sum(0), (G.abs() * A).sum(0)), (db, G.sum(0), G.abs().sum(0))):
        assert ((got.double() - ref).abs() <= half_step(a) * ref.abs() + E * (1 + half_step(a)) * abs_sum + torch.finfo(a).tiny).all()


def test_gradient_against_differences():
    """d/dz of sum(dy * y) by central differences in 64 bits, for x, weight and bias."""
    rows, width = 5, 37
    x, dy, w, b = make(rows, width, torch.float32, torch.float32, seed=3)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    zs.zero_layernorm_forward(x, w, b, y, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    space = torch.empty(zs.zero_layernorm_workspace(rows, width), dtype=torch.uint8, device=DEV)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, space)

    def value(x, w, b):
        mean = x.mean(1, keepdim=True)
        return (dy.double() * ((x - mean) / torch.sqrt((x - mean).square().mean(1, keepdim=True) + 1e-5) * w + b)).sum()

    at = [x.double(), w.double(), b.double()]
    h = 1e-6                      # differences are off by h^2 and 2^-52 / h: far below fp32
    for k, got in enumerate((dx, dw, db)):
        for j in range(0, got.numel(), 11):
            ends = []
            for sign in (1, -1):
                moved = [z.clone() for z in at]
                moved[k].view(-1)[j] += sign * h
                ends.append(value(*moved))
            d = ((ends[0] - ends[1]) / (2 * h)).item()
            assert abs(got.view(-1)[j].item() - d) <= 2e-5 * max(1.0, abs(d)), (k, j)


def test_strides_views_and_absent_arrays():
    x, dy, w, b = make(50, 130, torch.bfloat16, torch.bfloat16, seed=5, pad=3)       # odd row strides
    assert x.stride(0) == 133 and dy.stride(0) == 136
    buf = torch.zeros(50, 262, dtype=torch.bfloat16, device=DEV)
    y = buf[:, 1:131]                                            # columns of a wider buffer
    zs.zero_layernorm_forward(x, w, b, y)
    want = torch.empty(50, 130, dtype=torch.bfloat16, device=DEV)
    zs.zero_layernorm_forward(x.contiguous(), w, b, want)
    assert torch.equal(y, want) and not buf[:, 0].any() and not buf[:, 131:].any()
    # neither weight nor bias
    zs.zero_layernorm_forward(x, None, None, y)
    one, zero = torch.ones_like(w), torch.zeros_like(b)
    zs.zero_layernorm_forward(x, one, zero, want)
    assert torch.equal(y, want)
    # in place
    z = x.clone()
    zs.zero_layernorm_forward(z, None, None, z)
    assert torch.equal(z, want)
    mean, rstd = torch.empty(50, device=DEV), torch.empty(50, device=DEV)
    zs.zero_layernorm_forward(x, w, b, y, mean, rstd)
    full = [torch.empty(50, 130, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    space = torch.empty(zs.zero_layernorm_workspace(50, 130), dtype=torch.uint8, device=DEV)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, full[0], dw, db, space)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, buf[:, 131:261])                # dx alone
    assert torch.equal(buf[:, 131:261], full[0])
    only = torch.empty_like(b)
    zs.zero_layernorm_backward(dy, x, w, mean, rstd, full[1], None, only, space)
    assert torch.equal(only, db) and torch.equal(full[1], full[0])


def test_no_rows_and_constant_rows():
    w = torch.ones(40, device=DEV)
    x = torch.empty(0, 40, device=DEV)
    e = torch.empty(0, device=DEV)
    zs.zero_layernorm_forward(x, w, w, x.clone(), e, e.clone())
    dw, db = torch.full_like(w, 3.0), torch.full_like(w, 3.0)
    space = torch.empty(zs.zero_layernorm_workspace(0, 40), dtype=torch.uint8, device=DEV)
    zs.zero_layernorm_backward(x, x.clone(), w, e, e.clone(), x.clone(), dw, db, space)
    assert not dw.any() and not db.any()
    # rows without variance: xhat is 0, y is the bias
    x = torch.full((3, 40), 5.0, device=DEV)
    y = torch.empty_like(x)
    zs.zero_layernorm_forward(x, w, 2 * w, y)
    assert torch.equal(y, torch.full_like(y, 2.0))


def test_what_is_not_finite_stays_in_its_row():
    x, dy, w, b = make(9, 1000, torch.float32, torch.float32, seed=8)
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    zs.zero_layernorm_forward(x, w, b, y0)
    x[4, 17] = float("inf")
    x[6, 999] = float("nan")
    zs.zero_layernorm_forward(x, w, b, y1)
    rest = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y0[rest], y1[rest]) and torch.isnan(y1[6]).all() and torch.isnan(y1[4]).any()


def test_same_bits_other_streams_and_graphs():
    x, dy, w, b = make(3000, 777, torch.float16, torch.float32, seed=4)
    y, mean, rstd = torch.empty_like(x), torch.empty(3000, device=DEV), torch.empty(3000, device=DEV)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    space = torch.empty(zs.zero_layernorm_workspace(3000, 777), dtype=torch.uint8, device=DEV)

    def both(stream=None):
        zs.zero_layernorm_forward(x, w, b, y, mean, rstd, stream=stream)
        zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, space, stream=stream)

    both()
    torch.cuda.synchronize()
    first = [t.clone() for t in (y, dx, dw, db)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in (y, dx, dw, db):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, (y, dx, dw, db)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for k in range(4):
        for t in (y, dx, dw, db):
            t.zero_()
        x.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw, db)]
        both()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (y, dx, dw, db))), k


def test_refusals_on_the_gpu():
    x = torch.zeros(4, 8, device=DEV)
    host = torch.zeros(4, 8)
    with pytest.raises(zs.ZeroError, match="overlaps"):
        zs.zero_layernorm_forward(x, None, None, x, mean=x.view(-1)[:4])
    with pytest.raises(ValueError, match="last dimension"):
        zs.zero_layernorm_forward(x.t(), None, None, x.t().contiguous())
    with pytest.raises(ValueError, match="shape"):
        zs.zero_layernorm_forward(x, None, None, x[:3])
    with pytest.raises(ValueError, match="GPU"):
        zs.zero_layernorm_forward(x, None, None, host)
    with pytest.raises(zs.ZeroError, match="affine"):
        zs.zero_layernorm_forward(x.half(), x[0].bfloat16(), None, x.half())
    # a range past the end of its allocation, by address
    from zero_dp_sharded_amd import ops
    big = torch.empty(1 << 21, dtype=torch.uint8, device=DEV)
    far = 1 << 40
    s = ops.lib().zero_layernorm_forward(big.data_ptr(), 8, None, None, far // 8, 8, 3, 3, 1e-5, big.data_ptr(), 8,
                                         None, None, None)
    assert s in (zs.ZERO_ERR_INVALID_ARG, zs.ZERO_ERR_UNSUPPORTED)
    s = ops.lib().zero_layernorm_forward(big.data_ptr(), 8, None, None, 1 << 30, 8, 3, 3, 1e-5, big.data_ptr(), 8,
                                         None, None, None)
    assert s == zs.ZERO_ERR_INVALID_ARG and "past the end" in zs.zero_ops_last_error()
