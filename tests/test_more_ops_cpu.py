"""The boundary of the RMS norm, of packing and of the 8-bit product, checked without a GPU:
struct layouts, workspace sizes, and the refusals that come before any device work (the
arrays are made-up addresses: nothing is launched)."""
import ctypes

import pytest

import zero_dp_sharded_amd as zs
from test_ops_cpu import at, error
from zero_dp_sharded_amd import ops


def test_struct_layouts_match_header():
    assert ctypes.sizeof(ops.ZeroRmsnormDesc) == 80
    assert ctypes.sizeof(ops.ZeroRmsnormGradDesc) == 56


# ------------------------------------------------------------------ RMS norm

def forward(x=at(0), residual=at(1), w=at(2), h=at(3), y=at(4), rstd=at(5), codes=at(6), exps=at(7), desc=True, **d):
    f = dict(rows=4, width=200, type=2, affine=2, eps=1e-6, x_stride=200, residual_stride=200, h_stride=200, y_stride=200,
             codes_stride=200, exps_stride=2)
    f.update(d)
    c = ops.ZeroRmsnormDesc(**f)
    return error(ops.lib().zero_rmsnorm_forward, ctypes.byref(c) if desc else None, x, residual, w, h, y, rstd, codes, exps, None)


@pytest.mark.parametrize("kw,word", [
    (dict(desc=False), "NULL"), (dict(x=None), "NULL"), (dict(residual=None), "both or neither"), (dict(h=None), "both or neither"),
    (dict(codes=None), "both or neither"), (dict(exps=None), "both or neither"), (dict(y=None, codes=None, exps=None), "both NULL"),
    (dict(rows=-1), "rows"), (dict(width=0), "width"), (dict(type=0), "unknown type"), (dict(type=4), "unknown type"), (dict(affine=1), "affine"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=1e300), "eps"),
    (dict(x_stride=199), "stride"), (dict(residual_stride=199), "stride"), (dict(h_stride=0), "stride"), (dict(y_stride=199), "stride"),
    (dict(codes_stride=199), "stride"), (dict(exps_stride=1), "stride"), (dict(x_stride=1 << 62), "stride"),
    (dict(x=at(0, 1)), "aligned"), (dict(residual=at(1, 1)), "aligned"), (dict(rstd=at(5, 2)), "aligned"), (dict(w=at(2, 1)), "aligned"),
    (dict(h=at(0, 2)), "overlaps"), (dict(y=at(1)), "overlaps"), (dict(y=at(3)), "overlaps"), (dict(codes=at(4)), "overlaps"),
    (dict(exps=at(6, 5)), "overlaps"), (dict(h=at(1), h_stride=300), "overlaps"), (dict(codes=at(0)), "overlaps"),
])
def test_rmsnorm_forward_refuses(kw, word):
    s, msg = forward(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


def test_rmsnorm_what_may_be_the_same_array():
    for kw in (dict(h=at(0)), dict(h=at(1)), dict(y=at(0))):
        assert "overlaps" not in forward(**kw)[1]
    assert "overlaps" not in backward(dh=at(3), dx=at(3))[1]


def test_rmsnorm_unsupported_and_empty():
    wide = (1 << 24) + 1
    assert forward(width=wide)[0] == zs.ZERO_ERR_UNSUPPORTED
    assert forward(rows=1 << 31)[0] == zs.ZERO_ERR_UNSUPPORTED
    assert forward(rows=0, x=None, residual=None)[0] == zs.ZERO_OK
    assert backward(rows=0, dy=None, h=None, dh=None, dx=None, rstd=None, dw=None)[0] == zs.ZERO_OK


def backward(dy=at(0), h=at(1), w=at(2), rstd=at(3, 1 << 20), dh=at(4), dx=at(5), dw=at(6), ws=at(7), wn=1 << 20, desc=True, **d):
    f = dict(rows=4, width=200, type=2, affine=2, dy_stride=200, h_stride=200, dh_stride=200, dx_stride=200)
    f.update(d)
    c = ops.ZeroRmsnormGradDesc(**f)
    return error(ops.lib().zero_rmsnorm_backward, ctypes.byref(c) if desc else None, dy, h, w, rstd, dh, dx, dw, ws, wn, None)


@pytest.mark.parametrize("kw,word", [
    (dict(desc=False), "NULL"), (dict(dy=None), "NULL"), (dict(h=None), "NULL"), (dict(rstd=None), "NULL"), (dict(dx=None), "NULL"),
    (dict(ws=None), "workspace"), (dict(wn=4 * 200 * 4 - 1), "workspace"), (dict(dy_stride=1), "stride"), (dict(h_stride=1), "stride"),
    (dict(dh_stride=1), "stride"), (dict(dx_stride=199), "stride"), (dict(dx=at(0)), "overlaps"), (dict(dx=at(1)), "overlaps"),
    (dict(dx=at(4, 2)), "overlaps"), (dict(dw=at(2)), "overlaps"), (dict(ws=at(5)), "overlaps"), (dict(ws=at(7, 4)), "aligned"),
    (dict(dx=at(5, 1)), "aligned"), (dict(rows=-2), "rows"), (dict(width=0), "width"), (dict(affine=1), "affine"), (dict(type=9), "unknown type"),
])
def test_rmsnorm_backward_refuses(kw, word):
    s, msg = backward(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


def test_rmsnorm_workspace():
    assert zs.zero_rmsnorm_workspace(1, 10) == 40
    assert zs.zero_rmsnorm_workspace(1 << 20, 5120) == zs.zero_rmsnorm_workspace(1 << 30, 5120)
    for bad in ((-1, 5), (5, 0)):
        with pytest.raises(zs.ZeroError):
            zs.zero_rmsnorm_workspace(*bad)


# ------------------------------------------------------------------ packing

def pack(x=at(0), xs=300, rows=200, width=300, t=2, square=0, c=at(1), cs=300, e=at(2), es=3, ct=at(3), cts=200, et=at(4), ets=2):
    return error(ops.lib().zero_scaled_pack, x, xs, rows, width, t, square, c, cs, e, es, ct, cts, et, ets, None)


def unpack(c=at(1), cs=300, e=at(2), es=3, rows=200, width=300, square=0, t=3, out=at(0), os=300):
    return error(ops.lib().zero_scaled_unpack, c, cs, e, es, rows, width, square, t, out, os, None)


@pytest.mark.parametrize("kw,word", [
    (dict(x=None), "NULL"), (dict(c=None), "both or neither"), (dict(e=None), "both or neither"), (dict(ct=None), "both or neither"),
    (dict(et=None), "both or neither"), (dict(c=None, e=None, ct=None, et=None), "both NULL"), (dict(t=0), "unknown type"),
    (dict(square=2), "square"), (dict(square=-1), "square"), (dict(rows=-1), "rows"), (dict(width=-1), "width"), (dict(xs=299), "stride"),
    (dict(cs=299), "stride"), (dict(es=2), "stride"), (dict(cts=199), "stride"), (dict(ets=1), "stride"), (dict(x=at(0, 1)), "aligned"),
    (dict(c=at(0)), "overlaps"), (dict(ct=at(1)), "overlaps"), (dict(e=at(1, 7)), "overlaps"), (dict(et=at(2, 599)), "overlaps"),
])
def test_pack_refuses(kw, word):
    s, msg = pack(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


@pytest.mark.parametrize("kw,word", [
    (dict(c=None), "NULL"), (dict(e=None), "NULL"), (dict(out=None), "NULL"), (dict(t=5), "unknown type"), (dict(square=3), "square"),
    (dict(cs=1), "stride"), (dict(es=1), "stride"), (dict(os=299), "stride"), (dict(out=at(0, 2)), "aligned"), (dict(out=at(1)), "overlaps"),
])
def test_unpack_refuses(kw, word):
    s, msg = unpack(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


def test_scaled_unsupported_and_empty():
    for call in (pack, unpack):
        assert call(rows=1 << 31)[0] == zs.ZERO_ERR_UNSUPPORTED
        assert call(width=1 << 31)[0] == zs.ZERO_ERR_UNSUPPORTED
        assert call(rows=1 << 30, width=1 << 17)[0] == zs.ZERO_ERR_UNSUPPORTED
        assert call(rows=0)[0] == zs.ZERO_OK and call(width=0)[0] == zs.ZERO_OK
    # the exponents of squares are fewer
    assert "overlaps" not in pack(square=1, et=at(2, 599))[1]


# ------------------------------------------------------------------ the product

def product(a=at(0), ae=at(1), b=at(2), be=at(3), bias=at(4), out=at(5), ws=at(6), wn=1 << 29, desc=True, **d):
    f = dict(m=100, n=200, k=300, type=3, b_square=0, a_stride=300, a_exps_stride=3, b_stride=300, b_exps_stride=3, out_stride=200)
    f.update(d)
    c = ops.ZeroScaledProductDesc(**f)
    return error(ops.lib().zero_scaled_product, ctypes.byref(c) if desc else None, a, ae, b, be, bias, out, ws, wn, None)


@pytest.mark.parametrize("kw,word", [
    (dict(desc=False), "NULL"), (dict(a=None), "NULL"), (dict(ae=None), "NULL"), (dict(b=None), "NULL"), (dict(be=None), "NULL"),
    (dict(out=None), "NULL"), (dict(type=0), "unknown type"), (dict(b_square=2), "b_square"), (dict(m=-1), "m, n and k"),
    (dict(n=-1), "m, n and k"), (dict(k=-1), "m, n and k"), (dict(a_stride=299), "stride"), (dict(b_stride=1), "stride"),
    (dict(a_exps_stride=2), "stride"), (dict(b_exps_stride=2), "stride"), (dict(out_stride=199), "stride"), (dict(ws=None), "workspace"),
    (dict(wn=100), "workspace"), (dict(ws=at(6, 128)), "aligned"), (dict(out=at(5, 2)), "aligned"), (dict(bias=at(4, 1)), "aligned"),
    (dict(out=at(0)), "overlaps"), (dict(out=at(3)), "overlaps"), (dict(ws=at(2)), "overlaps"), (dict(out=at(4)), "overlaps"),
])
def test_product_refuses(kw, word):
    s, msg = product(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


def test_product_unsupported_and_empty():
    assert ctypes.sizeof(ops.ZeroScaledProductDesc) == 72
    for kw in (dict(m=1 << 31), dict(n=1 << 31), dict(m=1 << 25, n=1 << 20), dict(k=(1 << 22) + 1), dict(a_exps_stride=(1 << 22) + 1)):
        assert product(**kw)[0] == zs.ZERO_ERR_UNSUPPORTED, kw
    assert product(m=0, a=None, out=None)[0] == zs.ZERO_OK and product(n=0, b=None, out=None)[0] == zs.ZERO_OK
    # operands may be one array
    assert "overlaps" not in product(b=at(0), be=at(1))[1]
    for bad in ((-1, 1, 1), (1 << 31, 1, 1), (1, 1, (1 << 22) + 1)):
        with pytest.raises(zs.ZeroError):
            zs.zero_scaled_product_workspace(*bad)
    assert zs.zero_scaled_product_workspace(1, 6400, 1600) == 256
    import torch
    sizes = [zs.zero_scaled_product_workspace(500, 700, 900, t) for t in (torch.float16, torch.bfloat16, torch.float32)]
    assert sizes[0] == sizes[1] and zs.zero_scaled_product_workspace(500, 700, 900) == max(sizes)
    with pytest.raises(TypeError):
        zs.zero_scaled_product_workspace(1, 1, 1, torch.int8)
