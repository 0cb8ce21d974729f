"""The training operators' boundary, checked without a GPU: exported symbols,
struct layouts, workspace sizes, and the refusals that come before any device
work (the arrays are made-up addresses: nothing is launched)."""
import ctypes
import os
import re

import pytest
import torch

import zero_dp_sharded_amd as zs
from conftest import ROOT
from zero_dp_sharded_amd import build, ops

HEADER = os.path.join(ROOT, "include", "zero_ops.h")
A = 1 << 40                 # a made-up, well aligned address; arrays 1 GiB apart
GIB = 1 << 30


def at(k, off=0):
    return A + k * GIB + off


def error(call, *args):
    s = call(*args)
    return s, ops.lib().zero_ops_last_error().decode()


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    names = set(re.findall(r"\b(zero_[a-z_]+)\s*\(", text))
    assert names == set(ops.OPS_SYMBOLS)
    for n in names:
        assert hasattr(ops.lib(), n), n
        assert hasattr(zs, n), n
    assert zs.zero_ops_abi_version() == 1


def test_struct_layouts_match_header():
    assert ctypes.sizeof(ops.ZeroVocabLossDesc) == 88
    assert ctypes.sizeof(ops.ZeroAdamwTensor) == 88
    assert ctypes.sizeof(ops.ZeroAdamwCfg) == 24


def test_missing_library_fails_loudly(monkeypatch, tmp_path):
    monkeypatch.setattr(ops, "_lib", None)
    monkeypatch.setattr(ops, "LIB_PATH", str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match="no fallback"):
        zs.zero_ops_abi_version()


# ------------------------------------------------------------------ layer norm

def forward(x=at(0), xs=64, w=at(1), b=at(2), rows=4, width=64, t=2, at_=2, eps=1e-5, y=at(3), ys=64,
            mean=at(4), rstd=at(5)):
    return error(ops.lib().zero_layernorm_forward, x, xs, w, b, rows, width, t, at_, eps, y, ys, mean,
                 rstd, None)


def backward(dy=at(0), dys=64, x=at(1), xs=64, w=at(2), mean=at(3), rstd=at(4), rows=4, width=64, t=2,
             at_=2, dx=at(5), dxs=64, dw=at(6), db=at(7), ws=at(8), wn=1 << 20):
    return error(ops.lib().zero_layernorm_backward, dy, dys, x, xs, w, mean, rstd, rows, width, t, at_,
                 dx, dxs, dw, db, ws, wn, None)


@pytest.mark.parametrize("kw,word", [
    (dict(x=None), "NULL"), (dict(y=None), "NULL"), (dict(rows=-1), "rows"), (dict(width=0), "width"),
    (dict(xs=63), "stride"), (dict(ys=63), "stride"), (dict(xs=1 << 62), "stride"),
    (dict(t=0), "unknown type"), (dict(t=9), "unknown type"), (dict(at_=1), "affine"),
    (dict(eps=-1e-5), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(x=at(0, 1)), "aligned"), (dict(mean=at(4, 2)), "aligned"), (dict(w=at(1, 1)), "aligned"),
    (dict(y=at(0, 2)), "overlaps"), (dict(y=at(1)), "overlaps"), (dict(rstd=at(4)), "overlaps"),
    (dict(y=at(0), ys=128), "overlaps"), (dict(mean=at(3, 8)), "overlaps"),
])
def test_layernorm_forward_refuses(kw, word):
    s, msg = forward(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


def test_layernorm_unsupported_and_empty():
    assert forward(width=(1 << 24) + 1, xs=1 << 25, ys=1 << 25)[0] == zs.ZERO_ERR_UNSUPPORTED
    assert forward(rows=1 << 31)[0] == zs.ZERO_ERR_UNSUPPORTED
    assert forward(rows=0, x=None, y=None)[0] == zs.ZERO_OK
    assert backward(rows=0, dy=None, x=None, dx=None, mean=None, rstd=None, dw=None, db=None)[0] == zs.ZERO_OK


@pytest.mark.parametrize("kw,word", [
    (dict(dy=None), "NULL"), (dict(x=None), "NULL"), (dict(dx=None), "NULL"), (dict(mean=None), "NULL"),
    (dict(rstd=None), "NULL"), (dict(wn=0), "workspace"), (dict(ws=None), "workspace"),
    (dict(wn=4 * 2 * 64 * 4 - 1), "workspace"), (dict(dys=1), "stride"), (dict(dxs=63), "stride"),
    (dict(dx=at(0)), "overlaps"), (dict(dx=at(1)), "overlaps"), (dict(dw=at(7)), "overlaps"),
    (dict(ws=at(5)), "overlaps"), (dict(ws=at(8, 4)), "aligned"), (dict(dx=at(5, 1)), "aligned"),
    (dict(rows=-2), "rows"), (dict(width=0), "width"), (dict(at_=1), "affine"),
])
def test_layernorm_backward_refuses(kw, word):
    s, msg = backward(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


def test_layernorm_workspace():
    assert zs.zero_layernorm_workspace(0, 10) > 0
    assert zs.zero_layernorm_workspace(1, 10) == 80
    big = zs.zero_layernorm_workspace(1 << 20, 5120)
    assert big == zs.zero_layernorm_workspace(1 << 30, 5120)
    for bad in ((-1, 5), (5, 0)):
        with pytest.raises(zs.ZeroError):
            zs.zero_layernorm_workspace(*bad)


def test_columns_of_one_buffer_do_not_overlap():
    # x and y as columns [0, 64) and [64, 128) of rows of 128: found apart (the call then
    # goes on to ask for the device, which is not here)
    s, msg = forward(x=at(0), xs=128, y=at(0, 128), ys=128)
    assert "overlaps" not in msg
    s, msg = forward(x=at(0), xs=128, y=at(0, 126), ys=128)
    assert s == zs.ZERO_ERR_INVALID_ARG and "overlaps" in msg


# ------------------------------------------------------------------ vocabulary loss

def loss(hidden=at(0), weight=at(1), targets=at(2), losses=at(3), lse=at(4), out=at(5), dh=at(6), dw=at(7),
         ws=at(8), wn=1 << 29, desc=True, **d):
    f = dict(tokens=8, vocab=100, width=64, type=2, max_tokens=0, ignore_index=-100, hidden_stride=64,
             weight_stride=64, dhidden_stride=64, dweight_stride=64, grad_scale=1.0)
    f.update(d)
    c = ops.ZeroVocabLossDesc(**f)
    return error(ops.lib().zero_vocab_loss, ctypes.byref(c) if desc else None, hidden, weight, targets,
                 losses, lse, out, dh, dw, ws, wn, None)


@pytest.mark.parametrize("kw,word", [
    (dict(desc=False), "NULL"), (dict(hidden=None), "NULL"), (dict(weight=None), "NULL"),
    (dict(targets=None), "NULL"), (dict(losses=None), "NULL"), (dict(out=None), "NULL"),
    (dict(dh=None), "both or neither"), (dict(dw=None), "both or neither"), (dict(tokens=-1), "tokens"),
    (dict(vocab=0), "vocab"), (dict(width=0), "width"), (dict(hidden_stride=63), "stride"),
    (dict(weight_stride=1), "stride"), (dict(dhidden_stride=1), "stride"), (dict(dweight_stride=1), "stride"),
    (dict(max_tokens=-1), "max_tokens"), (dict(max_tokens=65536), "max_tokens"),
    (dict(grad_scale=float("inf")), "grad_scale"), (dict(grad_scale=float("nan")), "grad_scale"),
    (dict(type=7), "unknown type"), (dict(wn=100), "workspace"), (dict(ws=None), "workspace"),
    (dict(ws=at(8, 128)), "aligned"), (dict(hidden=at(0, 1)), "aligned"), (dict(targets=at(2, 4)), "aligned"),
    (dict(dh=at(0)), "overlaps"), (dict(dw=at(1)), "overlaps"), (dict(lse=at(3)), "overlaps"),
    (dict(ws=at(7, 256)), "overlaps"), (dict(out=at(3, 4)), "overlaps"),
])
def test_vocab_loss_refuses(kw, word):
    s, msg = loss(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


@pytest.mark.parametrize("kw", [dict(type=3), dict(width=(1 << 20) + 1, hidden_stride=1 << 21, weight_stride=1 << 21),
                                dict(vocab=1 << 21), dict(tokens=1 << 31)])
def test_vocab_loss_unsupported(kw):
    assert loss(**kw)[0] == zs.ZERO_ERR_UNSUPPORTED


def test_vocab_loss_workspace_grows_with_its_chunk():
    size = zs.zero_vocab_loss_workspace
    assert size(8192, 50257, 1600, gradient=False) < size(8192, 50257, 1600)
    # the chunk's exponentials are in it, and with several chunks the weight's fp32 sum
    assert size(8192, 50257, 1600) > 8192 * 50257 * 2
    assert size(8192, 50257, 1600, max_tokens=1024) > 1024 * 50257 * 2 + 50257 * 1600 * 4
    assert size(1 << 20, 50257, 1600, max_tokens=1024) < size(1 << 20, 50257, 1600)
    for bad in (dict(tokens=-1), dict(vocab=0), dict(width=0), dict(max_tokens=1 << 20)):
        kw = dict(tokens=1, vocab=1, width=1, max_tokens=0) | bad
        with pytest.raises(zs.ZeroError):
            size(kw["tokens"], kw["vocab"], kw["width"], max_tokens=kw["max_tokens"])


# ------------------------------------------------------------------ AdamW

def tensor(base=0, **kw):
    f = dict(numel=1000, type=2, grad=at(base), master=at(base + 1), param=at(base + 2), exp_avg=at(base + 3),
             exp_avg_sq=at(base + 4), exp_avg_exp=None, exp_avg_sq_exp=None, weight_decay=-1.0, lr_scale=1.0)
    f.update(kw)
    return ops.ZeroAdamwTensor(**f)


def init(tensors, hp=None, ls=None, n=None, **cfg):
    c = dict(state_bits=32, checked=1, max_grad_norm=0.0, seed=1)
    c.update(cfg)
    arr = (ops.ZeroAdamwTensor * max(1, len(tensors)))(*tensors)
    h = ctypes.c_void_p()
    hp = (hp or zs.AdamHParams()).to_c()
    ls = (ls or zs.LossScaleCfg()).to_c()
    s, msg = error(ops.lib().zero_adamw_init, arr, len(tensors) if n is None else n, ctypes.byref(hp),
                   ctypes.byref(ls), ctypes.byref(ops.ZeroAdamwCfg(**c)), ctypes.byref(h))
    assert not h.value
    return s, msg


@pytest.mark.parametrize("kw,word", [
    (dict(numel=-1), "numel"), (dict(type=5), "unknown type"), (dict(grad=None), "NULL"),
    (dict(master=None), "NULL"), (dict(param=None), "param"), (dict(type=3), "param"),
    (dict(exp_avg=None), "NULL"), (dict(exp_avg_sq=None), "NULL"), (dict(exp_avg_exp=at(9)), "exponents"),
    (dict(exp_avg_sq_exp=at(9)), "exponents"), (dict(weight_decay=float("nan")), "weight_decay"),
    (dict(lr_scale=-1.0), "lr_scale"), (dict(master=at(1, 2)), "aligned"), (dict(grad=at(0, 1)), "aligned"),
    (dict(param=at(1)), "overlaps"), (dict(grad=at(3, 4)), "overlaps"), (dict(exp_avg_sq=at(3, 3996)), "overlaps"),
])
def test_adamw_init_refuses_tensors(kw, word):
    s, msg = init([tensor(**kw)])
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


def test_adamw_init_refuses_the_rest():
    s, msg = init([tensor(0), tensor(10, master=at(1, 2000))])
    assert s == zs.ZERO_ERR_INVALID_ARG and "overlaps" in msg
    s, msg = init([tensor(0), tensor(10, grad=at(2, 100))])            # a read one inside a written one
    assert s == zs.ZERO_ERR_INVALID_ARG and "overlaps" in msg
    s, msg = init([tensor(0, numel=1 << 44)])
    assert s == zs.ZERO_ERR_UNSUPPORTED
    for cfg, word in ((dict(state_bits=16), "state_bits"), (dict(checked=2), "checked"),
                      (dict(max_grad_norm=-1.0), "max_grad_norm"), (dict(max_grad_norm=float("nan")), "max_grad_norm"),
                      (dict(max_grad_norm=1.0, checked=0), "checked"), (dict(state_bits=8), "exponents")):
        s, msg = init([tensor()], **cfg)
        assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (cfg, msg)
    s, msg = init([tensor(exp_avg_exp=at(5))], state_bits=8)
    assert s == zs.ZERO_ERR_INVALID_ARG and "one moment" in msg
    for n in (0, -3):
        assert init([tensor()], n=n)[0] == zs.ZERO_ERR_INVALID_ARG
    for hp in (dict(lr=-1.0), dict(beta1=1.0), dict(beta2=1 - 1e-9), dict(eps=0.0), dict(weight_decay=-1.0),
               dict(bias_correction=2), dict(initial_step=-1), dict(wd_mode=7)):
        s, msg = init([tensor()], hp=zs.AdamHParams(**hp))
        assert s == zs.ZERO_ERR_INVALID_ARG, hp
    for ls in (dict(init_scale=0.0), dict(min_scale=float("inf")), dict(dynamic=3), dict(growth_interval=0)):
        assert init([tensor()], ls=zs.LossScaleCfg(**ls))[0] == zs.ZERO_ERR_INVALID_ARG, ls


def test_adamw_dead_handles():
    out, t, sc, g = ops.ZeroStepInfo(), ctypes.c_int64(), ctypes.c_double(), ctypes.c_int64()
    L = ops.lib()
    for h in (None, ctypes.c_void_p(at(3))):
        assert L.zero_adamw_step(h, None, None) == zs.ZERO_ERR_STATE
        assert L.zero_adamw_result(h, None, ctypes.byref(out)) == zs.ZERO_ERR_STATE
        assert L.zero_adamw_set_grads(h, None, 1, None) == zs.ZERO_ERR_STATE
        assert L.zero_adamw_get_counters(h, None, ctypes.byref(t), ctypes.byref(sc), ctypes.byref(g)) == zs.ZERO_ERR_STATE
        assert L.zero_adamw_set_counters(h, None, 0, 1.0, 0) == zs.ZERO_ERR_STATE
        assert L.zero_adamw_destroy(h) == zs.ZERO_ERR_STATE


def test_moments_refuse():
    L = ops.lib()
    for args, word in (((None, 5, 1, at(1), at(2), None), "NULL"), ((at(0), -1, 1, at(1), at(2), None), "n outside"),
                       ((at(0), 5, 2, at(1), at(2), None), "is_signed"), ((at(0, 2), 5, 1, at(1), at(2), None), "aligned"),
                       ((at(0), 5, 1, at(0, 4), at(2), None), "overlaps")):
        s, msg = error(L.zero_moments_pack, *args)
        assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, msg
    for args, word in (((at(0), None, 5, 1, 3, at(2), None), "NULL"), ((at(0), at(1), 5, 1, 1, at(2), None), "out_type"),
                       ((at(0), at(1), 5, -1, 3, at(2), None), "is_signed"), ((at(0), at(1), 5, 1, 3, at(2, 2), None), "aligned"),
                       ((at(0), at(1), 5, 1, 3, at(1), None), "overlaps")):
        s, msg = error(L.zero_moments_unpack, *args)
        assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, msg
    assert L.zero_moments_pack(None, 0, 1, None, None, None) == zs.ZERO_OK
    assert L.zero_moments_unpack(None, None, 0, 0, 3, None, None) == zs.ZERO_OK


# ------------------------------------------------------------------ binding, code

def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        zs.zero_layernorm_forward(x, None, None, x)
    with pytest.raises(TypeError):
        zs.zero_layernorm_forward([1.0], None, None, x)
    with pytest.raises(ValueError, match="GPU"):
        zs.zero_vocab_loss(x, x, x, x, None, x)
    with pytest.raises(ValueError, match="GPU"):
        zs.zero_moments_pack(x, x, x, signed=True)
    with pytest.raises(ValueError, match="GPU"):
        zs.zero_adamw_init([zs.AdamWTensor(x, x, None, x, x)], hp=zs.AdamHParams(), ls=zs.LossScaleCfg())


@pytest.mark.parametrize("src", ["ops_norm.hip", "ops_loss.hip", "ops_adamw.hip"])
def test_kernels_have_no_packed_fp32(src):
    asm = build.device_asm(src)
    body = [ln for ln in asm.splitlines() if ln.startswith("\t") and not ln.startswith("\t.")]
    assert len(body) > 500
    assert not [ln for ln in body if re.match(r"\s*v_pk_(add|mul|fma)_f32", ln)]
    # no kernel keeps registers in memory
    assert set(re.findall(r"\.private_segment_fixed_size:\s*(\d+)", asm)) == {"0"}


def test_loads_into_lds_are_the_only_users_of_their_address_register():
    """The products' loads set m0 and use it in one piece of assembly; nothing
    else in the kernels may touch it."""
    asm = build.device_asm("ops_loss.hip").splitlines()
    uses = [k for k, ln in enumerate(asm) if re.search(r"\bm0\b", ln) and ln.startswith("\t") and not ln.startswith("\t.")]
    assert len(uses) > 8
    for k in uses:
        assert re.match(r"\s*s_mov_b32 m0, s\d+", asm[k]), asm[k]
        assert "buffer_load_dwordx4" in asm[k + 1] and "lds" in asm[k + 1], asm[k + 1]
