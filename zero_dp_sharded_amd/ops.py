"""The training operators of libzeroops.so (include/zero_ops.h): layer norm, the
softmax cross entropy over a vocabulary with its gradients, and AdamW over many
tensors with moments in 32 or 8 bits.

A thin ctypes binding, as the package's binding of libzeroshard.so is: functions
carry the C names, tensors become device pointers, strides and types, and the
library's checks raise ZeroError.  There is no CPU fallback.  Calls enqueue: a tensor given on
a stream other than its own must live, as for any such use, until that work has ended
(Tensor.record_stream); an AdamW handle keeps its tensors itself.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

from . import (AdamHParams, HERE, LossScaleCfg, StepInfo, ZERO_BF16, ZERO_FP16, ZERO_FP32, ZERO_OK,
               ZeroAdamHParams, ZeroError, ZeroLossScaleCfg, ZeroStepInfo, _stream_ptr)

LIB_PATH = os.environ.get("ZERO_OPS_LIB") or os.path.join(HERE, "libzeroops.so")

_i32, _i64, _u64, _f64, _vp = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_double,
                               ctypes.c_void_p)
_ptr = ctypes.POINTER

OPS_SYMBOLS = (
    "zero_layernorm_forward", "zero_layernorm_workspace", "zero_layernorm_backward",
    "zero_vocab_loss_workspace", "zero_vocab_loss", "zero_adamw_init", "zero_adamw_set_grads",
    "zero_adamw_step", "zero_adamw_result", "zero_adamw_get_counters", "zero_adamw_set_counters",
    "zero_adamw_destroy", "zero_moments_pack", "zero_moments_unpack", "zero_ops_last_error",
    "zero_ops_abi_version",
)

BLOCK = 256            # elements that share one exponent of 8-bit moments


class ZeroVocabLossDesc(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("vocab", _i64), ("width", _i64), ("type", ctypes.c_int),
                ("max_tokens", _i64), ("ignore_index", _i64), ("hidden_stride", _i64),
                ("weight_stride", _i64), ("dhidden_stride", _i64), ("dweight_stride", _i64),
                ("grad_scale", _f64)]


class ZeroAdamwTensor(ctypes.Structure):
    _fields_ = [("numel", _i64), ("type", ctypes.c_int), ("grad", _vp), ("master", _vp),
                ("param", _vp), ("exp_avg", _vp), ("exp_avg_sq", _vp), ("exp_avg_exp", _vp),
                ("exp_avg_sq_exp", _vp), ("weight_decay", _f64), ("lr_scale", _f64)]


class ZeroAdamwCfg(ctypes.Structure):
    _fields_ = [("state_bits", _i32), ("checked", _i32), ("max_grad_norm", _f64), ("seed", _u64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m zero_dp_sharded_amd.build` "
                "(or __graft_entry__.build()); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        L.zero_layernorm_forward.argtypes = [_vp, _i64, _vp, _vp, _i64, _i64, ctypes.c_int,
                                             ctypes.c_int, _f64, _vp, _i64, _vp, _vp, _vp]
        L.zero_layernorm_workspace.argtypes = [_i64, _i64, _ptr(_i64)]
        L.zero_layernorm_backward.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64,
                                              ctypes.c_int, ctypes.c_int, _vp, _i64, _vp, _vp, _vp,
                                              _i64, _vp]
        L.zero_vocab_loss_workspace.argtypes = [_i64, _i64, _i64, _i64, _i32, _ptr(_i64)]
        L.zero_vocab_loss.argtypes = [_ptr(ZeroVocabLossDesc), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _i64, _vp]
        L.zero_adamw_init.argtypes = [_ptr(ZeroAdamwTensor), _i32, _ptr(ZeroAdamHParams),
                                      _ptr(ZeroLossScaleCfg), _ptr(ZeroAdamwCfg), _ptr(_vp)]
        L.zero_adamw_set_grads.argtypes = [_vp, _ptr(_vp), _i32, _vp]
        L.zero_adamw_step.argtypes = [_vp, _ptr(ZeroAdamHParams), _vp]
        L.zero_adamw_result.argtypes = [_vp, _vp, _ptr(ZeroStepInfo)]
        L.zero_adamw_get_counters.argtypes = [_vp, _vp, _ptr(_i64), _ptr(_f64), _ptr(_i64)]
        L.zero_adamw_set_counters.argtypes = [_vp, _vp, _i64, _f64, _i64]
        L.zero_adamw_destroy.argtypes = [_vp]
        L.zero_moments_pack.argtypes = [_vp, _i64, _i32, _vp, _vp, _vp]
        L.zero_moments_unpack.argtypes = [_vp, _vp, _i64, _i32, ctypes.c_int, _vp, _vp]
        L.zero_ops_last_error.argtypes = []
        L.zero_ops_abi_version.argtypes = []
        for name in OPS_SYMBOLS:
            getattr(L, name).restype = ctypes.c_int
        L.zero_ops_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != ZERO_OK:
        raise ZeroError(status, where, lib().zero_ops_last_error().decode())


def zero_ops_abi_version() -> int:
    return int(lib().zero_ops_abi_version())


def zero_ops_last_error() -> str:
    return lib().zero_ops_last_error().decode()


# ------------------------------------------------------------------ marshalling

# torch and what of it every call needs, set by the first call (the library's
# host-only entry points work without torch)
torch = None
_CODES: dict = {}


def _load():
    global torch
    import torch as module
    _CODES.update({module.float16: ZERO_FP16, module.bfloat16: ZERO_BF16, module.float32: ZERO_FP32})
    torch = module
    return module


def _current(stream) -> int:
    """hipStream_t of a stream, or of torch's current stream if None (by the raw
    getter: the stream object alone would cost a small call a fifth of its time)."""
    if stream is not None:
        return _stream_ptr(stream)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _type_of(name: str, t) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float16, bfloat16 or float32, got {t.dtype}")
    return code


def _tensor(name: str, t, dtype) -> None:
    """A GPU tensor of the dtype (None: any)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must live on the GPU, got {t.device}")


def _matrix(name: str, t) -> tuple:
    _tensor(name, t, None)
    if t.dim() != 2:
        raise ValueError(f"{name}: expected two dimensions")
    return t.shape


def _rows(name: str, t, dtype, rows: int, width: int) -> tuple:
    """(address, row stride) of a [rows, width] tensor whose last dimension is
    contiguous; its row stride is free."""
    _tensor(name, t, dtype)
    if t.shape != (rows, width):
        raise ValueError(f"{name}: expected shape ({rows}, {width}), got {tuple(t.shape)}")
    stride, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), (stride if rows > 1 else max(width, 1))


def _flat(name: str, t, dtype, n: int) -> Optional[int]:
    """Address of a contiguous tensor of exactly n elements; None stays None."""
    if t is None:
        return None
    _tensor(name, t, dtype)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous with {n} elements, got {tuple(t.shape)}")
    return t.data_ptr()


def _space(t) -> tuple:
    if t is None:
        return None, 0
    _tensor("workspace", t, torch.uint8)
    if not t.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return t.data_ptr(), t.numel()


# ------------------------------------------------------------------ layer norm

def zero_layernorm_forward(x, weight, bias, y, mean=None, rstd=None, *, eps: float = 1e-5,
                           stream=None) -> None:
    """y = (x - mean) * rstd * weight + bias over the last of x's two dimensions;
    mean and rstd (fp32, one a row) for the backward pass.  weight and bias (both
    of x's type or both fp32) may be None."""
    torch or _load()
    rows, width = _matrix("x", x)
    t = _type_of("x", x)
    given = weight if weight is not None else bias
    at = t if given is None else _type_of("weight", given)
    xp, xs = _rows("x", x, x.dtype, rows, width)
    yp, ys = _rows("y", y, x.dtype, rows, width)
    adt = None if given is None else given.dtype
    _check(lib().zero_layernorm_forward(
        xp, xs, _flat("weight", weight, adt, width), _flat("bias", bias, adt, width), rows, width,
        t, at, eps, yp, ys, _flat("mean", mean, torch.float32, rows),
        _flat("rstd", rstd, torch.float32, rows), _current(stream)), "zero_layernorm_forward")


def zero_layernorm_workspace(rows: int, width: int) -> int:
    """Bytes of workspace for zero_layernorm_backward."""
    n = _i64()
    _check(lib().zero_layernorm_workspace(rows, width, ctypes.byref(n)), "zero_layernorm_workspace")
    return n.value


def zero_layernorm_backward(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, workspace=None,
                            *, stream=None) -> None:
    """dx, and (where given) dweight and dbias, for dy and the forward pass's x, mean
    and rstd.  workspace: uint8, zero_layernorm_workspace(rows, width) bytes, needed
    with dweight or dbias."""
    torch or _load()
    rows, width = _matrix("x", x)
    t = _type_of("x", x)
    given = next((g for g in (weight, dweight, dbias) if g is not None), None)
    at = t if given is None else _type_of("weight", given)
    adt = None if given is None else given.dtype
    dyp, dys = _rows("dy", dy, x.dtype, rows, width)
    xp, xs = _rows("x", x, x.dtype, rows, width)
    dxp, dxs = _rows("dx", dx, x.dtype, rows, width)
    wp, wn = _space(workspace)
    _check(lib().zero_layernorm_backward(
        dyp, dys, xp, xs, _flat("weight", weight, adt, width),
        _flat("mean", mean, torch.float32, rows), _flat("rstd", rstd, torch.float32, rows), rows,
        width, t, at, dxp, dxs, _flat("dweight", dweight, adt, width),
        _flat("dbias", dbias, adt, width), wp, wn, _current(stream)), "zero_layernorm_backward")


# ------------------------------------------------------------------ vocabulary loss

def zero_vocab_loss_workspace(tokens: int, vocab: int, width: int, *, gradient: bool = True,
                              max_tokens: int = 0) -> int:
    """Bytes of workspace for zero_vocab_loss."""
    n = _i64()
    _check(lib().zero_vocab_loss_workspace(tokens, vocab, width, max_tokens, int(gradient),
                                           ctypes.byref(n)), "zero_vocab_loss_workspace")
    return n.value


def zero_vocab_loss(hidden, weight, targets, losses, lse, loss, dhidden=None, dweight=None,
                    workspace=None, *, grad_scale: float = 1.0, ignore_index: int = -100,
                    max_tokens: int = 0, stream=None) -> None:
    """Softmax cross entropy of hidden [tokens, width] against weight [vocab, width]
    and targets [tokens] (int64): losses [tokens], lse [tokens] (or None) and the
    mean loss in fp32, and with dhidden and dweight both gradients of the mean
    times grad_scale.  workspace: uint8, zero_vocab_loss_workspace bytes."""
    torch or _load()
    (tokens, width), (vocab, _) = _matrix("hidden", hidden), _matrix("weight", weight)
    d = ZeroVocabLossDesc(tokens=tokens, vocab=vocab, width=width, type=_type_of("hidden", hidden),
                          max_tokens=max_tokens, ignore_index=ignore_index, grad_scale=grad_scale)
    hp, d.hidden_stride = _rows("hidden", hidden, hidden.dtype, tokens, width)
    wp, d.weight_stride = _rows("weight", weight, hidden.dtype, vocab, width)
    dhp = dwp = None
    if dhidden is not None:
        dhp, d.dhidden_stride = _rows("dhidden", dhidden, hidden.dtype, tokens, width)
    if dweight is not None:
        dwp, d.dweight_stride = _rows("dweight", dweight, hidden.dtype, vocab, width)
    sp, sn = _space(workspace)
    _check(lib().zero_vocab_loss(
        ctypes.byref(d), hp, wp, _flat("targets", targets, torch.int64, tokens),
        _flat("losses", losses, torch.float32, tokens), _flat("lse", lse, torch.float32, tokens),
        _flat("loss", loss, torch.float32, 1), dhp, dwp, sp, sn, _current(stream)),
        "zero_vocab_loss")


# ------------------------------------------------------------------ AdamW over tensors

@dataclass
class AdamWTensor:
    """One tensor of an AdamW handle: gradient, fp32 master, 2-byte param (None with fp32
    storage), the moments (fp32, or uint8 with their int8 exponents, one for every
    256 elements), its weight decay (None: the hyper-parameters') and a factor of
    the learning rate.  All contiguous."""
    grad: object
    master: object
    param: object
    exp_avg: object
    exp_avg_sq: object
    exp_avg_exp: object = None
    exp_avg_sq_exp: object = None
    weight_decay: Optional[float] = None
    lr_scale: float = 1.0

    def to_c(self, state_bits: int) -> ZeroAdamwTensor:
        torch or _load()
        _tensor("grad", self.grad, None)
        n, t = self.grad.numel(), _type_of("grad", self.grad)
        state = torch.float32 if state_bits == 32 else torch.uint8
        blocks = -(-n // BLOCK)
        if self.weight_decay is not None and self.weight_decay < 0:
            raise ValueError("weight_decay must be >= 0")
        return ZeroAdamwTensor(
            n, t, _flat("grad", self.grad, None, n), _flat("master", self.master, torch.float32, n),
            _flat("param", self.param, self.grad.dtype, n), _flat("exp_avg", self.exp_avg, state, n),
            _flat("exp_avg_sq", self.exp_avg_sq, state, n),
            _flat("exp_avg_exp", self.exp_avg_exp, torch.int8, blocks),
            _flat("exp_avg_sq_exp", self.exp_avg_sq_exp, torch.int8, blocks),
            -1.0 if self.weight_decay is None else self.weight_decay, self.lr_scale)


@dataclass
class _Held:
    """What a live handle made through this binding reads and writes, kept from being
    freed under it."""
    tensors: list
    grads: list
    # those that steps of these gradients were enqueued on and not waited for, as hipStream_t (a
    # stream that is not torch's must live as long)
    streams: set


_adamw = {}


def zero_adamw_init(tensors: Sequence[AdamWTensor], *, hp: AdamHParams, ls: LossScaleCfg,
                    state_bits: int = 32, checked: bool = True, max_grad_norm: float = 0.0,
                    seed: int = 0) -> int:
    """A handle over the tensors, which are kept alive until it is destroyed."""
    arr = (ZeroAdamwTensor * len(tensors))(*[t.to_c(state_bits) for t in tensors])
    cfg = ZeroAdamwCfg(state_bits, int(checked), max_grad_norm, seed)
    h = _vp()
    _check(lib().zero_adamw_init(arr, len(tensors), ctypes.byref(hp.to_c()), ctypes.byref(ls.to_c()),
                                 ctypes.byref(cfg), ctypes.byref(h)), "zero_adamw_init")
    _adamw[h.value] = _Held(list(tensors), [t.grad for t in tensors], set())
    return h.value


def zero_adamw_set_grads(h: int, grads: Sequence, stream=None) -> None:
    """Other gradient tensors, of the same types and sizes, for the steps that follow.  The
    old ones are let go, but their memory is not used again before the steps that were
    enqueued through this binding have read them (of a graph's replays the caller knows)."""
    torch or _load()
    known = _adamw.get(h)
    if known is not None:
        if len(grads) != len(known.grads):
            raise ValueError(f"expected {len(known.grads)} gradients, got {len(grads)}")
        ptrs = [_flat(f"gradient {i}", g, old.dtype, old.numel()) for i, (g, old) in enumerate(zip(grads, known.grads))]
    else:
        ptrs = [g.data_ptr() for g in grads]
    _check(lib().zero_adamw_set_grads(h, (_vp * len(ptrs))(*ptrs), len(ptrs), _current(stream)),
           "zero_adamw_set_grads")
    if known is not None:
        for s in known.streams:
            used = torch.cuda.ExternalStream(s) if s else torch.cuda.default_stream()
            for g in known.grads:
                if g.numel():
                    g.record_stream(used)
        known.grads, known.streams = list(grads), set()


def zero_adamw_step(h: int, hp: Optional[AdamHParams] = None, stream=None) -> None:
    """Enqueue one step of every tensor (capturable in a graph)."""
    torch or _load()
    hpc = ctypes.byref(hp.to_c()) if hp is not None else None
    s = _current(stream)
    _check(lib().zero_adamw_step(h, hpc, s), "zero_adamw_step")
    known = _adamw.get(h)
    if known is not None:
        known.streams.add(s)


def zero_adamw_result(h: int, stream=None) -> StepInfo:
    """The last step's result; waits for it."""
    torch or _load()
    out = ZeroStepInfo()
    s = _current(stream)
    _check(lib().zero_adamw_result(h, s, ctypes.byref(out)), "zero_adamw_result")
    _waited(h, s)
    return StepInfo.from_c(out)


def _waited(h: int, stream: int) -> None:
    """The stream's steps have ended."""
    known = _adamw.get(h)
    if known is not None:
        known.streams.discard(stream)


def zero_adamw_get_counters(h: int, stream=None):
    torch or _load()
    t, s, g = _i64(), _f64(), _i64()
    at = _current(stream)
    _check(lib().zero_adamw_get_counters(h, at, ctypes.byref(t), ctypes.byref(s),
                                         ctypes.byref(g)), "zero_adamw_get_counters")
    _waited(h, at)
    return t.value, s.value, g.value


def zero_adamw_set_counters(h: int, step_t: int, scale: float, good_steps: int, stream=None) -> None:
    torch or _load()
    _check(lib().zero_adamw_set_counters(h, _current(stream), step_t, scale, good_steps),
           "zero_adamw_set_counters")


def zero_adamw_destroy(h: int) -> None:
    _check(lib().zero_adamw_destroy(h), "zero_adamw_destroy")
    _adamw.pop(h, None)


def zero_moments_pack(x, codes, exps, *, signed: bool, stream=None) -> None:
    """fp32 moments to 8 bits: codes (uint8) and exps (int8, one for every 256 elements)."""
    torch or _load()
    _tensor("x", x, torch.float32)
    n = x.numel()
    _check(lib().zero_moments_pack(_flat("x", x, torch.float32, n), n, int(signed),
                                   _flat("codes", codes, torch.uint8, n),
                                   _flat("exps", exps, torch.int8, -(-n // BLOCK)),
                                   _current(stream)), "zero_moments_pack")


def zero_moments_unpack(codes, exps, out, *, signed: bool, stream=None) -> None:
    """What 8-bit moments stand for, into out (fp32 or bf16; exact in both)."""
    torch or _load()
    _tensor("codes", codes, torch.uint8)
    n = codes.numel()
    _check(lib().zero_moments_unpack(_flat("codes", codes, torch.uint8, n),
                                     _flat("exps", exps, torch.int8, -(-n // BLOCK)), n, int(signed),
                                     _type_of("out", out), _flat("out", out, None, n),
                                     _current(stream)), "zero_moments_unpack")
