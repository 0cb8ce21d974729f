"""The log probabilities' boundary, checked without a GPU: struct layouts, workspaces, and the
refusals that come before any device work."""
import ctypes

import pytest

import zero_dp_sharded_amd as zs
from test_ops_cpu import at, error
from zero_dp_sharded_amd import ops


def forward(h=at(0), w=at(1), ids=at(2), logp=at(3), lse=at(4), ent=at(5), ti=at(6), tl=at(7), ws=at(8), wn=1 << 29, desc=True, **d):
    f = dict(tokens=10, vocab=100, width=64, type=2, top=4, max_tokens=0, ignore_index=-100, hidden_stride=64, weight_stride=64)
    f.update(d)
    c = ops.ZeroTokenLogprobsDesc(**f)
    return error(ops.lib().zero_token_logprobs, ctypes.byref(c) if desc else None, h, w, ids, logp, lse, ent, ti, tl, ws, wn, None)


def backward(h=at(0), w=at(1), ids=at(2), lse=at(3), ent=at(4), dl=at(5), de=at(6), dh=at(7), dw=at(8), ws=at(9), wn=1 << 29, desc=True, **d):
    f = dict(tokens=10, vocab=100, width=64, type=2, max_tokens=0, ignore_index=-100, hidden_stride=64, weight_stride=64, dhidden_stride=64,
             dweight_stride=64)
    f.update(d)
    c = ops.ZeroTokenLogprobsGradDesc(**f)
    return error(ops.lib().zero_token_logprobs_backward, ctypes.byref(c) if desc else None, h, w, ids, lse, ent, dl, de, dh, dw, ws, wn, None)


COMMON = [(dict(desc=False), "NULL"), (dict(h=None), "NULL"), (dict(w=None), "NULL"), (dict(lse=None), "NULL"), (dict(tokens=-1), "tokens"),
          (dict(vocab=0), "vocab"), (dict(width=0), "width"), (dict(type=0), "unknown type"), (dict(hidden_stride=63), "stride"),
          (dict(weight_stride=63), "stride"), (dict(max_tokens=-1), "max_tokens"), (dict(max_tokens=65536), "max_tokens"), (dict(wn=100), "workspace"),
          (dict(ws=None), "workspace"), (dict(h=at(0, 1)), "aligned"), (dict(ids=at(2, 4)), "aligned"), (dict(lse=at(1)), "overlaps")]


@pytest.mark.parametrize("kw,word", COMMON[:-1] + [
    (dict(lse=at(1)), "overlaps"), (dict(ids=None), "both or neither"), (dict(logp=None), "both or neither"), (dict(top=-1), "top"),
    (dict(top=65), "top"), (dict(top=5, vocab=4), "top"), (dict(ti=None), "top_ids"), (dict(tl=None), "top_ids"), (dict(top=0), "top_ids"),
    (dict(ws=at(8, 128)), "aligned"), (dict(ent=at(3)), "overlaps"), (dict(ti=at(2)), "overlaps"), (dict(tl=at(8, 256)), "overlaps"),
])
def test_forward_refuses(kw, word):
    s, msg = forward(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


@pytest.mark.parametrize("kw,word", COMMON[:-1] + [
    (dict(ids=None), "NULL"), (dict(dl=None), "NULL"), (dict(dh=None), "NULL"), (dict(dw=None), "NULL"), (dict(ent=None), "dentropy"),
    (dict(dhidden_stride=63), "stride"), (dict(dweight_stride=1), "stride"), (dict(dh=at(0)), "overlaps"), (dict(dw=at(1)), "overlaps"),
    (dict(dw=at(7)), "overlaps"), (dict(ws=at(6)), "overlaps"), (dict(dl=at(5, 2)), "aligned"),
])
def test_backward_refuses(kw, word):
    s, msg = backward(**kw)
    assert s == zs.ZERO_ERR_INVALID_ARG and word in msg, (s, msg)


def test_unsupported_and_empty():
    assert ctypes.sizeof(ops.ZeroTokenLogprobsDesc) == 64 and ctypes.sizeof(ops.ZeroTokenLogprobsGradDesc) == 80
    for call in (forward, backward):
        for kw in (dict(type=3), dict(width=(1 << 20) + 1), dict(vocab=1 << 21), dict(tokens=1 << 31)):
            assert call(**kw)[0] == zs.ZERO_ERR_UNSUPPORTED, kw
    assert forward(tokens=0, h=None, w=None)[0] == zs.ZERO_OK
    assert "overlaps" not in backward(de=None, ent=at(7))[1]


def test_workspaces():
    n = zs.zero_token_logprobs_workspace
    assert n(1000, 5000, 64) < n(1000, 5000, 64, top=1) == n(1000, 5000, 64, top=9)
    assert n(1000, 5000, 64, gradient=True) > zs.zero_vocab_loss_workspace(1000, 5000, 64)
    assert n(100000, 5000, 64, max_tokens=1024, top=2) < n(100000, 5000, 64, top=2)
    for bad in ((-1, 5, 5), (1, 0, 5), (1, 5, 0)):
        with pytest.raises(zs.ZeroError):
            n(*bad)
    with pytest.raises(zs.ZeroError):
        n(1, 5, 5, top=6)
