"""What the operators' binding keeps alive, without a GPU: the library, torch's streams
and the gradients are stand-ins that note what is asked of them."""
import types

import pytest

import zero_dp_sharded_amd as zs
from zero_dp_sharded_amd import ops


class Grad:
    dtype = "t"

    def __init__(self, n=4):
        self.n, self.read_on = n, []

    def numel(self):
        return self.n

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.read_on.append(stream)


class Library:
    """Every call succeeds, or fails with `status`."""

    def __init__(self):
        self.status = zs.ZERO_OK

    def __getattr__(self, name):
        if name == "zero_ops_last_error":
            return lambda: b"refused"
        return lambda *a: self.status


@pytest.fixture
def handle(monkeypatch):
    lib = Library()
    cuda = types.SimpleNamespace(ExternalStream=lambda p: ("stream", p), default_stream=lambda: ("stream", 0))
    monkeypatch.setattr(ops, "torch", types.SimpleNamespace(cuda=cuda))
    monkeypatch.setattr(ops, "lib", lambda: lib)
    monkeypatch.setattr(ops, "_flat", lambda name, t, dtype, n: t.data_ptr())
    monkeypatch.setattr(ops, "_current", lambda stream: 7 if stream is None else stream)
    grads = [Grad(), Grad(0), Grad()]
    monkeypatch.setattr(ops, "_adamw", {99: ops._Held([], grads, set())})
    return types.SimpleNamespace(h=99, lib=lib, grads=grads)


def test_old_gradients_are_kept_from_reuse_on_the_streams_that_read_them(handle):
    h, first = handle.h, handle.grads
    zs.zero_adamw_step(h, stream=5)
    zs.zero_adamw_step(h, stream=5)
    zs.zero_adamw_step(h)
    zs.zero_adamw_step(h, stream=0)
    second = [Grad() for _ in range(3)]
    zs.zero_adamw_set_grads(h, second, stream=5)
    for g in (first[0], first[2]):
        assert sorted(g.read_on) == [("stream", 0), ("stream", 5), ("stream", 7)]
    assert not first[1].read_on and not any(g.read_on for g in second)
    # no step has read the second ones
    third = [Grad() for _ in range(3)]
    zs.zero_adamw_set_grads(h, third, stream=5)
    assert not any(g.read_on for g in second)
    assert ops._adamw[h].grads == third


def test_a_stream_that_was_waited_for_no_longer_reads(handle):
    h = handle.h
    zs.zero_adamw_step(h, stream=5)
    zs.zero_adamw_step(h, stream=6)
    zs.zero_adamw_result(h, stream=5)
    zs.zero_adamw_set_grads(h, [Grad() for _ in range(3)])
    assert handle.grads[0].read_on == [("stream", 6)]
    zs.zero_adamw_step(h, stream=6)
    zs.zero_adamw_get_counters(h, stream=6)
    last = ops._adamw[h].grads
    zs.zero_adamw_set_grads(h, [Grad() for _ in range(3)])
    assert not last[0].read_on


def test_refused_gradients_leave_everything_as_it_was(handle):
    h = handle.h
    zs.zero_adamw_step(h, stream=5)
    handle.lib.status = zs.ZERO_ERR_INVALID_ARG
    with pytest.raises(zs.ZeroError):
        zs.zero_adamw_set_grads(h, [Grad() for _ in range(3)])
    with pytest.raises(zs.ZeroError):
        zs.zero_adamw_step(h, stream=8)
    assert ops._adamw[h].grads == handle.grads and ops._adamw[h].streams == {5} and not handle.grads[0].read_on
