"""The example that runs the operators together: the loss falls, the update over
tensors has the same bits as the owner's step on the flat arrays, and 8-bit moments
train as fp32 ones do."""
import math

import pytest
import torch

from zero_dp_sharded_amd import train_head

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("update", ["adamw", "bytes"])
@pytest.mark.parametrize("storage", ["fp16", "bf16"])
def test_the_loss_falls(update, storage):
    seen, model, info = train_head.train(steps=60, update=update, storage=storage)
    assert abs(seen[0] - math.log(1009)) < 0.5
    assert all(math.isfinite(x) for x in seen)
    assert min(seen[-5:]) < 0.6 * seen[0], seen[::10]
    assert info.step_t == 60 and not info.skipped


def test_the_same_bits_as_the_owners_step():
    a, ma, ia = train_head.train(steps=8, update="adamw", width=200, vocab=601)
    b, mb, ib = train_head.train(steps=8, update="owner", width=200, vocab=601)
    assert a == b
    assert torch.equal(ma.master, mb.master) and torch.equal(ma.param, mb.param)
    assert (ia.step_t, ia.scale_next, ia.skipped) == (ib.step_t, ib.scale_next, ib.skipped)
    assert abs(ia.grad_norm - ib.grad_norm) <= 1e-12 * ib.grad_norm


def test_bytes_follow_fp32_moments():
    a, _, _ = train_head.train(steps=40, update="adamw")
    b, _, _ = train_head.train(steps=40, update="bytes")
    assert abs(a[-1] - b[-1]) < 0.15 * a[0], (a[-1], b[-1])
