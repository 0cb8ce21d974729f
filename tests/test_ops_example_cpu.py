"""The example's layout and arguments, without a GPU."""
import pytest
import torch

from zero_dp_sharded_amd import train_head


def test_the_tensors_are_views_of_flat_arrays():
    m = train_head.Model(101, 48, "bf16", torch.device("cpu"), 3)
    ends = 0
    for name, (at, n, shape) in m.spans.items():
        assert at % 256 == 0 and at >= ends
        ends = at + n
        v = m.view(m.grad, name)
        assert v.shape == shape and v.data_ptr() == m.grad.data_ptr() + 2 * at
    assert m.total % 256 == 0 and m.total >= ends
    assert torch.equal(m.param, m.master.to(torch.bfloat16))
    assert m.view(m.master, "norm.weight").eq(1).all() and not m.view(m.master, "norm.bias").any()


def test_arguments_are_refused():
    with pytest.raises(ValueError):
        train_head.train(update="sgd")
    with pytest.raises(SystemExit):
        train_head.main(["--storage", "fp8"])
