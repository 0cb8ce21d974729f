"""The example's model with a layer in 8 bits, and its arguments, without a GPU."""
import pytest
import torch

from zero_dp_sharded_amd import train_head


def test_the_tensors_of_the_layer():
    m = train_head.Model(101, 48, "bf16", torch.device("cpu"), 3, "bytes")
    assert list(m.spans) == ["embed", "norm.weight", "body", "norm2.weight", "head"]
    assert m.part("body").shape == (48, 48) and m.part("norm2.weight").eq(1).all()
    assert m.grad_of("body").data_ptr() == m.grad.data_ptr() + 2 * m.spans["body"][0]


def test_the_plain_model_is_what_it_was():
    a = train_head.Model(101, 48, "bf16", torch.device("cpu"), 3)
    b = train_head.Model(101, 48, "bf16", torch.device("cpu"), 3, "none")
    assert a.spans == b.spans and list(a.spans) == ["embed", "norm.weight", "norm.bias", "head"] and torch.equal(a.master, b.master)


def test_arguments_are_refused():
    with pytest.raises(SystemExit):
        train_head.main(["--body", "words"])
