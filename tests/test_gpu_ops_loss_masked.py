"""Tokens that the vocabulary loss leaves out: whatever their hidden states hold, the
others' losses and gradients are what they are without it, bit for bit."""
import pytest
import torch

from test_gpu_ops_loss import DEV, TYPES, check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,v,d,pad,chunk", [
    (1, 90, 64, 0, 0), (5, 300, 64, 0, 0), (31, 700, 57, 0, 0), (32, 513, 72, 1, 0), (60, 270, 64, 2, 0), (100, 500, 70, 0, 0),
    (130, 300, 67, 1, 0), (200, 513, 264, 0, 0), (301, 777, 96, 0, 64), (301, 777, 97, 0, 30), (520, 1531, 264, 6, 0)])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_what_a_token_left_out_holds_is_not_used(n, v, d, pad, chunk, kind, value):
    h, w, targets = make(n, v, d, TYPES[kind], seed=n + d, pad=pad)
    out = torch.arange(n, device=DEV) % 5 == 0
    out[n - 1] = True
    targets[out] = -100
    h[out] = 0.0
    want = run(h, w, targets, max_tokens=chunk)
    check(h, w, targets, want)
    h[out] = value
    before = h.clone()
    got = run(h, w, targets, max_tokens=chunk)
    for name, k in (("losses", 0), ("loss", 2), ("dhidden", 3), ("dweight", 4)):
        assert torch.equal(got[k], want[k]), name
    assert torch.equal(got[1][~out], want[1][~out])
    assert torch.equal(h.nan_to_num(nan=3.0), before.nan_to_num(nan=3.0))       # the caller's rows are only read
    one = torch.full((n,), -100, device=DEV)
    nothing = run(h, w, one, max_tokens=chunk)
    assert nothing[2].item() == 0 and all(torch.equal(z, torch.zeros_like(z)) for z in (nothing[0], nothing[3], nothing[4]))
