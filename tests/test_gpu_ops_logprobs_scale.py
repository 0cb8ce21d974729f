"""Gradients of the log probabilities under factors at both ends of fp32.  Tolerances are those of the operator's
tests."""
import pytest
import torch

from test_gpu_ops_logprobs import back, check_gradients, make, score

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIZES = [(3, 300), (40, 5003), (300, 1501)]


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("d,e", [(0.0, 6e37), (2.5e38, 0.0), (2e38, 3e37), (-1e38, -6e37), (1e-30, 6e37)])
def test_the_largest(n, v, d, e):
    """|d| + |e| (1 + log vocab) passes fp32; the gradients do not."""
    h, w, ids = make(n, v, 16, torch.bfloat16, seed=n)
    h.mul_(2.0 ** -3)
    w.mul_(2.0 ** -3)
    _, lse, ent, _, _ = score(h, w, ids)
    dl = torch.zeros(n, device=DEV)
    de = torch.zeros(n, device=DEV)
    dl[::2], de[::2] = d, e
    for given in (de, None) if d else (de,):
        got = back(h, w, ids, lse, ent, dl, given)
        check_gradients(h, w, ids, lse, ent, dl, given, got)
        assert all(torch.isfinite(x).all() and x.any() for x in got)


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("d", [1.2e-38, 1e-42, 3e-45])
def test_the_smallest(n, v, d):
    """Hidden states of 2^60 bring the weight's gradient into range."""
    h, w, ids = make(n, v, 16, torch.bfloat16, seed=n)
    h.mul_(2.0 ** 60)
    w.mul_(2.0 ** -60)
    _, lse, ent, _, _ = score(h, w, ids)
    dl = torch.full((n,), d, device=DEV)
    for given in (dl, None):
        got = back(h, w, ids, lse, ent, dl, given)
        check_gradients(h, w, ids, lse, ent, dl, given, got)
        assert torch.isfinite(got[1]).all() and got[1].any()


def test_no_gradient_at_all():
    h, w, ids = make(40, 500, 16, torch.float16, seed=1)
    _, lse, ent, _, _ = score(h, w, ids)
    zero = torch.zeros(40, device=DEV)
    dh, dw = back(h, w, ids, lse, ent, zero, zero)
    assert dh.eq(0).all() and dw.eq(0).all()
