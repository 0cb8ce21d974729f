"""Gradients of the log probabilities where probabilities are 0 in fp32: logits far below their row's largest, and of
-infinity.

Tolerances.  As the operator's tests': a logit is off by width * 2^-23 of its terms' absolute sum (dz) and lse, log p and
their difference by a few roundings of their sizes, so log p by `drift`; p by that relative to itself, and
an exponential below 2^-126 is 0 in fp32: an entry of G is off by another 2^-126 (|d| + |e| (|log p| + entropy)).  G is
rounded to 2 bytes once (fp16: down to steps of 2^-40 of the factor it is held with), the products are off
by their length of 2^-23, the results are rounded once."""
import math

import pytest
import torch

from test_gpu_ops_logprobs import R, TYPES, back, make, score

pytestmark = pytest.mark.gpu
DEV = "cuda"


def far(n, v, kind, seed):
    """Rows whose logits spread over some hundreds."""
    h, w, ids = make(n, v, 24, TYPES[kind], seed=seed)
    h.mul_(64.0)
    _, lse, ent, _, _ = score(h, w, ids)
    z = h.double() @ w.double().t()
    assert ((z - lse.double()[:, None]) < -120).any(1).all()
    return h, w, ids, lse, ent


SIZES = [(5, 500), (40, 501), (300, 777), (2100, 1301)]


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_they_are_the_formulas(n, v, kind):
    h, w, ids, lse, ent = far(n, v, kind, n)
    ids[: n // 2] = (h.double() @ w.double().t()).argmin(1)[: n // 2]        # ids of probability 0 among them
    dl, de = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    u = torch.finfo(h.dtype).eps / 2
    H, W, L, E, d = h.double(), w.double(), lse.double()[:, None], ent.double()[:, None], dl.double()[:, None]
    z = H @ W.t()
    lp = z - L
    p = torch.exp(lp)
    drift = 24 * 2.0 ** -23 * (H.abs() @ W.abs().t()) + 4 * R * (2 + z.abs() + L.abs())
    one = torch.zeros_like(p).scatter_(1, ids[:, None], 1.0)
    for given in (de, None):
        e = de.double()[:, None] if given is not None else torch.zeros_like(d)
        G = torch.where(one > 0, -d * torch.expm1(lp), -d * p) - e * p * (lp + E)
        off = (d.abs() * (p + one * p) * 2 + 2 * e.abs() * p * (1 + lp.abs() + E.abs())) * drift
        off = off + 4 * R * (d.abs() * p + e.abs() * p * (lp.abs() + E.abs())) + 2.0 ** -126 * (d.abs() + e.abs() * (lp.abs() + E.abs()))
        factor = 2.0 ** math.frexp((d.abs() + (1 + math.log(v)) * e.abs()).max().item())[1]
        dG = G.abs() * u + off * (1 + u) + (factor * 2.0 ** -40 if kind == "fp16" else 0.0)
        dh, dw = back(h, w, ids, lse, ent if given is not None else None, dl, given)
        low = torch.finfo(h.dtype).tiny * torch.finfo(h.dtype).eps
        for x, ref, bound in ((dh, G @ W, dG @ W.abs() + (v * 2.0 ** -23) * (G.abs() @ W.abs())),
                              (dw, G.t() @ H, dG.t() @ H.abs() + (n * 2.0 ** -23 + 2.0 ** -20) * (G.abs().t() @ H.abs()))):
            wrong = (x.double() - ref).abs() - (u * ref.abs() + bound * (1 + u) + low)
            assert (wrong <= 0).all(), wrong.max()


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [-1, None, 1 << 40])
def test_an_id_outside_gives_nan_everywhere(n, v, kind, bad):
    """Every id's entry of such a row is NaN, of whatever probability: so is all of the weight's gradient."""
    h, w, ids, lse, ent = far(n, v, kind, n + 1)
    ids[3] = v if bad is None else bad
    dl, de = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    for e in (de, None):
        dh, dw = back(h, w, ids, lse, ent if e is not None else None, dl, e)
        assert torch.isnan(dw).all() and torch.isnan(dh[3]).all()
        rest = torch.arange(n, device=DEV) != 3
        assert torch.isfinite(dh[rest]).all()


@pytest.mark.parametrize("n", [3, 300])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_a_given_token_of_minus_infinity(n, kind):
    """Its p log p is 0: the entry is d, with an entropy's gradient beside it too."""
    v = 200
    h, w, ids = torch.ones(n, 1, dtype=TYPES[kind], device=DEV), torch.randn(v, 1, device=DEV).to(TYPES[kind]), torch.full((n,), 7, device=DEV)
    w[[7, 9]] = float("-inf")
    logp, lse, ent, _, _ = score(h, w, ids)
    assert logp.eq(float("-inf")).all() and torch.isfinite(lse).all() and torch.isfinite(ent).all()
    dl, de = torch.ones(n, device=DEV), torch.full((n,), 0.5, device=DEV)
    for e in (de, None):
        _, dw = back(h, w, ids, lse, ent if e is not None else None, dl, e)
        # (n ones in 2 bytes, added in fp32: exact)
        assert dw[7].item() == n and dw[9].item() == 0 and torch.isfinite(dw).all()
