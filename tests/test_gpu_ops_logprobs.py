"""Log probabilities of tokens, entropy, alternatives, and their gradients on the GPU against
their definition in 64 bits, and against differences.

Tolerances, elementwise, from the inputs in 64 bits.  A logit is an fp32 sum of `width` exact
products: off by at most width * 2^-23 times the sum of their absolute values (dz).  lse is off by
dz and a few roundings, a log probability by 2 dz and a few roundings of its size.  The entropy
moves by sum p |log p + entropy| <= 2 entropy times dz; its sums of p and p (z - max) have
terms off by (1 + |z - max|) roundings each, 64 * 2^-24 of 1 + sum p (z - max)^2 with the
rest.  An entry of G is rounded to 2 bytes once (fp16: down to steps of 2^-40 of the factor it is
held with); before that it is off by what p and log p are."""
import math

import pytest
import torch

import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
R = 2.0 ** -24


def make(n, v, d, t, seed=0, pad=0, grid=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    w, ids = r(v, d) * d ** -0.5, torch.randint(0, v, (n,), generator=g, device=DEV)
    h = r(n, d) + 12.0 * (torch.arange(n, device=DEV) % 3 == 0)[:, None] * w[ids] / w[ids].norm(dim=1, keepdim=True).clamp_min(1e-6)
    if grid:                # every sum of products is exact in fp32: logits that are alike are alike
        w, h = (w * 16).round().clamp(-64, 64) / 16, (h * 4).round().clamp(-64, 64) / 4
    wide = lambda x: torch.empty(x.shape[0], d + pad, dtype=t, device=DEV)[:, :d].copy_(x)
    return wide(h), wide(w), ids


def score(h, w, ids, top=0, entropy=True, ignore=-100, max_tokens=0, stream=None):
    n = h.shape[0]
    new = lambda *s, dtype=torch.float32: torch.full(s, -7, dtype=dtype, device=DEV)
    logp, lse, ent = new(n) if ids is not None else None, new(n), new(n) if entropy else None
    top_ids, top_logp = (new(n, top, dtype=torch.int64), new(n, top)) if top else (None, None)
    space = torch.full((zs.zero_token_logprobs_workspace(n, w.shape[0], h.shape[1], top=top, max_tokens=max_tokens),), 255, dtype=torch.uint8, device=DEV)
    zs.zero_token_logprobs(h, w, ids, logp, lse, ent, top_ids, top_logp, space, ignore_index=ignore, max_tokens=max_tokens, stream=stream)
    return logp, lse, ent, top_ids, top_logp


def back(h, w, ids, lse, ent, dl, de, ignore=-100, max_tokens=0, stream=None):
    dh, dw = torch.full(h.shape, float("nan"), dtype=h.dtype, device=DEV), torch.full(w.shape, float("nan"), dtype=h.dtype, device=DEV)
    space = torch.full((zs.zero_token_logprobs_workspace(*h.shape[:1], *w.shape, gradient=True, max_tokens=max_tokens),), 255, dtype=torch.uint8, device=DEV)
    zs.zero_token_logprobs_backward(h, w, ids, lse, ent, dl, de, dh, dw, space, ignore_index=ignore, max_tokens=max_tokens, stream=stream)
    return dh, dw


def check_scores(h, w, ids, got, ignore=-100):
    logp, lse, ent, top_ids, top_logp = got
    H, W = h.double(), w.double()
    z = H @ W.t()
    dz = (h.shape[1] * 2.0 ** -23 * (H.abs() @ W.abs().t())).amax(1)
    want_lse = torch.logsumexp(z, 1)
    rough = 16 * R * (1 + want_lse.abs())
    assert ((lse.double() - want_lse).abs() <= dz + rough).all()
    lp = z - want_lse[:, None]
    if ids is not None:
        counts = ids != ignore
        want = torch.where(counts, lp.gather(1, torch.where(counts, ids, 0)[:, None])[:, 0], 0.0)
        assert ((logp.double() - want).abs() <= 2 * dz + rough + 4 * R * want.abs()).all()
        assert (logp[~counts] == 0).all()
    if ent is not None:
        p = torch.exp(lp)
        want = -(p * lp).sum(1)
        square = (p * (z - z.amax(1, keepdim=True)).square()).sum(1)
        assert ((ent.double() - want).abs() <= 2 * (1 + want) * dz + 64 * R * (1 + want + want_lse.abs() + square)).all()
    if top_ids is not None:
        k = top_ids.shape[1]
        assert ((top_ids >= 0) & (top_ids < w.shape[0])).all()
        taken = z.gather(1, top_ids)
        assert ((top_logp.double() - (taken - want_lse[:, None])).abs() <= (2 * dz + rough)[:, None] + 4 * R * taken.abs()).all()
        best = torch.sort(z, dim=1, descending=True).values[:, :k]
        assert ((taken - best).abs() <= 2 * dz[:, None]).all()
        assert (torch.sort(top_ids, 1).values.diff(dim=1) > 0).all()


def check_gradients(h, w, ids, lse, ent, dl, de, got, ignore=-100):
    t, u = h.dtype, torch.finfo(h.dtype).eps / 2
    H, W, L = h.double(), w.double(), lse.double()[:, None]
    n, v = h.shape[0], w.shape[0]
    z = H @ W.t()
    dz = h.shape[1] * 2.0 ** -23 * (H.abs() @ W.abs().t())
    counts = ids != ignore
    d = torch.where(counts, dl, 0.0).double()[:, None]
    e = (de.double() if de is not None else torch.zeros(n, dtype=torch.float64, device=DEV))[:, None]
    E = (ent.double() if ent is not None else torch.zeros(n, dtype=torch.float64, device=DEV))[:, None]
    active = ((d != 0) | (e != 0)).double()
    lp = z - L
    p = torch.exp(lp)
    one = torch.zeros_like(p).scatter_(1, torch.where(counts, ids, 0)[:, None], 1.0)
    G = torch.where(one > 0, -d * torch.expm1(lp), -d * p) - e * p * (lp + E)
    drift = dz + 4 * R * (2 + z.abs() + L.abs())            # of log p
    off = (d.abs() * (p + one * p) * 2 + 2 * e.abs() * p * (1 + lp.abs() + E.abs())) * drift + 4 * R * (d.abs() * p + e.abs() * p * (lp.abs() + E.abs()))
    reach = (d.abs() + (1 + math.log(v)) * e.abs()).max().item()
    factor = 2.0 ** math.frexp(reach)[1] if reach else 1.0
    dG = (G.abs() * u + off * (1 + u) + (factor * 2.0 ** -40 if t == torch.float16 else 0.0)) * active
    G = G * active
    # products are off by the sum's length of 2^-23; what passes through memory in parts by little more
    for x, ref, bound in ((got[0], G @ W, dG @ W.abs() + (v * 2.0 ** -23) * (G.abs() @ W.abs())),
                          (got[1], G.t() @ H, dG.t() @ H.abs() + (n * 2.0 ** -23 + 2.0 ** -20) * (G.abs().t() @ H.abs()))):
        low = torch.finfo(t).tiny * torch.finfo(t).eps
        wrong = (x.double() - ref).abs() - (u * ref.abs() + bound * (1 + u) + low)
        assert (wrong <= 0).all(), wrong.max()


SIZES = [(1, 2, 1), (1, 64, 8), (2, 65, 64), (3, 1000, 72), (17, 255, 65), (33, 257, 128), (64, 5003, 40), (129, 320, 96), (255, 513, 33),
         (256, 256, 256), (257, 700, 320), (100, 5003, 257), (520, 1531, 264), (40, 20000, 64)]


@pytest.mark.parametrize("n,v,d", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_forward(n, v, d, kind):
    h, w, ids = make(n, v, d, TYPES[kind], seed=n + v + d, pad=(n % 3) * 2)
    ids[torch.arange(n, device=DEV) % 7 == 3] = -100
    for top in (0, 1, min(v, 7)):
        check_scores(h, w, ids, score(h, w, ids, top))
    plain = score(h, w, ids, 0)
    bare = score(h, w, None, 0, entropy=False)
    assert bare[0] is None and bare[2] is None and torch.equal(bare[1], plain[1])


@pytest.mark.parametrize("n,v,d", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_backward(n, v, d, kind):
    h, w, ids = make(n, v, d, TYPES[kind], seed=n + v + d + 1, pad=(n % 3) * 2)
    ids[torch.arange(n, device=DEV) % 7 == 3] = -100
    _, lse, ent, _, _ = score(h, w, ids)
    g = torch.Generator(device=DEV).manual_seed(n)
    scale = 512.0 if kind == "fp16" else 1.0
    dl = torch.randn(n, generator=g, device=DEV) * scale
    de = torch.randn(n, generator=g, device=DEV) * scale
    de[torch.arange(n, device=DEV) % 5 == 1] = 0
    dl[torch.arange(n, device=DEV) % 4 == 2] = 0
    for e in (de, None):
        check_gradients(h, w, ids, lse, ent, dl, e, back(h, w, ids, lse, ent if e is not None else None, dl, e))


@pytest.mark.parametrize("n,v,d,top", [(1, 64, 16, 64), (3, 70, 8, 64), (5, 200, 24, 64), (40, 1000, 16, 20), (300, 777, 32, 33), (2, 140003, 16, 20),
                                       (150, 70001, 24, 5)])
def test_alternatives_in_order(n, v, d, top):
    """Logits on a grid: exactly the stable order, with many that are alike."""
    h, w, ids = make(n, v, d, torch.bfloat16, seed=v, grid=True)
    h[0] = 0                                       # a row of equal logits
    z = h.double() @ w.double().t()
    want = torch.sort(z, dim=1, descending=True, stable=True)
    _, lse, _, top_ids, top_logp = score(h, w, ids, top)
    assert torch.equal(top_ids, want.indices[:, :top])
    assert ((top_logp.double() - (want.values[:, :top] - lse.double()[:, None])).abs() <= 8 * R * (1 + want.values[:, :top].abs() + lse.double().abs()[:, None])).all()


def test_alternatives_among_what_is_not_finite():
    h = torch.zeros(4, 8, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(300, 8, dtype=torch.bfloat16, device=DEV)
    h[0, 0], h[1, 1], h[2, 2], h[3, 3] = 1, 1, 1, 1
    w[:, 0] = float("-inf")                        # row 0: nothing is possible
    w[:, 1] = float("-inf")
    w[[5, 250], 1] = 1.0                           # row 1: two are
    w[7, 2] = -0.0
    w[9, 2] = 0.0                                  # row 2: all alike, of either sign
    h2 = h.clone()
    # (0 * inf is NaN: rows of one factor each, by products that are 0 only for zeros)
    for r, want in ((0, [0, 1, 2, 3, 4]), (1, [5, 250, 0, 1, 2]), (2, [0, 1, 2, 3, 4])):
        only = w[:, r:r + 1].expand(300, 1).contiguous()
        one = torch.ones(1, 1, dtype=torch.bfloat16, device=DEV)
        ids = torch.tensor([5], device=DEV)
        logp, lse, ent, top_ids, top_logp = score(one, only, ids, 5)
        assert top_ids[0].tolist() == want, r
        if r == 0:
            assert lse.item() == float("-inf") and torch.isnan(logp).all() and torch.isnan(ent).all()
        if r == 1:
            assert abs(logp.item() + math.log(2)) < 1e-6 and abs(ent.item() - math.log(2)) < 1e-6
            assert top_logp[0, 2:].eq(float("-inf")).all()
        if r == 2:
            assert abs(ent.item() - math.log(300)) < 1e-5
    bad = torch.ones(3, 300, dtype=torch.bfloat16, device=DEV).t().contiguous()
    bad[17, 0], bad[40, 1] = float("nan"), float("inf")
    h3 = torch.eye(3, dtype=torch.bfloat16, device=DEV)
    # a NaN logit: the row's numbers are NaN, its alternatives the others; ids stay in range
    logp, lse, ent, top_ids, _ = score(h3[:1, :1].contiguous(), bad[:, :1].contiguous(), torch.tensor([1], device=DEV), 64)
    assert torch.isnan(lse).all() and top_ids[0].tolist() == [k for k in range(65) if k != 17]
    logp, lse, ent, top_ids, _ = score(h3[:1, :1].contiguous(), bad[:, 1:2].contiguous(), torch.tensor([1], device=DEV), 3)
    assert torch.isnan(lse).all() and top_ids[0].tolist() == [40, 0, 1]
    assert h2.equal(h)


def test_gradients_against_differences():
    n, v, d = 4, 23, 8
    h, w, ids = make(n, v, d, torch.bfloat16, seed=3)
    ids[2] = -100
    _, lse, ent, _, _ = score(h, w, ids)
    g = torch.Generator(device=DEV).manual_seed(1)
    dl, de = torch.randn(n, generator=g, device=DEV), torch.randn(n, generator=g, device=DEV)
    dh, dw = back(h, w, ids, lse, ent, dl, de)

    def value(h, w):
        lp = torch.log_softmax(h @ w.t(), 1)
        own = torch.where(ids >= 0, lp.gather(1, ids.clamp_min(0)[:, None])[:, 0], 0.0)
        return (dl.double() * own).sum() - (de.double() * (torch.exp(lp) * lp).sum(1)).sum()

    at, step = [h.double(), w.double()], 1e-6
    for k, got in enumerate((dh, dw)):
        for j in range(0, got.numel(), 3):
            ends = []
            for sign in (1, -1):
                moved = [z.clone() for z in at]
                moved[k].view(-1)[j] += sign * step
                ends.append(value(*moved))
            diff = ((ends[0] - ends[1]) / (2 * step)).item()
            # (G in pairs of bf16: the result's own rounding, and fp32's errors)
            assert abs(got.reshape(-1)[j].item() - diff) <= 2.0 ** -8 * abs(diff) + 1e-4, (k, j)


def test_rows_without_gradients_enter_nothing():
    n, v, d = 200, 500, 48
    h, w, ids = make(n, v, d, torch.bfloat16, seed=5)
    out = torch.arange(n, device=DEV) % 4 == 1
    ids[out] = -100
    clean = h.clone()
    clean[out] = 0
    _, lse, ent, _, _ = score(clean, w, ids)
    dl, de = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    de[out] = 0
    want = back(clean, w, ids, lse, ent, dl, de)
    h[out] = float("nan")
    h[5] = float("inf") if bool(out[5]) else h[5]
    lse[out], ent[out], dl[out] = float("nan"), float("nan"), float("nan")
    got = back(h, w, ids, lse, ent, dl, de)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and not got[0][out].any()
    ids[3] = v
    dh, dw = back(h, w, ids, lse, ent, dl, de)
    assert torch.isnan(dh[3]).all() and torch.isnan(dw).any() and torch.isfinite(dh[0]).all()
    logp = score(clean, w, ids)[0]
    assert torch.isnan(logp[3]) and torch.isfinite(logp[:3]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_chunks_of_tokens(kind):
    n, v, d = 700, 900, 72
    h, w, ids = make(n, v, d, TYPES[kind], seed=8)
    whole, parts = score(h, w, ids, 4), score(h, w, ids, 4, max_tokens=256)
    check_scores(h, w, ids, parts)
    assert torch.equal(whole[3], parts[3])
    lse, ent = whole[1], whole[2]
    g = torch.Generator(device=DEV).manual_seed(2)
    dl, de = torch.randn(n, generator=g, device=DEV), torch.randn(n, generator=g, device=DEV)
    for most in (0, 256, 100):
        check_gradients(h, w, ids, lse, ent, dl, de, back(h, w, ids, lse, ent, dl, de, max_tokens=most))


def test_no_tokens():
    h, w, ids = make(1, 50, 16, torch.bfloat16)
    empty = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    none, no_ids = torch.empty(0, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    zs.zero_token_logprobs(empty, w, no_ids, none, none.clone(), workspace=torch.empty(1 << 16, dtype=torch.uint8, device=DEV))
    dh, dw = back(empty, w, no_ids, none, none, none, none)
    assert dw.shape == w.shape and not dw.any()


@pytest.mark.parametrize("d,shift", [(64, 1), (65, 0), (67, 1), (130, 0)])
def test_operands_that_cannot_be_loaded_as_they_lie(d, shift):
    n, v = 150, 333
    h, w, ids = make(n, v, d, torch.float16, seed=d)
    at = lambda x: torch.empty(x.numel() + shift, dtype=x.dtype, device=DEV)[shift:].view(x.shape).copy_(x)
    a, b = score(h, w, ids, 3), score(at(h), at(w), ids, 3)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    dl, de = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    p, q = back(h, w, ids, a[1], a[2], dl, de), back(at(h), at(w), ids, a[1], a[2], dl, de)
    assert all(torch.equal(x, y) for x, y in zip(p, q))


@pytest.mark.parametrize("n", [12, 300])
def test_same_bits_streams_and_graphs(n):
    v, d, top = 3001, 120, 6
    h, w, ids = make(n, v, d, torch.bfloat16, seed=n)
    outs = [torch.empty(n, device=DEV) for _ in range(3)]
    top_ids, top_logp = torch.empty(n, top, dtype=torch.int64, device=DEV), torch.empty(n, top, device=DEV)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    dl, de = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    space = [torch.empty(zs.zero_token_logprobs_workspace(n, v, d, top=top, gradient=g), dtype=torch.uint8, device=DEV) for g in (False, True)]
    every = [*outs, top_ids, top_logp, dh, dw]

    def both(stream=None):
        zs.zero_token_logprobs(h, w, ids, outs[0], outs[1], outs[2], top_ids, top_logp, space[0], stream=stream)
        zs.zero_token_logprobs_backward(h, w, ids, outs[1], outs[2], dl, de, dh, dw, space[1], stream=stream)

    both()
    torch.cuda.synchronize()
    first = [x.clone() for x in every]
    s = torch.cuda.Stream()
    for x in every:
        x.zero_()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, every))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for k in range(3):
        for x in every:
            x.zero_()
        h.mul_(0.9)
        dl.mul_(2.0)
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in every]
        both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, every)), k


@pytest.mark.parametrize("n,v,d", [(2100, 33001, 136), (8200, 5001, 72), (1100, 90007, 40)])
def test_large_tiles(n, v, d):
    """Walks over tiles, logits past the last cache, more pieces than a wave keeps, chunks."""
    h, w, ids = make(n, v, d, torch.bfloat16, seed=n)
    got = score(h, w, ids, 5)
    part = slice(0, n, 97)
    check_scores(h[part], w, ids[part], [x[part] for x in got])
    rest = score(h, w, ids, 0)                     # (other tiles)
    check_scores(h[part], w, ids[part], [x[part] if x is not None else None for x in rest])
    dl, de = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    dl[n // 2:] = 0
    de[n // 3:] = 0
    dh, dw = back(h, w, ids, got[1], got[2], dl, de)
    assert not dh[n // 2:].any()
    few = slice(0, n // 2)
    check_gradients(h[few], w, ids[few], got[1][few], got[2][few], dl[few], de[few], (dh[few], dw))


def test_refusals():
    h, w, ids = make(5, 50, 16, torch.bfloat16)
    lse, logp = torch.empty(5, device=DEV), torch.empty(5, device=DEV)
    space = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    with pytest.raises(zs.ZeroError, match="both or neither"):
        zs.zero_token_logprobs(h, w, ids, None, lse, workspace=space)
    with pytest.raises(ValueError, match="shape"):
        zs.zero_token_logprobs(h, w, ids, logp, lse, None, torch.empty(5, 3, dtype=torch.int64, device=DEV), torch.empty(5, 2, device=DEV), space)
    with pytest.raises(zs.ZeroError, match="top"):
        zs.zero_token_logprobs(h, w, ids, logp, lse, None, torch.empty(5, 51, dtype=torch.int64, device=DEV), torch.empty(5, 51, device=DEV), space)
    with pytest.raises(zs.ZeroError, match="workspace"):
        zs.zero_token_logprobs(h, w, ids, logp, lse)
