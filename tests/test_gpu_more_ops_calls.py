"""Calls of the scaled product and the log probabilities that a program may make and that their own tests do not: all
logits alike, alternatives alone, an ignored id of the vocabulary, an array as both operands, two calls at
once, the smallest sizes, results among rows that are another's.  Tolerances are those of the operators' tests."""
import math

import pytest
import torch

import zero_dp_sharded_amd as zs
from test_gpu_ops_logprobs import back, make, score
from test_gpu_ops_product import check, packed, reference, space

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("n,v,top", [(5, 50257, 64), (300, 5003, 64), (2100, 33001, 5), (1030, 70001, 64)])
def test_all_logits_alike(n, v, top):
    h = torch.randn(n, 24, device=DEV).bfloat16()
    w = torch.zeros(v, 24, dtype=torch.bfloat16, device=DEV)
    ids = torch.randint(0, v, (n,), device=DEV)
    logp, lse, ent, top_ids, top_logp = score(h, w, ids, top)
    assert torch.equal(top_ids, torch.arange(top, device=DEV).expand(n, top))
    # (a sum of up to 70001 ones in fp32 pieces of 64 and in 64 bits over them: exact; then the logarithm's rounding)
    for x, want in ((logp, -math.log(v)), (lse, math.log(v)), (ent, math.log(v)), (top_logp, -math.log(v))):
        assert (x.double() - want).abs().max().item() <= 2 * 2.0 ** -24 * math.log(v)


@pytest.mark.parametrize("n", [7, 300])
def test_alternatives_alone_are_those_beside_log_probabilities(n):
    h, w, ids = make(n, 2001, 64, torch.bfloat16, seed=n)
    logp, lse, ent, top_ids, top_logp = score(h, w, ids, 9)
    none, lse2, no_entropy, ids2, logp2 = score(h, w, None, 9, entropy=False)
    assert none is None and no_entropy is None
    assert torch.equal(lse, lse2) and torch.equal(top_ids, ids2) and torch.equal(top_logp, logp2)


@pytest.mark.parametrize("n", [20, 300])
def test_an_ignored_id_of_the_vocabulary_and_the_same_id_twice(n):
    v, d = 777, 48
    h, w, ids = make(n, v, d, torch.float16, seed=3)
    ids[: n // 2] = 5
    ids[n // 2:] = 11
    logp, lse, ent, _, _ = score(h, w, ids, ignore=5)
    plain = score(h, w, ids)
    assert logp[: n // 2].eq(0).all() and torch.equal(logp[n // 2:], plain[0][n // 2:])
    assert torch.equal(lse, plain[1]) and torch.equal(ent, plain[2])
    dl = torch.randn(n, device=DEV)
    dh, dw = back(h, w, ids, lse, None, dl, None, ignore=5)
    zeroed = dl.clone()
    zeroed[: n // 2] = 0
    dh2, dw2 = back(h, w, ids, lse, None, zeroed, None)
    assert dh[: n // 2].eq(0).all() and torch.equal(dh, dh2) and torch.equal(dw, dw2)


def test_one_of_one():
    for n in (1, 200):
        h, w = torch.ones(n, 1, device=DEV).bfloat16(), torch.full((1, 1), 3.0, device=DEV).bfloat16()
        ids = torch.zeros(n, dtype=torch.int64, device=DEV)
        logp, lse, ent, top_ids, top_logp = score(h, w, ids, 1)
        assert logp.eq(0).all() and lse.eq(3).all() and ent.eq(0).all() and top_ids.eq(0).all() and top_logp.eq(0).all()
        dh, dw = back(h, w, ids, lse, ent, torch.ones(n, device=DEV), torch.ones(n, device=DEV))
        assert dh.eq(0).all() and dw.eq(0).all()


@pytest.mark.parametrize("n", [9, 260])
def test_gradients_among_others_columns(n):
    v, d = 501, 40
    h, w, ids = make(n, v, d, torch.bfloat16, seed=1)
    _, lse, ent, _, _ = score(h, w, ids)
    dl, de = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    want = back(h, w, ids, lse, ent, dl, de)
    whole = [torch.full((rows, d + 9), 7.0, dtype=h.dtype, device=DEV) for rows in (n, v)]
    parts = [x[:, 4:4 + d] for x in whole]
    ws = torch.empty(zs.zero_token_logprobs_workspace(n, v, d, gradient=True), dtype=torch.uint8, device=DEV)
    zs.zero_token_logprobs_backward(h, w, ids, lse, ent, dl, de, *parts, ws)
    for x, part, y in zip(whole, parts, want):
        assert torch.equal(part, y)
        assert x[:, :4].eq(7).all() and x[:, 4 + d:].eq(7).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(300, 300, 1), (300, 257, 15), (513, 300, 128), (300, 70, 129), (1200, 500, 257)])
def test_short_depths_of_many_rows(m, n, k, kind):
    a, ae = packed(m, k, False, 1, pad=1)
    b, be = packed(n, k, False, 2, pad=2)
    whole = torch.full((m + 2, n + 3), 7.0, dtype=kind, device=DEV)
    out = whole[1:-1, 1:-2]
    zs.zero_scaled_product(a, ae, b, be, out, None, space(m, n, k))
    want, off = reference(a, ae, b, be, kind)
    check(out, want, off)
    assert whole[0].eq(7).all() and whole[-1].eq(7).all() and whole[:, 0].eq(7).all() and whole[:, -2:].eq(7).all()


@pytest.mark.parametrize("kind", [torch.float16, torch.float32])
@pytest.mark.parametrize("n", [20, 600])
def test_an_array_by_itself(n, kind):
    a, ae = packed(n, 700, False, 5)
    out = torch.empty(n, n, dtype=kind, device=DEV)
    zs.zero_scaled_product(a, ae, a, ae, out, None, space(n, n, 700))
    want, off = reference(a, ae, a, ae, kind)
    # (the diagonal's sums of squares pass fp16's 65504: what is not below it by what the sum may be off by is
    # infinite, or within twice that of it)
    top = torch.finfo(kind).max
    past = want + off >= top
    assert (out[past].double() >= top - 2 * off[past]).all()
    check(out.masked_fill(past, 0.0), want.masked_fill(past, 0.0), off)
    assert (past & ~torch.eye(n, dtype=torch.bool, device=DEV)).sum() == 0


def test_products_in_fp32_captured():
    for m, n, k in ((1200, 700, 4099), (30, 700, 1601), (4801, 1601, 500)):
        a, ae = packed(m, k, False, 1)
        b, be = packed(n, k, False, 2)
        out, ws = torch.empty(m, n, device=DEV), space(m, n, k)
        zs.zero_scaled_product(a, ae, b, be, out, None, ws)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            zs.zero_scaled_product(a, ae, b, be, out, None, ws)
        for _ in range(3):
            be.sub_(1)
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            got = out.clone()
            zs.zero_scaled_product(a, ae, b, be, out, None, ws)
            assert torch.equal(got, out)


def test_two_calls_at_once():
    m, n, k, v = 1100, 1500, 2000, 3001
    a, ae = packed(m, k, False, 1)
    b, be = packed(n, k, True, 2)
    h, w, ids = make(m, v, 96, torch.bfloat16, seed=2)
    size = zs.zero_token_logprobs_workspace(m, v, 96, top=4)

    def results():
        return ([torch.zeros(m, n, dtype=t, device=DEV) for t in (torch.bfloat16, torch.float32)]
                + [torch.zeros(m, device=DEV) for _ in range(3)] + [torch.zeros(m, 4, dtype=torch.int64, device=DEV), torch.zeros(m, 4, device=DEV)])

    def calls(r, spaces, stream):
        for _ in range(3):
            zs.zero_scaled_product(a, ae, b, be, r[0], None, spaces[0], stream=stream)
            zs.zero_token_logprobs(h, w, ids, r[2], r[3], r[4], r[5], r[6], spaces[1], stream=stream)
            zs.zero_scaled_product(a, ae, b, be, r[1], None, spaces[0], stream=stream)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [(space(m, n, k), torch.empty(size, dtype=torch.uint8, device=DEV)) for _ in range(3)]
    want, got = results(), [results(), results()]
    calls(want, spaces[2], torch.cuda.current_stream())
    torch.cuda.synchronize()
    for s, r, p in zip(streams, got, spaces):
        calls(r, p, s)
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(x, y) for x, y in zip(r, want))
