"""Alternatives of rows with NaN among their logits: those that are not NaN first, then NaN, each in the order of
ids, exactly; every place of a row is written.  Logits are sums of products on a grid, exact in fp32."""
import pytest
import torch

from test_gpu_ops_logprobs import R, make, score

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def in_order(z, top):
    """Ids by value, the lower first where they are alike, NaN behind all."""
    ids = torch.sort(z.nan_to_num(nan=-INF, posinf=INF, neginf=-INF), dim=1, descending=True, stable=True).indices
    last = torch.sort(torch.isnan(z).gather(1, ids).to(torch.uint8), dim=1, stable=True).indices
    return ids.gather(1, last)[:, :top]


def check(h, w, got, top, rows):
    _, lse, _, top_ids, top_logp = got
    z = h[rows].double() @ w.double().t()
    want = in_order(z, top)
    assert torch.equal(top_ids[rows], want)
    bad = torch.isnan(z).any(1)
    assert torch.equal(torch.isnan(lse[rows]), bad)
    assert torch.isnan(top_logp[rows][bad]).all()
    fine, taken = top_logp[rows][~bad].double(), z.gather(1, want)[~bad]
    off = (fine - (taken - lse[rows][~bad].double()[:, None])).abs()
    finite = torch.isfinite(taken)
    assert (off <= 8 * R * (1 + taken.abs() + lse[rows][~bad].double().abs()[:, None]))[finite].all()
    assert fine[~finite].eq(-INF).all()


SIZES = [(3, 300), (40, 5003), (40, 5056), (5, 70001), (5, 70016), (1100, 70001), (1100, 70016), (2100, 33001)]


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("top", [1, 5, 64])
def test_hidden_states_of_nan_beside_others(n, v, top):
    h, w, ids = make(n, v, 16, torch.bfloat16, seed=v, grid=True)
    out = torch.arange(n, device=DEV) % 3 == 1
    h[out, 5] = NAN
    rows = torch.arange(0, n, 1 if n < 100 else 50, device=DEV)
    got = score(h, w, ids, top)
    check(h, w, got, top, rows)
    assert torch.equal(got[3][out], torch.arange(top, device=DEV).expand(int(out.sum()), top))


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("top", [1, 5, 64])
@pytest.mark.parametrize("left", [0, 1, 4, 70])
def test_few_logits_that_are_not_nan(n, v, top, left):
    """Weights of NaN but for `left` rows, one of them the last; half of those give -infinity."""
    h, w, ids = make(n, v, 1, torch.bfloat16, seed=v + left, grid=True)
    h.abs_().clamp_(min=0.25)
    g = torch.Generator(device=DEV).manual_seed(top)
    keep = torch.randperm(v - 1, generator=g, device=DEV)[:max(left - 1, 0)]
    if left:
        keep = torch.cat([keep, torch.tensor([v - 1], device=DEV)])
    some = w[keep].clone()
    some[1::2] = -INF
    w.fill_(NAN)
    w[keep] = some
    check(h, w, score(h, w, ids, top), top, torch.arange(0, n, 1 if n < 100 else 50, device=DEV))


@pytest.mark.parametrize("v", [130, 5003, 5056, 70001])
@pytest.mark.parametrize("last", [-INF, NAN, 0.5])
def test_the_piece_that_ends_the_vocabulary(v, last):
    """NaN everywhere but the last row of the weight, -infinity, NaN or a number: what lies behind it in its
    piece is no alternative and ranks before none."""
    h = torch.ones(2, 1, dtype=torch.bfloat16, device=DEV)
    w = torch.full((v, 1), NAN, dtype=torch.bfloat16, device=DEV)
    w[v - 1] = last
    ids = torch.zeros(2, dtype=torch.int64, device=DEV)
    for top in (1, 2, 64):
        check(h, w, score(h, w, ids, top), top, torch.arange(2, device=DEV))


def test_what_is_written_is_this_calls():
    """Ids of a row of NaN after a call with other results in the same arrays."""
    import zero_dp_sharded_amd as zs
    n, v, top = 6, 50257, 20
    h, w, ids = make(n, v, 32, torch.bfloat16, seed=1, grid=True)
    lse = torch.empty(n, device=DEV)
    top_ids, top_logp = torch.empty(n, top, dtype=torch.int64, device=DEV), torch.empty(n, top, device=DEV)
    space = torch.empty(zs.zero_token_logprobs_workspace(n, v, 32, top=top), dtype=torch.uint8, device=DEV)
    call = lambda: zs.zero_token_logprobs(h, w, None, None, lse, None, top_ids, top_logp, space)
    call()
    before = top_ids.clone()
    h[2] = NAN
    call()
    rest = [0, 1, 3, 4, 5]
    assert torch.equal(top_ids[rest], before[rest])
    assert torch.equal(top_ids[2], torch.arange(top, device=DEV)) and torch.isnan(top_logp[2]).all()
