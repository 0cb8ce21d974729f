"""The vocabulary loss and its gradients on the GPU against their definition in 64
bits, and against differences of the loss.

Tolerances, elementwise, from the inputs in 64 bits.  A logit is an fp32 sum of
`width` exact products: off by at most width * 2^-23 times the sum of their absolute
values (dz; twice the step of rounding to nearest, since the matrix cores' adders
may truncate).  The loss is off by 2 max(dz) and a few roundings of its size.  An
entry of G is exp of a difference of logits, rounded to 2 bytes at most twice:
off by 2 half steps (2^-8 each for bf16, 2^-11 for fp16) and 4 dz of itself; the target's,
p - 1, by a half step and 4 dz.  fp16 holds 2^15 G down to steps of 2^-24: 2^-39.
The products add vocab or tokens terms in fp32, and the result is rounded once."""
import pytest
import torch

import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def make(n, v, d, t, seed=0, lean=12.0, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    w = torch.empty(v, d + pad, dtype=t, device=DEV)[:, :d]
    w.copy_(r(v, d) * d ** -0.5)
    targets = torch.randint(0, v, (n,), generator=g, device=DEV)
    h = torch.empty(n, d + pad, dtype=t, device=DEV)[:, :d]
    row = w[targets].float()
    h.copy_(r(n, d) + lean * (torch.arange(n, device=DEV) % 3 == 0)[:, None] * row / row.norm(dim=1, keepdim=True).clamp_min(1e-6))
    return h, w, targets


def run(h, w, targets, grad=True, scale=1.0, ignore=-100, max_tokens=0, stream=None, fill=float("nan")):
    n, d = h.shape
    losses, lse, loss = (torch.full(s, fill, device=DEV) for s in ((n,), (n,), ()))
    dh, dw = (torch.full(tuple(z.shape), fill, dtype=h.dtype, device=DEV) if grad else None for z in (h, w))
    space = torch.full((zs.zero_vocab_loss_workspace(n, w.shape[0], d, gradient=grad, max_tokens=max_tokens),), 255,
                       dtype=torch.uint8, device=DEV)
    zs.zero_vocab_loss(h, w, targets, losses, lse, loss, dh, dw, space, grad_scale=scale, ignore_index=ignore,
                       max_tokens=max_tokens, stream=stream)
    return losses, lse, loss, dh, dw


def check(h, w, targets, got, scale=1.0, ignore=-100):
    losses, lse, loss, dh, dw = got
    t = h.dtype
    n, d = h.shape
    H, W = h.double(), w.double()
    z = H @ W.t()
    dz = d * 2.0 ** -23 * (H.abs() @ W.abs().t())
    counts = targets != ignore
    many = max(1, int(counts.sum()))
    at = torch.where(counts, targets, 0)[:, None]
    want_lse = torch.logsumexp(z, 1)
    want = torch.where(counts, want_lse - z.gather(1, at)[:, 0], 0.0)
    tol = 2 * dz.max(1).values + 16 * 2.0 ** -24 * (1 + want_lse.abs() + z.gather(1, at)[:, 0].abs())
    assert ((lse.double() - want_lse).abs() <= tol).all()
    assert ((losses.double() - want).abs() <= tol).all()
    assert (losses[~counts] == 0).all()
    assert abs(loss.item() - want.sum().item() / many) <= tol.max().item()
    if dh is None:
        return
    u = torch.finfo(t).eps / 2
    p = torch.exp(z - want_lse[:, None]) * counts[:, None]
    one = torch.zeros_like(p).scatter_(1, at, 1.0) * counts[:, None]
    # p - 1 of the target from the others, which does not cancel
    G = p * (1 - one)
    G = G - one * G.sum(1, keepdim=True)
    drift = 4 * (dz.max(1).values + 16 * 2.0 ** -24 * (1 + want_lse.abs()))[:, None]
    dG = G.abs() * 2 * u * (1 + u) + (p * (1 - one) + one * p) * drift + (2.0 ** -39 if t == torch.float16 else 0.0)
    k = scale / many
    for got_g, ref, off, terms in ((dh, G @ W, dG @ W.abs(), G.abs() @ W.abs() * (w.shape[0] * 2.0 ** -23)),
                                   (dw, G.t() @ H, dG.t() @ H.abs(), G.abs().t() @ H.abs() * (n * 2.0 ** -23 + 2.0 ** -20))):
        ref, off = ref * k, (off + terms) * abs(k)
        fine = torch.finfo(t)
        low = fine.tiny * fine.eps           # the smallest number of the type
        assert ((got_g.double() - ref).abs() <= u * ref.abs() + off * (1 + u) + low).all(), ((got_g.double() - ref).abs() - (u * ref.abs() + off)).max()


SIZES = [(1, 2, 1), (1, 64, 8), (2, 65, 64), (3, 1000, 72), (17, 255, 65), (64, 257, 128), (255, 513, 33), (256, 256, 256),
         (257, 700, 320), (100, 5003, 257), (520, 1531, 264), (40, 20000, 64)]


@pytest.mark.parametrize("n,v,d", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_against_the_definition(n, v, d, kind):
    h, w, targets = make(n, v, d, TYPES[kind], seed=n + v + d)
    targets[torch.arange(n, device=DEV) % 7 == 3] = -100
    scale = 4096.0 if kind == "fp16" else 1.0
    check(h, w, targets, run(h, w, targets, scale=scale), scale=scale)
    alone = run(h, w, targets, grad=False)
    check(h, w, targets, alone)


@pytest.mark.parametrize("chunk", [1, 3, 64, 100, 300, 301, 8192])
def test_chunks_of_tokens(chunk):
    h, w, targets = make(301, 777, 96, torch.bfloat16, seed=9)
    targets[5] = targets[300] = -100
    check(h, w, targets, run(h, w, targets, max_tokens=chunk))


def test_gradient_against_differences():
    """The gradients of the mean loss by central differences in 64 bits."""
    n, v, d = 9, 50, 24
    h, w, targets = make(n, v, d, torch.float16, seed=2, lean=4.0)
    targets[4] = -100
    _, _, _, dh, dw = run(h, w, targets, scale=8.0)

    def value(H, W):
        z = H @ W.t()
        keep = targets != -100
        return 8.0 * (torch.logsumexp(z, 1) - z.gather(1, targets.clamp_min(0)[:, None])[:, 0])[keep].mean()

    at, step = [h.double(), w.double()], 1e-5
    for k, got in enumerate((dh, dw)):
        scale = got.double().abs().max().item()
        for j in range(0, got.numel(), 37):
            ends = []
            for sign in (1, -1):
                moved = [z.clone() for z in at]
                moved[k].view(-1)[j] += sign * step
                ends.append(value(*moved))
            diff = ((ends[0] - ends[1]) / (2 * step)).item()
            # three roundings of 2^-11 of terms that are at most the largest gradient
            assert abs(got.view(-1)[j].item() - diff) <= 3 * 2.0 ** -11 * scale + 1e-9, (k, j)


def test_strides_and_addresses():
    h, w, targets = make(70, 300, 64, torch.bfloat16, seed=3)
    want = run(h, w, targets)
    # odd strides, an address off by one element: copied first, the same results
    for off in (1, 4, 8):
        hb = torch.zeros(70 * 75 + 8, dtype=torch.bfloat16, device=DEV)[off:off + 70 * 75].view(70, 75)[:, :64]
        wb = torch.zeros(300 * 67 + 8, dtype=torch.bfloat16, device=DEV)[off:off + 300 * 67].view(300, 67)[:, :64]
        hb.copy_(h)
        wb.copy_(w)
        dhb = torch.zeros(70, 71, dtype=torch.bfloat16, device=DEV)
        dwb = torch.zeros(300, 65, dtype=torch.bfloat16, device=DEV)
        losses, loss = torch.empty(70, device=DEV), torch.empty(1, device=DEV)
        space = torch.empty(zs.zero_vocab_loss_workspace(70, 300, 64), dtype=torch.uint8, device=DEV)
        zs.zero_vocab_loss(hb, wb, targets, losses, None, loss, dhb[:, 3:67], dwb[:, 1:], space)
        assert torch.equal(losses, want[0]) and torch.equal(loss[0], want[2])
        assert torch.equal(dhb[:, 3:67], want[3]) and torch.equal(dwb[:, 1:], want[4])
        assert not dhb[:, :3].any() and not dhb[:, 67:].any() and not dwb[:, 0].any()


@pytest.mark.parametrize("n,v,d,pad", [(50, 333, 70, 0), (5, 700, 1380, 0), (130, 300, 67, 1), (9, 129, 1, 1), (200, 513, 66, 4),
                                       (60, 270, 64, 2), (140, 700, 328, 6), (17, 99, 8, 10), (300, 90, 258, 0), (1000, 100, 40, 0),
                                       (2115, 788, 256, 0)])
def test_what_lies_between_rows_and_behind_them_is_not_used(n, v, d, pad):
    """NaN between the rows and behind the last, at widths that are a multiple of 8 and
    that are none; and products of few tiles and long depth, which go in parts."""
    h, w, targets = make(n, v, d, torch.bfloat16, seed=n + d)
    big = [torch.full((rows + 1, d + pad), float("nan"), dtype=torch.bfloat16, device=DEV)[:rows, :d] for rows in (n, v)]
    big[0].copy_(h)
    big[1].copy_(w)
    targets[n // 2] = -100
    check(big[0], big[1], targets, run(big[0], big[1], targets))


def test_ignored_unknown_and_no_tokens():
    h, w, targets = make(30, 90, 64, torch.float16, seed=6)
    # none counts: loss 0, gradients 0, whatever the logits
    h[3, 5] = float("inf")
    losses, lse, loss, dh, dw = run(h, w, torch.full_like(targets, -1), ignore=-1)
    assert loss.item() == 0 and not losses.any()
    assert not dh.any() and not torch.isnan(dh).any()
    h[3, 5] = 1.0
    # an ignored token with logits that are not finite leaves the others as they are
    a = run(h, w, targets.clone().index_fill_(0, torch.tensor([3], device=DEV), -100))
    assert torch.isfinite(a[3]).all() and torch.isfinite(a[4]).all() and not a[3][3].any()
    # a target that is not an id: NaN, where it is
    for bad in (90, -5, 1 << 40):
        t = targets.clone()
        t[7] = bad
        losses, lse, loss, dh, dw = run(h, w, t)
        assert torch.isnan(losses[7]) and torch.isnan(loss) and torch.isnan(dh[7]).all() and torch.isnan(dw).any()
        rest = [k for k in range(30) if k != 7]
        assert torch.isfinite(losses[rest]).all() and torch.isfinite(dh[rest]).all() and torch.isfinite(lse).all()
    # no tokens
    losses, lse, loss, dh, dw = run(h[:0], w, targets[:0])
    assert loss.item() == 0 and not dw.any() and not torch.isnan(dw).any()
    assert run(h[:0], w, targets[:0], grad=False)[2].item() == 0


def test_large_logits_and_what_is_not_finite():
    n, v, d = 12, 300, 64
    h, w, targets = make(n, v, d, torch.bfloat16, seed=8)
    h *= 300.0                     # logits of some hundreds: exp of the logits themselves would overflow
    got = run(h, w, targets)
    check(h, w, targets, got)
    w[250] = float("-inf") * torch.sign(h[0].float()).to(w.dtype)      # token 0's logit of id 250: -infinity
    targets[0] = 3
    one = run(h[:1], w, targets[:1], grad=False)
    z = torch.where(torch.arange(v, device=DEV) == 250, float("-inf"), (h[:1].double() @ torch.where(torch.isinf(w), 0, w).double().t())[0])
    assert abs(one[1].item() - torch.logsumexp(z, 0).item()) <= 1e-3 * max(1, abs(z.max().item()))
    h2, w2, t2 = make(5, 100, 64, torch.bfloat16, seed=9)
    h2[2, 1] = float("nan")
    losses, lse, loss, dh, dw = run(h2, w2, t2)
    assert torch.isnan(losses[2]) and torch.isfinite(losses[[0, 1, 3, 4]]).all() and torch.isnan(loss)
    assert torch.isnan(dh[2]).all() and torch.isfinite(dh[[0, 1, 3, 4]]).all()


def test_confident_tokens_keep_their_gradient():
    """p - 1 of a target with p within 1e-4 of 1 is small, and still has its 8 bits."""
    n, v, d = 32, 500, 128
    h, w, targets = make(n, v, d, torch.bfloat16, seed=11, lean=0.0)
    row = w[targets].float()
    h.copy_(15.0 * row / row.square().sum(1, keepdim=True))
    got = run(h, w, targets)
    check(h, w, targets, got)
    assert (got[0] < 1e-2).all()


def test_same_bits_other_streams_and_graphs():
    h, w, targets = make(300, 3001, 200, torch.bfloat16, seed=12)
    first = run(h, w, targets)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n, d = h.shape
    outs = [torch.empty(n, device=DEV), torch.empty(n, device=DEV), torch.empty((), device=DEV), torch.empty_like(h),
            torch.empty_like(w)]
    space = torch.empty(zs.zero_vocab_loss_workspace(n, 3001, d), dtype=torch.uint8, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    zs.zero_vocab_loss(h, w, targets, *outs, space, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zs.zero_vocab_loss(h, w, targets, *outs, space)
    for k in range(4):
        h.mul_(0.9)
        targets[k] = -100
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(run(h, w, targets), outs)), k


def test_types_are_refused():
    h, w, targets = make(4, 10, 8, torch.bfloat16)
    out = torch.empty(4, device=DEV)
    space = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    with pytest.raises(zs.ZeroError, match="2-byte"):
        zs.zero_vocab_loss(h.float(), w.float(), targets, out, None, out[:1].clone(), workspace=space)
    with pytest.raises(TypeError):
        zs.zero_vocab_loss(h, w.half(), targets, out, None, out[:1].clone(), workspace=space)
    with pytest.raises(TypeError):
        zs.zero_vocab_loss(h, w, targets.int(), out, None, out[:1].clone(), workspace=space)
    with pytest.raises(zs.ZeroError, match="both or neither"):
        zs.zero_vocab_loss(h, w, targets, out, None, out[:1].clone(), dweight=w.clone(), workspace=space)
    with pytest.raises(zs.ZeroError, match="workspace"):
        zs.zero_vocab_loss(h, w, targets, out, None, out[:1].clone(), workspace=space[:256])


@pytest.mark.parametrize("n,v,d,t", [(1, 3644, 160, "bf16"), (1, 2271, 57, "fp16"), (4, 1003, 57, "fp16"), (5, 900, 64, "bf16"),
                                     (9, 3001, 200, "fp16"), (31, 513, 96, "bf16"), (32, 777, 41, "fp16")])
def test_few_tokens_lose_nothing_to_the_held_gradient(n, v, d, t):
    """Up to 32 tokens an entry of G is held in two numbers, so a gradient is off by its
    own rounding (u) and, relative to the sum of its terms' magnitudes, by: the two numbers'
    u^2, twice; 2 dz of a logit and of lse; the exponent's argument, below 2^6, rounded to
    fp32 and some roundings beside (2^-16 in all); the fp32 sums (as in check).  A step of
    fp16's smallest numbers under 2^15 is 2^-39 of G, and there are two of them."""
    t = TYPES[t]
    h, w, targets = make(n, v, d, t, seed=n + v, lean=6.0)
    _, _, _, dh, dw = run(h, w, targets, scale=64.0)
    H, W = h.double().cpu(), w.double().cpu()
    z = H @ W.t()
    p = torch.softmax(z, 1)
    one = torch.nn.functional.one_hot(targets.cpu(), v).double()
    G = p * (1 - one)
    G = G - one * G.sum(1, keepdim=True)
    dz = (d * 2.0 ** -23 * (H.abs() @ W.abs().t())).max(1, keepdim=True).values
    u = torch.finfo(t).eps / 2
    dG = G.abs() * 2 * u * u * (1 + u) + p * (4 * dz + 2.0 ** -16) + one * 2.0 ** -22 + 2.0 ** -38
    low = torch.finfo(t).tiny * torch.finfo(t).eps
    for got, ref, off in ((dh, G @ W, dG @ W.abs() + G.abs() @ W.abs() * (v * 2.0 ** -23)),
                          (dw, G.t() @ H, dG.t() @ H.abs() + G.abs().t() @ H.abs() * (2 * n * 2.0 ** -23 + 2.0 ** -20))):
        ref, off = ref * (64.0 / n), off * (64.0 / n)
        assert ((got.double().cpu() - ref).abs() <= u * ref.abs() + off * (1 + u) + low).all()
