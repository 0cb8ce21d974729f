"""The vocabulary loss at sizes that take its large tiles: several tiles a workgroup one
after the other (the next one's loads under way), tiles of 256 x 320, products in parts and
whole, chunks of tokens, and exponentials past the last cache.  Which of them a size
takes is asserted without a GPU in test_ops_plan_cpu.py.  Definition, tolerances and their
derivation: test_gpu_ops_loss.py."""
import pytest
import torch

import zero_dp_sharded_amd as zs
from test_gpu_ops_loss import DEV, TYPES, check, make, run

pytestmark = pytest.mark.gpu

# tokens, vocab, width, max_tokens: (rows of 32 by columns of 64 of the logits' tile, several
# tiles a workgroup; the same of the hidden states' gradient, in parts; of the weight's, in
# parts; exponentials past the last cache)
CASES = {
    (1029, 22001, 1600, 0): ((8, 4), True, (8, 5), True, (8, 5), False, False),
    (1300, 50257, 640, 0): ((8, 5), True, (8, 5), True, (8, 5), False, False),
    (1030, 131101, 72, 0): ((8, 5), True, (8, 4), True, (8, 4), False, True),
    (2100, 64003, 72, 0): ((8, 4), True, (8, 4), True, (8, 4), False, True),
    (5000, 9973, 200, 0): ((8, 5), True, (8, 4), True, (8, 4), True, False),
    (4099, 4001, 1601, 0): ((8, 5), False, (8, 4), True, (8, 4), True, False),
    (600, 60007, 300, 0): ((8, 4), True, (8, 5), True, (8, 5), False, False),
    (8192, 3001, 5120, 0): ((8, 4), True, (8, 5), False, (8, 4), False, False),
    (5958, 5491, 640, 0): ((8, 5), True, (8, 4), True, (8, 5), True, False),
    (3001, 30011, 640, 1101): ((8, 5), True, (8, 4), True, (8, 5), False, False),
    (100, 70001, 40, 0): ((2, 4), True, (2, 4), True, (2, 4), False, False),
    (20, 140003, 24, 0): ((2, 4), True, (2, 4), True, (2, 4), False, False),
}


@pytest.mark.parametrize("n,v,d,chunk", CASES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_against_the_definition(n, v, d, chunk, kind):
    h, w, targets = make(n, v, d, TYPES[kind], seed=n + v + d)
    targets[torch.arange(n, device=DEV) % 7 == 3] = -100
    targets[n - 1], targets[0] = v - 1, 0                      # the last id of the last tile, the first of the first
    scale = 4096.0 if kind == "fp16" else 1.0
    check(h, w, targets, run(h, w, targets, scale=scale, max_tokens=chunk), scale=scale)
    check(h, w, targets, run(h, w, targets, grad=False, max_tokens=chunk))


@pytest.mark.parametrize("n,v,d,pad", [(1300, 50257, 640, 1), (600, 60007, 300, 4), (1029, 22001, 1600, 8)])
def test_rows_apart(n, v, d, pad):
    """Rows that are copied first, or loaded where they lie with NaN between them."""
    h, w, targets = make(n, v, d, torch.bfloat16, seed=n)
    big = [torch.full((rows + 1, d + pad), float("nan"), dtype=torch.bfloat16, device=DEV)[:rows, :d] for rows in (n, v)]
    big[0].copy_(h)
    big[1].copy_(w)
    targets[n // 2] = -100
    got = run(big[0], big[1], targets)
    check(big[0], big[1], targets, got)
    assert all(torch.equal(a, b) for a, b in zip(got, run(h, w, targets)))


@pytest.mark.parametrize("n,v,d,chunk", [(1300, 50257, 640, 0), (1030, 131101, 72, 0), (3001, 30011, 640, 1101), (100, 70001, 40, 0)])
def test_same_bits_and_replays(n, v, d, chunk):
    h, w, targets = make(n, v, d, torch.bfloat16, seed=5)
    first, second = (run(h, w, targets, max_tokens=chunk) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    outs = [torch.empty(n, device=DEV), torch.empty(n, device=DEV), torch.empty((), device=DEV), torch.empty_like(h), torch.empty_like(w)]
    space = torch.empty(zs.zero_vocab_loss_workspace(n, v, d, max_tokens=chunk), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zs.zero_vocab_loss(h, w, targets, *outs, space, max_tokens=chunk)
    for k in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(run(h, w, targets, max_tokens=chunk), outs)), k
        h.mul_(0.9)
        targets[k] = -100
