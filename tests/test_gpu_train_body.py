"""The example with a layer in 8 bits: the operators run together as they are used, and their gradients are
those of the layer as it is computed (its operands held in 8 bits), by the formulas in 64 bits."""
import math

import pytest
import torch

import ops_scaled_common as sc
import zero_dp_sharded_amd as zs
from zero_dp_sharded_amd import train_head

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("update", ["adamw", "bytes", "owner"])
@pytest.mark.parametrize("storage", ["fp16", "bf16"])
def test_it_runs(update, storage):
    seen, model, info = train_head.train(steps=6, update=update, storage=storage, body="bytes")
    assert abs(seen[0] - math.log(1009)) < 0.5 and all(math.isfinite(x) for x in seen) and not info.skipped
    logp, entropy, among = train_head.evaluate(model)
    assert logp < 0 and 0 <= entropy <= math.log(1009) + 1e-3 and 0 <= among <= 1


def held(x, square):
    """The values that x is held as in 8 bits, in 64 bits."""
    x = x.double()
    _, big = sc.blocks_of(x, square)
    scale = torch.exp2(sc.spread(sc.scale_byte(big).double(), *x.shape, square) - 127)
    table = sc.E4M3.to(x.device)
    c = sc.codes(x / scale)
    return torch.where(c > 127, -table[c & 127], table[c & 127]) * scale


def norm(x, w):
    rstd = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6)
    return x * rstd * w, rstd


def norm_back(dy, x, w, rstd):
    xhat, g = x * rstd, dy * w
    return rstd * (g - xhat * (g * xhat).mean(1, keepdim=True)), (dy * xhat).sum(0)


@pytest.mark.parametrize("tokens,width", [(70, 192), (333, 130)])
def test_gradients_of_the_layer(tokens, width):
    model = train_head.Model(50, width, "bf16", torch.device(DEV), 3, "bytes")
    layers = train_head._Bytes(model, tokens, width, torch.device(DEV))
    g = torch.Generator(device=DEV).manual_seed(1)
    x, dy = (torch.randn(tokens, width, generator=g, device=DEV).bfloat16() for _ in range(2))
    dx = torch.empty_like(x)
    y = layers.forward(x)
    layers.backward(x, dy, dx)
    D = lambda t: t.double()
    w1, w2, body = (D(model.part(n)) for n in ("norm.weight", "norm2.weight", "body"))
    near = lambda got, want, tol: ((D(got) - want).norm() / want.norm()).item() <= tol
    # each by the arrays that the step before has left: a rounding to bf16, 2^-9 in the mean at most
    u = 2.0 ** -8
    y1, r1 = norm(D(x), w1)
    assert near(layers.y1, y1, u)
    held_y1 = sc.values(*layers.y1_held, False)
    assert near(layers.u, held_y1 @ held(model.part("body"), True).t(), u + 2.0 ** -10)
    s = D(layers.u) + D(x)
    y2, r2 = norm(D(layers.s), w2)
    assert near(layers.s, s, u) and near(y, y2, u)
    ds, dw2 = norm_back(D(dy), D(layers.s), w2, r2)
    assert near(layers.ds, ds, u) and near(model.grad_of("norm2.weight"), dw2, u)
    held_ds = held(layers.ds, False)
    assert near(layers.dy1, held_ds @ held(model.part("body"), True), u + 2.0 ** -10)
    dbody = held(layers.ds.t().contiguous(), False) @ held(layers.y1.t().contiguous(), False).t()
    assert near(model.grad_of("body"), dbody, u + 2.0 ** -10)
    back, dw1 = norm_back(D(layers.dy1), D(x), w1, r1)
    assert near(dx, back + D(layers.ds), u) and near(model.grad_of("norm.weight"), dw1, u)
    # and the whole against the layer without 8 bits: two factors held to 2^-4 at most each way
    whole = norm_back(D(layers.ds) @ body, D(x), w1, r1)[0] + D(layers.ds)
    assert near(dx, whole, 2.0 ** -3) and near(model.grad_of("body"), D(layers.ds).t() @ y1, 2.0 ** -3)


def test_the_loss_and_log_probabilities_agree():
    """The same hidden states through both: the loss is the mean of -logprobs, and with dlogprobs -1/counted the
    gradients are the loss's within both's roundings."""
    n, v, d = 300, 1201, 96
    g = torch.Generator(device=DEV).manual_seed(5)
    h = torch.randn(n, d, generator=g, device=DEV).bfloat16()
    w = (0.1 * torch.randn(v, d, generator=g, device=DEV)).bfloat16()
    ids = torch.randint(0, v, (n,), generator=g, device=DEV)
    ids[::9] = -100
    many = int((ids != -100).sum())
    losses, lse, loss = torch.empty(n, device=DEV), torch.empty(n, device=DEV), torch.empty((), device=DEV)
    a = [torch.empty_like(h), torch.empty_like(w)]
    zs.zero_vocab_loss(h, w, ids, losses, lse, loss, *a, torch.empty(zs.zero_vocab_loss_workspace(n, v, d), dtype=torch.uint8, device=DEV))
    logp, lse2 = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    zs.zero_token_logprobs(h, w, ids, logp, lse2, workspace=torch.empty(zs.zero_token_logprobs_workspace(n, v, d), dtype=torch.uint8, device=DEV))
    assert (losses + logp).abs().max() <= 1e-5 * losses.abs().max() and (lse - lse2).abs().max() <= 1e-5
    b = [torch.empty_like(h), torch.empty_like(w)]
    space = torch.empty(zs.zero_token_logprobs_workspace(n, v, d, gradient=True), dtype=torch.uint8, device=DEV)
    zs.zero_token_logprobs_backward(h, w, ids, lse2, None, torch.full((n,), -1.0 / many, device=DEV), None, *b, space)
    for p, q in zip(a, b):
        assert ((p.double() - q.double()).norm() / p.double().norm()).item() <= 2 * 2.0 ** -8
