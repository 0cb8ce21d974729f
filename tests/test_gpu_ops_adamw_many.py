"""AdamW over tensors with many elements: the check's partials joined by a launch of their
own (from 2M elements), the update's large chunks (from 8M, with fp32 and with 8-bit
moments) and the moments' packing past the caches, bit for bit as in test_gpu_ops_adamw.py."""
import dataclasses

import pytest
import torch

import test_gpu_ops_adamw as small
import zero_dp_sharded_amd as zs
from test_gpu_ops_adamw import DEV, HP, check, make, step_by_hand, unpack

pytestmark = pytest.mark.gpu

LARGE = 8 << 20                 # elements from which on chunks are large, as in ops_internal.h
MODELS = {"3M": [1500003, 700001, 5, 1000000, 0, 70001], "9M": [5000011, 1, 3999999, 12289, 700, 300007]}


def held(x, r, least, signed):
    """small.held for all blocks at once (the same value, block by block)."""
    n = x.numel()
    blocks = -(-n // 256)
    fold = lambda z: torch.nn.functional.pad(z.double(), (0, blocks * 256 - n)).view(blocks, 256)
    y = fold(x)
    big = y.abs().amax(1, keepdim=True)
    frac, e = torch.frexp(big)
    e = torch.where(big == 0, -100, (e - 1 + (frac > 0.9375)).clamp_min(-100)).double()
    z = y.abs() * torch.exp2(-e)
    k = torch.frexp(z)[1] - 1
    step = torch.exp2(k.double().clamp_min(least) - 3)
    q = torch.clamp_max(torch.floor(z / step + (fold(r) + 0.5) / 65536) * step, 1.875)
    out = torch.sign(y) * q * torch.exp2(e)
    return torch.where(torch.isfinite(big), out, float("nan")).view(-1)[:n]


@pytest.mark.parametrize("signed,least", [(True, -14), (False, -30)])
def test_the_blocks_at_once_are_the_blocks_one_by_one(signed, least):
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(5003, generator=g, device=DEV) * torch.exp2(torch.randint(-140, 30, (5003,), generator=g, device=DEV).float())
    x = x if signed else x.abs()
    x[600:1300] = 0.0
    x[2000] = float("inf")
    r = torch.randint(0, 65536, (5003,), generator=g, device=DEV)
    assert small.same(held(x, r, least, signed), small.held(x, r, least, signed))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("name,kinds,scale,max_norm,off,checked", [
    ("3M", ["bf16", "fp32", "fp16"], 16.0, 0.3, 1, True), ("3M", ["fp32"], 1.0, 0.0, 0, False),
    ("9M", ["bf16", "fp32", "fp16"], 16.0, 0.3, 0, True), ("9M", ["fp16"], 1024.0, 0.0, 3, True), ("9M", ["bf16"], 1.0, 0.0, 0, False),
    ("9M", ["fp32"], 1.0, 5.0, 1, True)])
def test_steps_by_hand(monkeypatch, bits, name, kinds, scale, max_norm, off, checked):
    monkeypatch.setattr(small, "held", held)
    model = make(MODELS[name], kinds, bits, seed=7, scale=scale, off=off, zero_state=not checked)
    assert (sum(MODELS[name]) >= LARGE) == (name == "9M")
    hp = dataclasses.replace(HP, initial_step=2)
    seed = (9 << 32) + 5
    h = zs.zero_adamw_init(model.tensors, hp=hp, ls=zs.LossScaleCfg(init_scale=scale, dynamic=0), state_bits=bits,
                           max_grad_norm=max_norm, seed=seed, checked=checked)
    try:
        for t in (3, 4):
            _, norm, new = step_by_hand(model, hp, scale, t, bits, seed, max_norm, checked=checked)
            zs.zero_adamw_step(h)
            info = zs.zero_adamw_result(h)
            assert (info.overflow, info.skipped, info.step_t, info.scale_next) == (0, 0, t, scale)
            assert abs(info.grad_norm - norm) <= 1e-12 * norm if checked else info.grad_norm == 0
            check(model, new, bits)
            for g in model.grads:
                g.mul_(-1.25)
    finally:
        zs.zero_adamw_destroy(h)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("name", ["3M", "9M"])
def test_overflow_skips_wherever_it_is(bits, name):
    model = make(MODELS[name], ["bf16"], bits, seed=1)
    h = zs.zero_adamw_init(model.tensors, hp=HP, ls=zs.LossScaleCfg(init_scale=64.0), state_bits=bits)
    try:
        before = [a.clone() for a in model.arrays()]
        scale = 64.0
        for tensor, at in ((0, 0), (0, MODELS[name][0] - 1), (2, MODELS[name][2] // 2), (5, MODELS[name][5] - 1)):
            keep = model.grads[tensor][at].clone()
            model.grads[tensor][at] = float("inf")
            zs.zero_adamw_step(h)
            info = zs.zero_adamw_result(h)
            model.grads[tensor][at] = keep
            scale /= 2
            assert (info.skipped, info.step_t, info.scale_next) == (1, 0, scale)
            assert all(torch.equal(a, b) for a, b in zip(before, model.arrays())), (tensor, at)
        zs.zero_adamw_step(h)
        assert zs.zero_adamw_result(h).step_t == 1
    finally:
        zs.zero_adamw_destroy(h)


@pytest.mark.parametrize("bits", [32, 8])
def test_replays_are_the_eager_steps(bits):
    a, b = (make(MODELS["9M"], ["bf16", "fp32"], bits, seed=6) for _ in range(2))
    kw = dict(hp=HP, ls=zs.LossScaleCfg(init_scale=2.0, growth_interval=2), state_bits=bits, max_grad_norm=0.2, seed=3)
    ha, hb = zs.zero_adamw_init(a.tensors, **kw), zs.zero_adamw_init(b.tensors, **kw)
    try:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            zs.zero_adamw_step(ha)
        for k in range(4):
            if k == 2:
                a.grads[2][9] = b.grads[2][9] = float("nan")
            g.replay()
            zs.zero_adamw_step(hb)
            ia, ib = zs.zero_adamw_result(ha), zs.zero_adamw_result(hb)
            assert (ia.step_t, ia.skipped, ia.scale_next) == (ib.step_t, ib.skipped, ib.scale_next) and ia.skipped == (k == 2)
            assert all(torch.equal(x, y) for x, y in zip(a.arrays(), b.arrays())), k
            a.grads[2][9] = b.grads[2][9] = 0.25
    finally:
        zs.zero_adamw_destroy(ha)
        zs.zero_adamw_destroy(hb)


@pytest.mark.parametrize("signed,least", [(True, -14), (False, -30)])
@pytest.mark.parametrize("n,off", [(LARGE - 1, 0), (LARGE, 1), (LARGE + 255, 0), (LARGE + 8191, 3)])
def test_moments_past_the_caches(signed, least, n, off):
    g = torch.Generator(device=DEV).manual_seed(n)
    base = torch.randn(n + off, generator=g, device=DEV)
    base *= torch.exp2(torch.randint(-12, 3, (n + off,), generator=g, device=DEV).float())
    x = (base if signed else base.square())[off:]
    room = torch.full((n + off + 9,), 85, dtype=torch.uint8, device=DEV)
    codes, exps = room[off:off + n], torch.full((-(-n // 256) + 3,), 85, dtype=torch.int8, device=DEV)
    zs.zero_moments_pack(x, codes, exps[:-3], signed=signed)
    want = held(x, torch.full((n,), 32767, device=DEV), least, signed)
    assert torch.equal(unpack(codes, exps[:-3], signed).double(), want)
    out = torch.full((n + off + 9,), 7.0, dtype=torch.bfloat16, device=DEV)
    zs.zero_moments_unpack(codes, exps[:-3], out[off:off + n], signed=signed)
    assert torch.equal(out[off:off + n].double(), want)
    # what lies before and behind
    assert (room[:off] == 85).all() and (room[off + n:] == 85).all() and (exps[-3:] == 85).all()
    assert (out[:off] == 7).all() and (out[off + n:] == 7).all()
