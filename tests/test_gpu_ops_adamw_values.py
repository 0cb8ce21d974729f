"""AdamW over tensors at values where its arithmetic leaves fp32's usual range, bit for
bit against the same operations one by one in numpy (every one rounded once, so there
is no tolerance)."""
import dataclasses

import numpy as np
import pytest
import torch

import zero_dp_sharded_amd as zs
from test_gpu_ops_adamw import DEV, f32, step_by_hand

pytestmark = pytest.mark.gpu


class One:
    """One fp32 tensor with the given moments, and its gradient."""

    def __init__(self, p, m, v, g):
        place = lambda x: torch.as_tensor(x, dtype=torch.float32).to(DEV)
        self.tensors = [zs.AdamWTensor(place(g), place(p), None, place(m), place(v))]
        self.grads = [self.tensors[0].grad]


def bits(x):
    """The bits, every NaN the same."""
    b = x.cpu().numpy().view(np.uint32).copy()
    b[np.isnan(x.cpu().numpy())] = 0x7fc00000
    return b


def one_step(model, hp, t, checked=True):
    """The step by hand and on the GPU: (master, m, v) of both, as bits."""
    _, _, new = step_by_hand(model, hp, 1.0, t, 32, 0, 0.0, checked=checked)
    h = zs.zero_adamw_init(model.tensors, hp=hp, ls=zs.LossScaleCfg(init_scale=1.0, dynamic=0), checked=checked)
    try:
        zs.zero_adamw_step(h)
        torch.cuda.synchronize()
    finally:
        zs.zero_adamw_destroy(h)
    x = model.tensors[0]
    p, _, m, v = new[0]
    return [bits(z) for z in (x.master, x.exp_avg, x.exp_avg_sq)], [bits(z) for z in (p, m, v)]


@pytest.mark.parametrize("t0,beta1,beta2", [(0, 0.9, 0.999), (0, 0.9, 0.95), (3, 0.9, 0.999), (0, 0.5, 0.9999), (900, 0.9, 0.999)])
def test_bias_corrected_moments_past_the_largest_number(t0, beta1, beta2):
    """Moments whose quotient by the bias correction passes fp32's range: it is infinite, as
    the division makes it, the root of an infinite second moment stops the element, and
    nothing becomes NaN that is a number by the formula."""
    big = np.float32(3.4e38) * np.exp2(-np.arange(0, 64, 0.25, dtype=np.float64)).astype(np.float32)
    n = big.size
    m = np.concatenate([np.zeros(n), big, -big, np.full(n, 1e-3)]).astype(np.float32)
    v = np.concatenate([big, np.full(n, 1e-6), np.full(n, 2.0), big]).astype(np.float32)
    p = np.linspace(-1, 1, 4 * n).astype(np.float32)
    hp = zs.AdamHParams(lr=1e-2, beta1=beta1, beta2=beta2, weight_decay=0.1, initial_step=t0)
    got, want = one_step(One(p, m, v, np.zeros(4 * n)), hp, t0 + 1)
    for name, a, b in zip(("master", "m", "v"), got, want):
        assert np.array_equal(a, b), (name, int((a != b).sum()), np.flatnonzero(a != b)[:5])
    # an element without a first moment keeps its value but for the decay, however large the second
    assert np.isfinite(got[0][:n].view(np.float32)).all()


def test_zeros_keep_their_signs():
    """Every sign of a zero parameter, moment and gradient, with and without decay."""
    z = [0.0, -0.0]
    p, m, g = (np.array(a, dtype=np.float32).ravel() for a in np.meshgrid(z, z, z))
    for wd in (0.0, 0.1):
        hp = zs.AdamHParams(lr=1e-2, weight_decay=wd)
        got, want = one_step(One(p, m, np.zeros(8), g), hp, 1)
        for name, a, b in zip(("master", "m", "v"), got, want):
            assert np.array_equal(a, b), (name, wd, a, b)


@pytest.mark.parametrize("t", [1 << 40, 1 << 62])
def test_a_counter_of_any_size_is_taken_at_once(t):
    """The host's powers of the betas end where they no longer change; a step from there
    has corrections of 1."""
    hp = zs.AdamHParams(lr=1e-2)
    p, m, v, g = (np.linspace(a, 1, 300).astype(np.float32) for a in (-1, -0.5, 0.1, -0.2))
    model, plain = One(p, m, v, g), One(p, m, v, g)
    h = zs.zero_adamw_init(model.tensors, hp=hp, ls=zs.LossScaleCfg(init_scale=1.0, dynamic=0))
    k = zs.zero_adamw_init(plain.tensors, hp=dataclasses.replace(hp, bias_correction=0), ls=zs.LossScaleCfg(init_scale=1.0, dynamic=0))
    try:
        zs.zero_adamw_set_counters(h, t, 1.0, 5)
        assert zs.zero_adamw_get_counters(h) == (t, 1.0, 5)
        zs.zero_adamw_step(h)
        zs.zero_adamw_step(k)
        assert zs.zero_adamw_result(h).step_t == t + 1
        assert torch.equal(model.tensors[0].master, plain.tensors[0].master)
    finally:
        zs.zero_adamw_destroy(h)
        zs.zero_adamw_destroy(k)


@pytest.mark.parametrize("signed,least", [(True, -14), (False, -30)])
def test_codes_at_the_borders_of_the_noise(signed, least):
    """Values below the code's least normal exponent, as near to a border of the rounding as
    fp32 has them on either side: the held value is the definition's."""
    from test_gpu_ops_adamw import held, unpack
    r = 32767
    x = []
    for code in range(9):
        border = code + 1 - (r + 0.5) / 65536                       # of steps: from here on the code is the next
        at = np.float32(border)
        for away in range(-6, 7):
            x.append(np.float32(at) + np.float32(away) * np.spacing(at))
    x = np.array(x, dtype=np.float32) * np.float32(2.0 ** (least - 3))
    for e in (-90, -1, 0, 17):
        values = np.zeros(512, dtype=np.float32)
        values[:x.size] = x * np.float32(2.0 ** e)
        values[200], values[300:300 + x.size] = 1.875 * 2.0 ** e, -x * np.float32(2.0 ** e) if signed else x * np.float32(2.0 ** e)
        values[511] = 1.5 * 2.0 ** e
        v = torch.from_numpy(values).to(DEV)
        codes, exps = torch.empty(512, dtype=torch.uint8, device=DEV), torch.empty(2, dtype=torch.int8, device=DEV)
        zs.zero_moments_pack(v, codes, exps, signed=signed)
        assert (exps == e).all()
        want = held(v, torch.full((512,), r, device=DEV), least, signed)
        assert torch.equal(unpack(codes, exps, signed).double(), want), e
