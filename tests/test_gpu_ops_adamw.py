"""AdamW over tensors on the GPU: bit for bit the update of the oracle's shard step
with 32-bit moments, and with 8-bit moments the update and the held values of the
definition, step by step.

The update's arithmetic is fp32, each operation rounded once, so numpy's
elementwise operations give the same bits (torch's on the GPU do not: they divide by
a number by multiplying with its reciprocal); nothing here has a tolerance but the
norm (an fp64 sum in another order) and the statistics of the random rounding
(their own deviations)."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import oracle
import zero_dp_sharded_amd as zs

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = [0, 1, 3, 255, 256, 257, 4095, 4096, 4097, 20000, 12289, 5]


@dataclasses.dataclass
class Model:
    tensors: list
    grads: list

    def arrays(self):
        return [a for t in self.tensors for a in (t.master, t.param, t.exp_avg, t.exp_avg_sq, t.exp_avg_exp, t.exp_avg_sq_exp)
                if a is not None]


def make(sizes, kinds, bits, seed=0, scale=1.0, off=0, zero_state=True):
    """Tensors of the sizes, type by type in turn, each `off` elements into its allocation."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    tensors, grads = [], []
    for k, n in enumerate(sizes):
        t = TYPES[kinds[k % len(kinds)]]

        def place(x):
            base = torch.empty(n + off + 8, dtype=x.dtype, device=DEV)
            base[off:off + n].copy_(x)
            return base[off:off + n]

        r = lambda s: torch.randn(n, generator=g, device=DEV) * s
        grad = place((r(1e-2) * scale).to(t))
        master = place(r(0.5))
        m, v = (r(0.0), r(0.0)) if zero_state else (r(1e-2), r(1e-2).square())
        state = {}
        if bits == 8:
            blocks = -(-n // 256)
            cm, cv = (torch.zeros(n + off + 8, dtype=torch.uint8, device=DEV)[off:off + n] for _ in range(2))
            em, ev = (torch.zeros(blocks, dtype=torch.int8, device=DEV) for _ in range(2))
            if not zero_state:
                zs.zero_moments_pack(m, cm, em, signed=True)
                zs.zero_moments_pack(v, cv, ev, signed=False)
            state = dict(exp_avg_exp=em, exp_avg_sq_exp=ev)
            m, v = cm, cv
        else:
            m, v = place(m), place(v)
        tensors.append(zs.AdamWTensor(grad, master, None if t == torch.float32 else place(master.to(t)), m, v,
                                      weight_decay=[None, 0.0, 0.1][k % 3], lr_scale=[1.0, 0.5][k % 2], **state))
        grads.append(grad)
    return Model(tensors, grads)


def f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B9) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xB504F333) & 0xFFFFFFFF
    return x ^ (x >> 16)


def noise(seed, t, tensor, n):
    key = seed & 0xFFFFFFFF
    for more in (seed >> 32, t, tensor, 0):
        key = mix((mix(key) + more) & 0xFFFFFFFF)
    return mix((key + torch.arange(n, device=DEV) * 0xDDB3D743) & 0xFFFFFFFF)


def held(x, r, least, signed):
    """The value an element of a block of 256 is held as, in 64 bits: on the block's
    grid, up with the odds of the 16 bits r."""
    out = torch.empty_like(x, dtype=torch.float64)
    for b in range(0, x.numel(), 256):
        y, rr = x[b:b + 256].double(), r[b:b + 256].double()
        top = y.abs().max().item()
        if not math.isfinite(top):
            out[b:b + 256] = float("nan")
            continue
        e = -100 if top == 0 else max(-100, math.frexp(top)[1] - 1 + (math.frexp(top)[0] > 0.9375))
        z = y.abs() * 2.0 ** -e
        k = torch.frexp(z)[1] - 1
        step = torch.exp2(k.double().clamp_min(least) - 3)
        q = torch.clamp_max(torch.floor(z / step + (rr + 0.5) / 65536) * step, 1.875)
        out[b:b + 256] = torch.sign(y) * q * 2.0 ** e
    return out


def unpack(codes, exps, signed):
    x = torch.empty(codes.numel(), device=DEV)
    zs.zero_moments_unpack(codes, exps, x, signed=signed)
    return x


def step_by_hand(model, hp, ls_scale, t, bits, seed, max_norm, checked=True):
    """One step in fp32 elementwise operations; returns (skipped, norm, new arrays)."""
    inv = f32(1 / ls_scale)
    gs = [g.float() * inv for g in model.grads]
    sumsq = sum(g.double().square().sum().item() for g in gs)
    skip = checked and not math.isfinite(sumsq)
    coef = 1.0
    if checked and max_norm and not skip:
        coef = f32(min(1.0, max_norm / (math.sqrt(sumsq) + 1e-6)))
    new = []
    b1, b2 = f32(hp.beta1), f32(hp.beta2)
    p1 = p2 = 1.0
    for _ in range(t):
        p1, p2 = p1 * b1, p2 * b2
    bc1, bc2 = (f32(1 - p1), f32(1 - p2)) if hp.bias_correction else (1.0, 1.0)
    for k, (x, g) in enumerate(zip(model.tensors, gs)):
        wd = f32(hp.weight_decay if x.weight_decay is None else x.weight_decay)
        lr = (torch.tensor(hp.lr, dtype=torch.float32) * torch.tensor(x.lr_scale, dtype=torch.float32)).item()
        m = unpack(x.exp_avg, x.exp_avg_exp, True) if bits == 8 else x.exp_avg
        v = unpack(x.exp_avg_sq, x.exp_avg_sq_exp, False) if bits == 8 else x.exp_avg_sq
        F = np.float32
        g, m, v, p = (z.cpu().numpy() for z in (g, m, v, x.master))
        with np.errstate(all="ignore"):
            g = g * F(coef)
            if hp.wd_mode == zs.ZERO_WD_L2:
                g = g + F(wd) * p
            m = F(b1) * m + F(1 - b1) * g
            v = F(b2) * v + F(1 - b2) * (g * g)
            u = (m / F(bc1)) / (np.sqrt(v / F(bc2)) + F(hp.eps))
            if hp.wd_mode != zs.ZERO_WD_L2:
                u = u + F(wd) * p
            p = p - F(lr) * u
        assert all(z.dtype == np.float32 for z in (p, m, v))
        p, m, v = (torch.from_numpy(z).to(DEV) for z in (p, m, v))
        if bits == 8:
            r = noise(seed, t, k, g.size)
            m, v = held(m, r & 0xFFFF, -14, True), held(v, r >> 16, -30, False)
        new.append((p, None if x.param is None else p.cpu().to(x.param.dtype).to(DEV), m, v))
    return skip, math.sqrt(sumsq) if math.isfinite(sumsq) else math.nan, new


def same(a, b):
    return torch.equal(a.double().nan_to_num(nan=1e300), b.double().nan_to_num(nan=1e300))


def check(model, new, bits):
    for k, (x, (p, low, m, v)) in enumerate(zip(model.tensors, new)):
        gm = unpack(x.exp_avg, x.exp_avg_exp, True) if bits == 8 else x.exp_avg
        gv = unpack(x.exp_avg_sq, x.exp_avg_sq_exp, False) if bits == 8 else x.exp_avg_sq
        for name, a, b in (("master", x.master, p), ("m", gm, m), ("v", gv, v), ("param", x.param, low)):
            equal = b is None or same(a, b)
            assert equal, (k, name)


HP = zs.AdamHParams(lr=1e-2, beta1=0.9, beta2=0.95, weight_decay=0.02)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kinds,scale,max_norm,mode,off", [
    (["bf16"], 1.0, 0.0, 0, 0), (["fp16"], 1024.0, 0.5, 0, 1), (["fp32"], 1.0, 100.0, 1, 3),
    (["bf16", "fp32", "fp16"], 16.0, 0.3, 0, 2)])
def test_steps_by_hand(bits, kinds, scale, max_norm, mode, off):
    model = make(SIZES, kinds, bits, seed=7, scale=scale, off=off, zero_state=off == 1)
    hp = dataclasses.replace(HP, wd_mode=mode, initial_step=3)
    seed = (5 << 32) + 99
    h = zs.zero_adamw_init(model.tensors, hp=hp, ls=zs.LossScaleCfg(init_scale=scale, dynamic=0), state_bits=bits,
                           max_grad_norm=max_norm, seed=seed)
    try:
        for t in range(4, 8):
            skip, norm, new = step_by_hand(model, hp, scale, t, bits, seed, max_norm)
            zs.zero_adamw_step(h)
            info = zs.zero_adamw_result(h)
            assert (info.overflow, info.skipped, info.step_t, info.scale_next) == (0, 0, t, scale)
            assert abs(info.grad_norm - norm) <= 1e-12 * norm
            check(model, new, bits)
            for g in model.grads:
                g.mul_(-1.25)
    finally:
        zs.zero_adamw_destroy(h)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
def test_same_bits_as_the_shards_oracle(kind):
    """The tensors' update against the oracle's step on the same elements laid end to end."""
    code = {"fp16": oracle.FP16, "bf16": oracle.BF16, "fp32": oracle.FP32}[kind]
    sizes = [700, 1, 4096, 333]
    scale = 256.0
    model = make(sizes, [kind], 32, seed=3, scale=scale)
    for x in model.tensors:
        x.weight_decay, x.lr_scale = None, 1.0
    hp = zs.AdamHParams(lr=1e-3, weight_decay=0.01)
    ohp, ols = oracle.AdamHP(lr=1e-3, weight_decay=0.01), oracle.LossScale(init_scale=scale)
    cat = lambda name: torch.cat([getattr(x, name) for x in model.tensors])
    bits = lambda t: t.cpu().numpy() if kind == "fp32" else t.view(torch.int16).cpu().numpy().view(np.uint16)
    st = oracle.new_state(code, cat("master").cpu().numpy(), cat("exp_avg").cpu().numpy(), cat("exp_avg_sq").cpu().numpy(), ohp, ols)
    h = zs.zero_adamw_init(model.tensors, hp=hp, ls=zs.LossScaleCfg(init_scale=scale), max_grad_norm=0.5)
    try:
        for _ in range(3):
            oi = oracle.step(st, [bits(torch.cat(model.grads))], 1 << 20, ohp, ols, max_norm=0.5)
            zs.zero_adamw_step(h)
            info = zs.zero_adamw_result(h)
            assert (info.overflow, info.step_t, info.scale_next) == (oi.overflow, oi.step_t, oi.scale_next)
            assert abs(info.grad_norm - oi.grad_norm) <= 1e-12 * oi.grad_norm
            for name, want in (("master", st.master), ("exp_avg", st.m), ("exp_avg_sq", st.v)):
                assert np.array_equal(cat(name).cpu().numpy().view(np.uint32), want.view(np.uint32)), name
            if kind != "fp32":
                assert np.array_equal(bits(cat("param")), st.param)
    finally:
        zs.zero_adamw_destroy(h)


@pytest.mark.parametrize("bits", [32, 8])
def test_overflow_skips_and_rescales(bits):
    model = make([1000, 300], ["fp16"], bits, seed=1, scale=64.0)
    h = zs.zero_adamw_init(model.tensors, hp=HP, ls=zs.LossScaleCfg(init_scale=64.0, growth_interval=2, min_scale=16.0),
                           state_bits=bits)
    try:
        seen = []
        for k in range(7):
            before = [a.clone() for a in model.arrays()]
            bad = k in (1, 2, 3)
            keep = model.grads[1][299].clone()
            if bad:
                model.grads[1][299] = float("inf") if k == 1 else float("nan")
            zs.zero_adamw_step(h)
            info = zs.zero_adamw_result(h)
            model.grads[1][299] = keep
            unchanged = all(torch.equal(a, b) for a, b in zip(before, model.arrays()))
            assert unchanged == bad
            assert info.overflow == int(bad) and (not bad or not math.isfinite(info.grad_norm))
            seen.append((info.step_t, info.scale_used, info.scale_next))
        assert seen == [(1, 64.0, 64.0), (1, 64.0, 32.0), (1, 32.0, 16.0), (1, 16.0, 16.0), (2, 16.0, 16.0), (3, 16.0, 32.0),
                        (4, 32.0, 32.0)]
        assert zs.zero_adamw_get_counters(h) == (4, 32.0, 1)
    finally:
        zs.zero_adamw_destroy(h)


@pytest.mark.parametrize("bits", [32, 8])
def test_unchecked_steps_apply_what_they_get(bits):
    model = make([600, 256, 77], ["bf16"], bits, seed=2)
    hp = dataclasses.replace(HP, bias_correction=0)
    h = zs.zero_adamw_init(model.tensors, hp=hp, ls=zs.LossScaleCfg(dynamic=0), state_bits=bits, checked=False, seed=4)
    try:
        model.grads[0][300] = float("nan")
        model.grads[2][0] = float("inf")
        _, _, new = step_by_hand(model, hp, 1.0, 1, bits, 4, 0.0, checked=False)
        zs.zero_adamw_step(h)
        info = zs.zero_adamw_result(h)
        assert (info.overflow, info.step_t, info.grad_norm) == (0, 1, 0.0)
        check(model, new, bits)
        x = model.tensors[0]
        lost = torch.isnan(unpack(x.exp_avg, x.exp_avg_exp, True) if bits == 8 else x.exp_avg)
        # 32 bits lose the element, 8 bits its block
        assert lost.sum().item() == (1 if bits == 32 else 256) and lost[300]
    finally:
        zs.zero_adamw_destroy(h)


def test_random_rounding_keeps_the_mean():
    """A gradient that moves v by a thousandth a step: nearest rounding would never
    move it.  After s steps the held v's mean over n elements must be the exact one
    within 5 deviations: each step adds an independent error of at most half a code
    (2^-4 of v) an element."""
    n, steps = 1 << 16, 40
    grad = torch.full((n,), 2.0, device=DEV)
    arrays = [torch.zeros(n, device=DEV)]
    v0 = torch.full((n,), 1.1, device=DEV)
    v0[::256] = 1.875 * 4                       # the blocks' largest, which sets the grid
    cm, cv = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    em, ev = (torch.zeros(n // 256, dtype=torch.int8, device=DEV) for _ in range(2))
    zs.zero_moments_pack(v0, cv, ev, signed=False)
    start = unpack(cv, ev, False).double()
    hp = zs.AdamHParams(lr=0.0, beta1=0.9, beta2=0.999)
    h = zs.zero_adamw_init([zs.AdamWTensor(grad, arrays[0], None, cm, cv, em, ev)], hp=hp, ls=zs.LossScaleCfg(dynamic=0),
                           state_bits=8, checked=False, seed=77)
    try:
        for _ in range(steps):
            zs.zero_adamw_step(h)
    finally:
        zs.zero_adamw_destroy(h)
    rest = torch.arange(n, device=DEV) % 256 != 0
    got = unpack(cv, ev, False).double()[rest]
    b2 = f32(0.999)
    want = (start * b2 ** steps + 4.0 * (1 - b2 ** steps))[rest]
    deviation = 0.0625 * 2.0 * math.sqrt(steps) / math.sqrt(rest.sum().item())
    assert abs(got.mean().item() - want.mean().item()) <= 5 * deviation
    assert want.mean().item() - start[rest].mean().item() > 20 * deviation      # it has to have moved
    m = unpack(cm, em, True).double()
    assert abs(m.mean().item() - 2.0 * (1 - f32(0.9) ** steps)) <= 5 * 0.125 * 2.0 * math.sqrt(10) / math.sqrt(n)


@pytest.mark.parametrize("signed,least", [(True, -14), (False, -30)])
def test_codes(signed, least):
    # every code stands for what the header says, and packs to itself
    n = 128 if signed else 256
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    for e in (-100, -1, 0, 5, 120):
        exps = torch.full((1,), e, dtype=torch.int8, device=DEV)
        c = torch.arange(n, device=DEV)
        mag = torch.where(c < 8, (c & 7).double() * 2.0 ** (least - 3), (1 + (c & 7).double() / 8) * torch.exp2((c >> 3).double() - 1 + least))
        want = (torch.cat([mag, -mag]) if signed else mag) * 2.0 ** e
        got = unpack(codes, exps, signed)
        assert torch.equal(got.double(), want)
        low = torch.empty(256, dtype=torch.bfloat16, device=DEV)
        zs.zero_moments_unpack(codes, exps, low, signed=signed)
        assert torch.equal(low.double(), want)
        back, be = torch.empty_like(codes), torch.empty_like(exps)
        zs.zero_moments_pack(got, back, be, signed=signed)
        assert be.item() == e
        mask = codes != 128 if signed else codes >= 0          # -0 packs to 0
        assert torch.equal(back[mask], codes[mask])
    # 127 and what is not finite: NaN, for the block alone
    x = torch.randn(700, device=DEV).abs()
    x[300] = float("inf")
    c, e = torch.empty(700, dtype=torch.uint8, device=DEV), torch.empty(3, dtype=torch.int8, device=DEV)
    zs.zero_moments_pack(x, c, e, signed=signed)
    y = unpack(c, e, signed)
    assert e[1].item() == 127 and torch.isnan(y[256:512]).all() and torch.isfinite(y[:256]).all() and torch.isfinite(y[512:]).all()
    # nearest: off by at most half a step
    keep = torch.cat([torch.arange(256), torch.arange(512, 700)]).to(DEV)
    top = torch.where(torch.arange(700, device=DEV) < 256, x[:256].max(), x[512:].max()).double()
    assert ((y.double() - x.double()).abs()[keep] <= (torch.maximum(x.double() * 2.0 ** -4, top * 2.0 ** (least - 3)) * (1 + 2.0 ** -15))[keep]).all()
    # zeros, and values below every code
    z = torch.tensor([0.0, -0.0, 1e-42], device=DEV)
    c, e = torch.empty(3, dtype=torch.uint8, device=DEV), torch.empty(1, dtype=torch.int8, device=DEV)
    zs.zero_moments_pack(z, c, e, signed=signed)
    assert e.item() == -100 and not unpack(c, e, signed).any()


def test_other_gradients_counters_and_hyperparameters():
    sizes = [300] * 300 + [5]                   # more tensors than one launch of pointers
    model = make(sizes, ["fp32"], 32, seed=5)
    h = zs.zero_adamw_init(model.tensors, hp=HP, ls=zs.LossScaleCfg(dynamic=0))
    try:
        model.grads = [g * 3 for g in model.grads]
        zs.zero_adamw_set_grads(h, model.grads)
        for t in (1, 2):
            hp = dataclasses.replace(HP, lr=HP.lr / t, weight_decay=0.3)
            _, _, new = step_by_hand(model, hp, 1.0, t, 32, 0, 0.0)
            zs.zero_adamw_step(h, hp)
            assert zs.zero_adamw_result(h).step_t == t
            check(model, new, 32)
        zs.zero_adamw_set_counters(h, 41, 1.0, 7)
        assert zs.zero_adamw_get_counters(h) == (41, 1.0, 7)
        _, _, new = step_by_hand(model, HP, 1.0, 42, 32, 0, 0.0)
        zs.zero_adamw_step(h)
        check(model, new, 32)
        with pytest.raises(zs.ZeroError, match="betas"):
            zs.zero_adamw_step(h, dataclasses.replace(HP, beta1=0.8))
        with pytest.raises(ValueError):
            zs.zero_adamw_set_grads(h, model.grads[:-1])
        with pytest.raises(TypeError):
            zs.zero_adamw_set_grads(h, [g.half() for g in model.grads])
        with pytest.raises(zs.ZeroError):
            zs.zero_adamw_set_counters(h, -1, 1.0, 0)
    finally:
        zs.zero_adamw_destroy(h)
    with pytest.raises(zs.ZeroError, match="live"):
        zs.zero_adamw_step(h)


@pytest.mark.parametrize("bits", [32, 8])
def test_graphs_and_streams(bits):
    """Replays of one captured step are the steps of another handle, one by one."""
    a, b = (make(SIZES, ["bf16", "fp32"], bits, seed=6) for _ in range(2))
    kw = dict(hp=HP, ls=zs.LossScaleCfg(init_scale=2.0, growth_interval=2), state_bits=bits, max_grad_norm=0.2, seed=3)
    ha, hb = zs.zero_adamw_init(a.tensors, **kw), zs.zero_adamw_init(b.tensors, **kw)
    try:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            zs.zero_adamw_step(ha)
        s = torch.cuda.Stream()
        for k in range(5):
            if k == 3:
                a.grads[4][9] = b.grads[4][9] = float("inf")
            torch.cuda.synchronize()
            g.replay()
            zs.zero_adamw_step(hb, stream=s)
            ia, ib = zs.zero_adamw_result(ha), zs.zero_adamw_result(hb, stream=s)
            if k != 3:
                assert ia == ib
            else:
                assert ia.skipped == ib.skipped == 1 and ia.scale_next == ib.scale_next
            assert all(torch.equal(x, y) for x, y in zip(a.arrays(), b.arrays())), k
            a.grads[4][9] = b.grads[4][9] = 0.25
    finally:
        zs.zero_adamw_destroy(ha)
        zs.zero_adamw_destroy(hb)


def test_tensors_past_their_memory_are_refused():
    x = torch.zeros(1000, device=DEV)
    model = make([1000], ["fp32"], 32)
    t = model.tensors[0]
    from zero_dp_sharded_amd import ops
    import ctypes
    c = t.to_c(32)
    c.numel = 1 << 36
    h = ctypes.c_void_p()
    cfg = ops.ZeroAdamwCfg(32, 1, 0.0, 0)
    s = ops.lib().zero_adamw_init(ctypes.byref(c), 1, ctypes.byref(HP.to_c()), ctypes.byref(zs.LossScaleCfg().to_c()),
                                  ctypes.byref(cfg), ctypes.byref(h))
    assert s == zs.ZERO_ERR_INVALID_ARG and not h.value
    with pytest.raises(ValueError):
        zs.zero_adamw_init([dataclasses.replace(t, master=x[:999])], hp=HP, ls=zs.LossScaleCfg())
    with pytest.raises(TypeError):
        zs.zero_adamw_init([t], hp=HP, ls=zs.LossScaleCfg(), state_bits=8)
