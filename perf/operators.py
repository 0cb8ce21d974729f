"""The training operators next to the owner's step, as they are measured: layer norm (forward, and backward with the
reduction of the weight's gradient), the softmax cross entropy over a vocabulary taken straight from hidden states and
the output weight (with both gradients, and no logits returned), and AdamW over the tensors of a model at once, with
states in 32 or in 8 bits.  run() has each operator in a plain form, of elementary torch operations, and as the calls
of zero_dp_sharded_amd.

Shapes follow the tensors of a transformer of width h: ln1.w, ln1.b, qkv.w, qkv.b, proj.w, proj.b, ln2.w, ln2.b, fc1.w,
fc1.b, fc2.w, fc2.b for each layer, and an embedding of the vocabulary that is the output weight too."""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 256          # elements that share one exponent where states are held in 8 bits


def listed():
    return [
        # one row: the norm of a single token when a model answers, nothing but latency
        {"name": "norm_forward_token", "op": "norm", "backward": False, "rows": 1, "width": 1600, "type": "bf16", "affine": "bf16"},
        # the rows of one micro-batch of the 13B model (width 5120), statistics kept for the backward pass
        {"name": "norm_forward_batch", "op": "norm", "backward": False, "rows": 8192, "width": 5120, "type": "fp16", "affine": "fp16"},
        # rows and width that fit no tile, in 4-byte storage
        {"name": "norm_backward_odd", "op": "norm", "backward": True, "rows": 4099, "width": 1601, "type": "fp32", "affine": "fp32"},
        # a micro-batch of the 1.5B model (width 1600); fp32 weights beside 2-byte activations
        {"name": "norm_backward_batch", "op": "norm", "backward": True, "rows": 16384, "width": 1600, "type": "bf16", "affine": "fp32"},
        # an evaluation: the loss alone, odd counts of tokens and ids
        {"name": "loss_evaluation_odd", "op": "loss", "grad": False, "tokens": 2047, "vocab": 32003, "width": 768, "type": "fp16", "scale": 1.0},
        # the last tokens of a short prompt that is trained on: the weight's bytes count, not the products
        {"name": "loss_gradient_short", "op": "loss", "grad": True, "tokens": 16, "vocab": 50257, "width": 1600, "type": "bf16", "scale": 1.0},
        # one micro-batch in fp16 under the loss scale of the 1.5B workload
        {"name": "loss_gradient_scaled", "op": "loss", "grad": True, "tokens": 2048, "vocab": 50257, "width": 1600, "type": "fp16", "scale": 65536.0},
        # the largest: eight sequences of 1024 tokens of the 1.5B model
        {"name": "loss_gradient_batch", "op": "loss", "grad": True, "tokens": 8192, "vocab": 50257, "width": 1600, "type": "bf16", "scale": 1.0},
        # a model of a test's size: 25 tensors, most of them tiny; latency counts
        {"name": "adamw_small", "op": "adamw", "bits": 32, "layers": 2, "width": 256, "vocab": 1000, "type": "fp16", "scale": 1024.0, "checked": True, "max_norm": 0.0},
        # eight layers of the 1.5B model and its embedding, clipped
        {"name": "adamw_layers", "op": "adamw", "bits": 32, "layers": 8, "width": 1600, "vocab": 50257, "type": "bf16", "scale": 1.0, "checked": True, "max_norm": 1.0},
        # a small model in 4-byte storage, states in 8 bits, its embedding of an odd count of rows
        {"name": "adamw_bytes_small", "op": "adamw", "bits": 8, "layers": 4, "width": 640, "vocab": 32003, "type": "fp32", "scale": 1.0, "checked": True, "max_norm": 1.0},
        # the same eight layers with states in 8 bits, in bf16 without a check: one pass over everything
        {"name": "adamw_bytes_layers", "op": "adamw", "bits": 8, "layers": 8, "width": 1600, "vocab": 50257, "type": "bf16", "scale": 1.0, "checked": False, "max_norm": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "loss", "loss", "adamw"])
    if op == "norm":
        rows, width = _log(rng, 1, 16384), _log(rng, 16, 8192)
        kind = rng.choice(["fp16", "bf16", "fp32"])
        return {"op": op, "backward": rng.random() < 0.6, "rows": rows, "width": width, "type": kind, "affine": rng.choice([kind, "fp32"])}
    if op == "loss":
        tokens, vocab, width = _log(rng, 1, 8192), _log(rng, 500, 60000), _log(rng, 32, 2048)
        if rng.random() < 0.5:
            width = -(-width // 64) * 64
        while tokens * vocab * width > 8192 * 50257 * 1600:
            tokens = -(-tokens // 2)
        kind = rng.choice(["fp16", "bf16"])
        return {"op": op, "grad": rng.random() < 0.7, "tokens": tokens, "vocab": vocab, "width": width, "type": kind,
                "scale": rng.choice([1.0, 1024.0, 65536.0]) if kind == "fp16" else 1.0}
    kind = rng.choice(["fp16", "bf16", "fp32"])
    return {"op": op, "bits": rng.choice([8, 32]), "layers": rng.randint(1, 8), "width": _log(rng, 33, 1600), "vocab": _log(rng, 100, 50000), "type": kind,
            "scale": 4096.0 if kind == "fp16" else 1.0, "checked": rng.random() < 0.7, "max_norm": 0.0}


def _sizes(case):
    h = case["width"]
    layer = [h, h, 3 * h * h, 3 * h, h * h, h, h, h, 4 * h * h, 4 * h, 4 * h * h, h]
    return [case["vocab"] * h] + layer * case["layers"]


def work(case):
    size = lambda name: 4 if case[name] == "fp32" else 2
    if case["op"] == "norm":
        n, e, a = case["rows"] * case["width"], size("type"), size("affine")
        if case["backward"]:   # dy and x in, dx out; weight in, its and the bias's gradient out; the rows' statistics in
            return {"bytes": 3 * n * e + 3 * case["width"] * a + 8 * case["rows"], "flops": 14 * n}
        return {"bytes": 2 * n * e + 2 * case["width"] * a + 8 * case["rows"], "flops": 8 * n}
    if case["op"] == "loss":
        t, v, d = case["tokens"], case["vocab"], case["width"]
        operands = 2 * (t * d + v * d)
        rows = 8 * t + 8 * t + 4          # targets in, losses and log sums out, the mean
        if case["grad"]:                  # three products: the logits, the hidden states' gradient, the weight's
            return {"bytes": 2 * operands + rows, "flops": 6 * t * v * d}
        return {"bytes": operands + rows, "flops": 2 * t * v * d}
    n, e = sum(_sizes(case)), size("type")
    # both moments read and written; those in 8 bits also returned as the values they stand for, in 2 bytes
    moments = 2 * 2 * 4 if case["bits"] == 32 else 2 * (2 * (1 + 1 / BLOCK) + 2)
    return {"bytes": n * (e + 8 + moments + (e if e == 2 else 0)), "flops": 16 * n}


# ---------------------------------------------------------------- inputs

def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


class _Steps:
    """A handle that goes with its state."""

    def __init__(self, zs, h):
        self.zs, self.h = zs, h

    def __del__(self):
        self.zs.zero_adamw_destroy(self.h)


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1009 + 17)
    state = {"case": case, "op": case["op"], "type": TYPES[case["type"]]}
    {"norm": _prepare_norm, "loss": _prepare_loss, "adamw": _prepare_adamw}[case["op"]](case, state, gen)
    return state


def _prepare_norm(case, state, gen):
    rows, width, t, a = case["rows"], case["width"], state["type"], TYPES[case["affine"]]
    dev = gen.device
    # a residual stream: rows of different size and mean, a few channels far above the others
    x = _randn((rows, width), gen) * torch.exp(0.5 * _randn((rows, 1), gen)) + 0.3 * _randn((rows, 1), gen)
    x[:, :: max(1, width // 7)] *= 12.0
    state |= {"eps": 1e-5, "x": x.to(t), "weight": (1 + 0.2 * _randn((width,), gen)).to(a), "bias": (0.1 * _randn((width,), gen)).to(a)}
    state |= {"mean": torch.empty(rows, device=dev), "rstd": torch.empty(rows, device=dev)}
    if case["backward"]:
        state["dy"] = (1e-2 * _randn((rows, width), gen)).to(t)
        f = state["x"].float()      # what the forward pass has left
        mean = f.mean(1)
        state["mean"].copy_(mean)
        state["rstd"].copy_(torch.rsqrt((f - mean[:, None]).square().mean(1) + state["eps"]))
        state |= {"dx": torch.empty_like(state["x"]), "dweight": torch.empty_like(state["weight"]), "dbias": torch.empty_like(state["bias"])}
        if own:
            import zero_dp_sharded_amd as zs
            state["space"] = torch.empty(zs.zero_layernorm_workspace(rows, width), dtype=torch.uint8, device=dev)
    else:
        state["y"] = torch.empty_like(state["x"])


def _prepare_loss(case, state, gen):
    n, v, d, t = case["tokens"], case["vocab"], case["width"], state["type"]
    dev = gen.device
    weight = (0.02 * _randn((v, d), gen)).to(t)
    # ids by a falling law, a twentieth of them left out of the loss
    u = torch.rand(n, generator=gen, device=dev)
    targets = (torch.exp(u * math.log(v)) - 1).long().clamp_(0, v - 1)
    hidden = _randn((n, d), gen)
    # part of the tokens are predicted well: their hidden states lean towards their target's row
    row = weight[targets].float()
    lean = 15.0 * torch.rand((n, 1), generator=gen, device=dev) * (torch.rand((n, 1), generator=gen, device=dev) < 0.5)
    hidden = hidden + lean * row / row.norm(dim=1, keepdim=True).clamp_min(1e-6)
    left_out = torch.rand(n, generator=gen, device=dev) < 0.05
    left_out[0] = False
    targets[left_out] = -100
    state |= {"hidden": hidden.to(t), "weight": weight, "targets": targets, "scale": case["scale"]}
    state |= {"losses": torch.empty(n, device=dev), "lse": torch.empty(n, device=dev), "loss": torch.empty((), device=dev)}
    if case["grad"]:
        state |= {"dhidden": torch.empty_like(state["hidden"]), "dweight": torch.empty_like(weight)}
    if own:
        import zero_dp_sharded_amd as zs
        state["space"] = torch.empty(zs.zero_vocab_loss_workspace(n, v, d, gradient=case["grad"]), dtype=torch.uint8, device=dev)


def _prepare_adamw(case, state, gen):
    dev, t = gen.device, state["type"]
    sizes = _sizes(case)
    blocks = [-(-n // BLOCK) for n in sizes]
    total = sum(blocks) * BLOCK
    # one arena an array; each tensor begins at a whole block, the rest of its last block stays zero
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device=dev), torch.tensor(blocks, device=dev))
    begin = torch.tensor([0] + blocks, device=dev).cumsum(0)[:-1]
    within = torch.arange(sum(blocks), device=dev) - begin[tensor]
    lane = torch.arange(BLOCK, device=dev)
    held = within[:, None] * BLOCK + lane < torch.tensor(sizes, device=dev)[tensor][:, None]
    decay = torch.tensor([0.01 if n > 4 * case["width"] else 0.0 for n in sizes], device=dev)
    fill = lambda std: _randn((sum(blocks), BLOCK), gen) * std * held
    size_of_tensor = torch.exp(0.7 * _randn((len(sizes),), gen))[tensor][:, None]
    master = fill(0.02)
    state |= {"sizes": sizes, "blocks": blocks, "tensor": tensor, "within": within, "decay": decay[tensor][:, None], "master": master,
              "grad": (fill(1e-3) * size_of_tensor * case["scale"]).to(t), "t": 9, "seed": seed_of(case),
              "lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "scale": case["scale"], "max_norm": case["max_norm"], "checked": case["checked"]}
    if t != torch.float32:
        state["param"] = master.to(t)
    m, v = fill(3e-4) * size_of_tensor, fill(1e-3).square() * size_of_tensor.square() * (torch.rand((total // BLOCK, 1), generator=gen, device=dev) + 0.2)
    if case["bits"] == 32:
        state |= {"m": m, "v": v}
    else:
        half = torch.full((1, 1), 32767, device=dev, dtype=torch.int64)
        state["m"], state["m_exp"], _ = _encode(m, half, True)
        state["v"], state["v_exp"], _ = _encode(v, half, False)
        # at most 4 significant bits: bf16 has what 8 bits hold as it is
        state["m_values"], state["v_values"] = (torch.empty_like(m, dtype=torch.bfloat16) for _ in range(2))
    if own:
        import zero_dp_sharded_amd as zs
        tensors, at = [], 0
        for k, (n, b) in enumerate(zip(sizes, blocks)):
            part = lambda name, width=BLOCK: state[name].reshape(-1)[at * width: at * width + (n if width == BLOCK else b)] if name in state else None
            tensors.append(zs.AdamWTensor(grad=part("grad"), master=part("master"), param=part("param"), exp_avg=part("m"), exp_avg_sq=part("v"),
                                          exp_avg_exp=part("m_exp", 1), exp_avg_sq_exp=part("v_exp", 1), weight_decay=0.01 if n > 4 * case["width"] else 0.0))
            at += b
        hp = zs.AdamHParams(lr=state["lr"], beta1=state["beta1"], beta2=state["beta2"], eps=state["eps"], initial_step=state["t"])
        h = zs.zero_adamw_init(tensors, hp=hp, ls=zs.LossScaleCfg(init_scale=case["scale"], dynamic=0), state_bits=case["bits"],
                               checked=case["checked"], max_grad_norm=case["max_norm"], seed=state["seed"])
        state["steps"] = _Steps(zs, h)


def seed_of(case):
    return 12345 + case["layers"] * 1000003 + (case["width"] << 33)


# ---------------------------------------------------------------- one pass

def run(state):
    return {"norm": _norm, "loss": _loss, "adamw": _adamw}[state["op"]](state)


def _norm(s):
    if "dy" in s:
        if own:
            import zero_dp_sharded_amd as zs
            zs.zero_layernorm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"], s["space"])
        else:
            x, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
            xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
            g = dy * w
            dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
            s["dx"].copy_(dx)
            s["dweight"].copy_((dy * xhat).sum(0))
            s["dbias"].copy_(dy.sum(0))
        return [s["dx"], s["dweight"], s["dbias"]]
    if own:
        import zero_dp_sharded_amd as zs
        zs.zero_layernorm_forward(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], eps=s["eps"])
    else:
        x = s["x"].float()
        mean = x.mean(1)
        centred = x - mean[:, None]
        rstd = torch.rsqrt(centred.square().mean(1) + s["eps"])
        s["y"].copy_(centred * rstd[:, None] * s["weight"].float() + s["bias"].float())
        s["mean"].copy_(mean)
        s["rstd"].copy_(rstd)
    return [s["y"], s["mean"], s["rstd"]]


def _loss(s):
    outs = [s["losses"], s["lse"], s["loss"]] + ([s["dhidden"], s["dweight"]] if "dhidden" in s else [])
    if own:
        import zero_dp_sharded_amd as zs
        zs.zero_vocab_loss(s["hidden"], s["weight"], s["targets"], s["losses"], s["lse"], s["loss"], s.get("dhidden"), s.get("dweight"), s["space"],
                           grad_scale=s["scale"], ignore_index=-100)
        return outs
    hidden, weight, targets = s["hidden"].float(), s["weight"].float(), s["targets"]
    logits = hidden @ weight.t()
    top = logits.max(1, keepdim=True).values
    lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(1))
    counts = targets != -100
    at = torch.where(counts, targets, 0)[:, None]
    losses = torch.where(counts, lse - logits.gather(1, at)[:, 0], 0.0)
    many = counts.sum()
    s["losses"].copy_(losses)
    s["lse"].copy_(lse)
    s["loss"].copy_(losses.double().sum() / many.clamp_min(1))
    if "dhidden" in s:
        factor = counts.float() * (s["scale"] / many.clamp_min(1))
        p = torch.exp(logits - lse[:, None])
        p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
        p *= factor[:, None]
        s["dhidden"].copy_(p @ weight)
        s["dweight"].copy_(p.t() @ hidden)
    return outs


def _mix(x):
    """32 bits of noise from 32 bits, held in 64: multiplications by the fractions of the golden ratio and of the root of two."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B9) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xB504F333) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _noise(s, t):
    """The 32 bits that round element i of tensor j at step t, by (blocks, BLOCK)."""
    low = lambda n: torch.full((1,), n & 0xFFFFFFFF, device=s["tensor"].device, dtype=torch.int64)
    key = low(s["seed"])
    for more in (low(s["seed"] >> 32), low(t), s["tensor"], (s["within"] * BLOCK) >> 32):
        key = _mix((_mix(key) + more) & 0xFFFFFFFF)
    i = s["within"][:, None] * BLOCK + torch.arange(BLOCK, device=key.device)
    return _mix((key[:, None] + (i & 0xFFFFFFFF) * 0xDDB3D743) & 0xFFFFFFFF)


def _top(signed):
    """The least exponent of a normal value beside the largest value's, 0: 4 bits of exponent beside a sign, or 5."""
    return -14 if signed else -30


def _encode(x, r, signed):
    """Codes of x, the blocks' exponents, and what both stand for: 3 bits of mantissa, rounded up with the odds that r (16 bits) says."""
    big = x.abs().amax(1)
    frac, e = torch.frexp(big)                           # big = frac * 2^e, frac in [0.5, 1)
    e = torch.where(big > 0, e - 1 + (frac > 0.9375), -100).clamp(-100, 127)
    y = x.abs().double() * torch.exp2(-e.double())[:, None]
    _, k = torch.frexp(y)
    step = torch.exp2((k - 1).clamp_min(_top(signed)).double() - 3)
    q = torch.floor(y / step + (r.double() + 0.5) / 65536)
    y = torch.clamp_max(q * step, 1.875)
    # the code: exponent field and mantissa, counted on from the least
    frac, k = torch.frexp(y)
    field = k - _top(signed)
    code = torch.where((y > 0) & (field > 0), field * 8 + (frac * 16).long() - 8, (y * 2.0 ** (3 - _top(signed))).long())
    if signed:
        code = code + 128 * (x < 0)
        y = torch.where(x < 0, -y, y)
    return code.to(torch.uint8), e.to(torch.int8), y * torch.exp2(e.double())[:, None]


def _decode(code, e, signed):
    c = code.long()
    low = c & 127 if signed else c
    field, mantissa = low >> 3, (low & 7).double()
    y = torch.where(field > 0, (8 + mantissa) * torch.exp2((field + _top(signed) - 4).double()), mantissa * 2.0 ** (_top(signed) - 3))
    if signed:
        y = torch.where(c > 127, -y, y)
    return (y * torch.exp2(e.double())[:, None]).float()


def _f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def _adamw(s):
    bits = s["case"]["bits"]
    if own:
        zs = s["steps"].zs
        zs.zero_adamw_step(s["steps"].h)
        if bits == 8:
            zs.zero_moments_unpack(s["m"], s["m_exp"], s["m_values"], signed=True)
            zs.zero_moments_unpack(s["v"], s["v_exp"], s["v_values"], signed=False)
    else:
        s["t"] += 1
        b1, b2 = _f32(s["beta1"]), _f32(s["beta2"])
        bc1, bc2 = _f32(1 - b1 ** s["t"]), _f32(1 - b2 ** s["t"])
        m = s["m"] if bits == 32 else _decode(s["m"], s["m_exp"], True)
        v = s["v"] if bits == 32 else _decode(s["v"], s["v_exp"], False)
        g = s["grad"].float() * _f32(1 / s["scale"])
        if s["checked"]:
            square = g.double().square().sum()
            skip = ~torch.isfinite(square)
            if s["max_norm"]:
                g = g * (s["max_norm"] / (square.sqrt() + 1e-6)).clamp_max(1).float()
        m = m * b1 + g * _f32(1 - b1)
        v = v * b2 + (g * g) * _f32(1 - b2)
        u = (m / bc1) / ((v / bc2).sqrt() + _f32(s["eps"])) + s["decay"] * s["master"]
        p = s["master"] - u * _f32(s["lr"])
        new = {"master": p}
        if "param" in s:
            new["param"] = p.to(s["type"])
        if bits == 32:
            new |= {"m": m, "v": v}
        else:
            r = _noise(s, s["t"])
            new["m"], new["m_exp"], new["m_values"] = _encode(m, r & 0xFFFF, True)
            new["v"], new["v_exp"], new["v_values"] = _encode(v, r >> 16, False)
            if s["checked"]:    # where the step is left out, the values of what is held already
                new["m_values"], new["v_values"] = (torch.where(skip, _decode(s[n], s[n + "_exp"], n == "m"), new[n + "_values"]) for n in "mv")
        for name, x in new.items():
            s[name].copy_(torch.where(skip, s[name], x) if s["checked"] and "values" not in name else x)
    m, v = (s["m"], s["v"]) if bits == 32 else (s["m_values"], s["v_values"])
    return [s["master"], m, v] + ([s["param"]] if "param" in s else [])


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "loss": _exact_loss, "adamw": _exact_adamw}[case["op"]](case, s)


def _exact_norm(case, s):
    x, w = s["x"].double(), s["weight"].double()
    if not case["backward"]:
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + s["eps"])
        return [(x - mean[:, None]) * (w * rstd[:, None]) + s["bias"].double(), mean, rstd]
    # the gradient by the rows' own statistics: d/dx of sum(dy * (w * xhat + b))
    dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    xhat = (x - mean) * rstd
    a = (dy * w).sum(1, keepdim=True) / case["width"]
    b = (dy * w * xhat).sum(1, keepdim=True) / case["width"]
    return [rstd * dy * w - rstd * a - rstd * xhat * b, (dy * xhat).sum(0), dy.sum(0)]


def _exact_loss(case, s):
    h, w, targets = s["hidden"].double(), s["weight"].double(), s["targets"]
    kept = torch.nonzero(targets != -100)[:, 0]
    n, many = case["tokens"], max(1, kept.numel())
    losses, lse = h.new_zeros(n), h.new_zeros(n)
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for at in range(0, n, 2048):
        z = h[at:at + 2048] @ w.t()
        lse[at:at + 2048] = torch.logsumexp(z, 1)
        rows = kept[(kept >= at) & (kept < at + 2048)]
        losses[rows] = lse[rows] - z[rows - at, targets[rows]]
        if case["grad"]:
            # p_i - [i is the target], for the target by the others' sum, which does not cancel
            d = torch.softmax(z[rows - at], 1)
            line = torch.arange(rows.numel(), device=rows.device)
            d[line, targets[rows]] = 0
            d[line, targets[rows]] = -d.sum(1)
            d *= s["scale"] / many
            dh[rows] = d @ w
            dw += d.t() @ h[rows]
    return [losses, lse, losses.sum() / many] + ([dh, dw] if case["grad"] else [])


def _exact_code(x, r, signed):
    """The value that x of a block is held as: on the grid of 4 significant bits, down to the least exponent, with the odds of r."""
    big = x.abs().amax(1, keepdim=True)
    # the largest value is at most 1.875 times a power of two; below 2^-100 the power stays
    power = torch.ceil(torch.log2(big.clamp_min(1e-300) / 1.875))
    power = power + (big > 1.875 * torch.exp2(power)).double() - (big <= 0.9375 * torch.exp2(power)).double()
    unit = torch.exp2(power.clamp_min(-100.0))
    y = x.abs() / unit
    e = torch.floor(torch.log2(y.clamp_min(1e-300)))
    e = e + (y >= torch.exp2(e + 1)).double() - (y < torch.exp2(e)).double()
    grid = torch.exp2(e.clamp_min(-14.0 if signed else -30.0)) / 8
    up = (2 * r.double() + 1) / 131072
    return torch.sign(x) * torch.minimum(torch.floor(y / grid + up) * grid, torch.full_like(y, 1.875)) * unit


def _exact_adamw(case, s):
    big = sum(_sizes(case)) > 1 << 29
    if big:
        return None
    t = s["t"] + 1
    b1, b2 = _f32(s["beta1"]), _f32(s["beta2"])          # a step's constants are given as 32-bit numbers
    g = s["grad"].double() / s["scale"]
    if s["checked"] and s["max_norm"]:
        g *= min(1.0, s["max_norm"] / (g.square().sum().sqrt().item() + 1e-6))
    m, v = s["m"], s["v"]
    if case["bits"] == 8:
        m, v = (_exact_held(s[n], s[n + "_exp"], n == "m") for n in ("m", "v"))
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    p = s["master"].double()
    step = (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + _f32(s["eps"])) + s["decay"].double() * p
    p = p - _f32(s["lr"]) * step
    if case["bits"] == 8:
        noise = _exact_noise(s, t)
        m, v = _exact_code(m, noise % 65536, True), _exact_code(v, noise // 65536, False)
    return [p, m, v] + ([p] if "param" in s else [])


def _exact_held(code, e, signed):
    """What codes stand for: a table of the 128 or 256 magnitudes, and the blocks' powers of two."""
    least = -14 if signed else -30
    table = [(j & 7) * 2.0 ** (least - 3) if j < 8 else (1 + (j & 7) / 8) * 2.0 ** ((j >> 3) - 1 + least) for j in range(128 if signed else 256)]
    table = torch.tensor(table + ([-x for x in table] if signed else []), dtype=torch.float64, device=code.device)
    return table[code.long()] * (2.0 ** e.double())[:, None]


def _exact_noise(s, t):
    """The noise, word by word, by remainders."""
    word, gold, two, three = 2 ** 32, 0x9E3779B9, 0xB504F333, 0xDDB3D743

    def mix(x):
        x = x ^ x // 65536
        x = (x * gold) % word
        x = x ^ x // 32768
        x = (x * two) % word
        return x ^ x // 65536

    first = torch.zeros_like(s["tensor"])
    key = first + s["seed"] % word
    key = mix((mix(key) + s["seed"] // word) % word)
    key = mix((mix(key) + t) % word)
    key = mix((mix(key) + s["tensor"]) % word)
    key = mix((mix(key) + s["within"] * BLOCK // word) % word)
    i = (s["within"][:, None] * BLOCK + torch.arange(BLOCK, device=first.device)) % word
    return mix((key[:, None] + i * three) % word)
