"""More of the training operators, as they are measured: the root-mean-square norm with the residual's addition and an
output in 8 bits (and its backward pass), packing to 8 bits with a power of two for every 128 elements, the matrix product
of what is packed so, and the log probabilities of given tokens with entropy and top alternatives, straight from hidden
states and the output weight (with both gradients).  run() has each operator in a plain form, of elementary torch
operations, and as the calls of zero_dp_sharded_amd.

8-bit numbers are e4m3 (a sign, 4 bits of exponent, 3 of mantissa, up to 448); 128 of them side by side, or a square of
128 x 128, share a power of two, held as its exponent plus 127 in a byte."""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128          # elements that share a scale
LARGEST = 448.0      # of e4m3


def listed():
    return [
        # one token when a model answers: latency alone; what the next product reads comes out in 8 bits
        {"name": "norm_forward_token", "op": "norm", "backward": False, "rows": 1, "width": 1600, "type": "bf16", "affine": "bf16", "bytes": True},
        # a micro-batch of the 13B model (width 5120) before a product in 8 bits
        {"name": "norm_forward_batch", "op": "norm", "backward": False, "rows": 8192, "width": 5120, "type": "bf16", "affine": "fp32", "bytes": True},
        # rows and width that fit no tile, the result in storage
        {"name": "norm_forward_odd", "op": "norm", "backward": False, "rows": 4099, "width": 1601, "type": "fp16", "affine": "fp16", "bytes": False},
        # the backward pass of a micro-batch of the 1.5B model, with the gradient that comes down the residual's way
        {"name": "norm_backward_batch", "op": "norm", "backward": True, "rows": 16384, "width": 1600, "type": "bf16", "affine": "fp32"},
        # a gradient of the 1.5B model's wide layer, for both products of its backward pass: along rows and turned
        {"name": "pack_both_batch", "op": "pack", "rows": 8192, "width": 6400, "type": "bf16", "square": False, "turned": True},
        # a small model's fp32 master weight after an update: squares, odd sizes
        {"name": "pack_square_odd", "op": "pack", "rows": 4801, "width": 1601, "type": "fp32", "square": True, "turned": False},
        # one token through a layer of the 1.5B model: the weight's bytes count
        {"name": "product_token", "op": "product", "m": 1, "n": 6400, "k": 1600, "type": "bf16", "square": True, "bias": True},
        # the gradient of a weight of odd sizes over an odd count of tokens: scales along the tokens on both sides
        {"name": "product_gradient_odd", "op": "product", "m": 4801, "n": 1601, "k": 4099, "type": "fp32", "square": False, "bias": False},
        # the largest: a micro-batch through the 13B model's wide layer
        {"name": "product_batch", "op": "product", "m": 8192, "n": 20480, "k": 5120, "type": "bf16", "square": True, "bias": False},
        # the tokens that sixteen sequences answer with, and their alternatives
        {"name": "logprobs_answers", "op": "logprobs", "grad": False, "tokens": 16, "vocab": 50257, "width": 1600, "type": "bf16", "top": 20, "entropy": True},
        # what a policy gave eight sequences of 1024 tokens
        {"name": "logprobs_batch", "op": "logprobs", "grad": False, "tokens": 8192, "vocab": 50257, "width": 1600, "type": "bf16", "top": 5, "entropy": True},
        # the gradients of a policy's loss on a micro-batch, an entropy bonus in it, under a loss scale
        {"name": "logprobs_gradient", "op": "logprobs", "grad": True, "tokens": 2048, "vocab": 50257, "width": 1600, "type": "fp16", "entropy": True, "scale": 4096.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "pack", "product", "product", "logprobs", "logprobs"])
    if op == "norm":
        rows, width = _log(rng, 1, 16384), _log(rng, 16, 8192)
        kind, backward = rng.choice(["fp16", "bf16", "fp32"]), rng.random() < 0.5
        case = {"op": op, "backward": backward, "rows": rows, "width": width, "type": kind, "affine": rng.choice([kind, "fp32"])}
        return case if backward else case | {"bytes": rng.random() < 0.6}
    if op == "pack":
        rows, width = _log(rng, 1, 16384), _log(rng, 16, 8192)
        return {"op": op, "rows": rows, "width": width, "type": rng.choice(["fp16", "bf16", "fp32"]), "square": rng.random() < 0.5,
                "turned": rng.random() < 0.6}
    if op == "product":
        m, n, k = _log(rng, 1, 8192), _log(rng, 16, 20480), _log(rng, 16, 20480)
        if rng.random() < 0.5:
            n, k = -(-n // 64) * 64, -(-k // 64) * 64
        while m * n * k > 8192 * 20480 * 5120:
            m = -(-m // 2)
        return {"op": op, "m": m, "n": n, "k": k, "type": rng.choice(["fp16", "bf16", "fp32"]), "square": rng.random() < 0.6, "bias": rng.random() < 0.4}
    tokens, vocab, width = _log(rng, 1, 8192), _log(rng, 500, 60000), _log(rng, 32, 2048)
    if rng.random() < 0.5:
        width = -(-width // 64) * 64
    grad = rng.random() < 0.4
    while tokens * vocab * width * (3 if grad else 1) > 8192 * 50257 * 1600:
        tokens = -(-tokens // 2)
    kind = rng.choice(["fp16", "bf16"])
    case = {"op": op, "grad": grad, "tokens": tokens, "vocab": vocab, "width": width, "type": kind, "entropy": rng.random() < 0.7}
    return case | {"scale": 4096.0 if kind == "fp16" else 1.0} if grad else case | {"top": rng.choice([0, 1, 5, 20, rng.randint(2, 32)])}


def work(case):
    size = lambda name: 4 if case[name] == "fp32" else 2
    if case["op"] == "norm":
        n, e, a, rows, width = case["rows"] * case["width"], size("type"), size("affine"), case["rows"], case["width"]
        if case["backward"]:   # dy, h and the residual's gradient in, dx out; weight in, its gradient out; a statistic a row
            return {"bytes": 4 * n * e + 2 * width * a + 4 * rows, "flops": 10 * n}
        # x and the residual in, their sum out; the result, or its codes with their scales and the values they stand for
        out = n + rows * -(-width // BLOCK) + 2 * n if case["bytes"] else e * n
        return {"bytes": 3 * n * e + out + width * a + 4 * rows, "flops": 6 * n}
    if case["op"] == "pack":
        n = case["rows"] * case["width"]
        return {"bytes": n * (size("type") + (6 if case["turned"] else 3)), "flops": 4 * n}     # with the values, in 2 bytes
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = -(-k // BLOCK)
        scales = m * blocks + (-(-n // BLOCK) if case["square"] else n) * blocks
        return {"bytes": m * k + n * k + scales + m * n * size("type") + (n * size("type") if case["bias"] else 0), "flops": 2 * m * n * k}
    t, v, d = case["tokens"], case["vocab"], case["width"]
    operands = 2 * (t * d + v * d)
    if case["grad"]:           # three products: the logits, the hidden states' gradient, the weight's
        return {"bytes": 2 * operands + 24 * t, "flops": 6 * t * v * d}
    return {"bytes": operands + t * (8 + 8 + 4 * case["entropy"] + 12 * case["top"]), "flops": 2 * t * v * d}


# ---------------------------------------------------------------- inputs

def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


def _rand(shape, gen):
    return torch.rand(shape, generator=gen, device=gen.device)


def prepare(case, seed):
    gen = torch.Generator(device=torch.device("cuda", 0))
    gen.manual_seed(seed * 1013 + 29)
    state = {"case": case, "op": case["op"], "type": TYPES[case["type"]]}
    {"norm": _prepare_norm, "pack": _prepare_pack, "product": _prepare_product, "logprobs": _prepare_logprobs}[case["op"]](case, state, gen)
    return state


def _stream_of_rows(rows, width, gen):
    """A residual stream: rows of different size, a few channels far above the others."""
    x = _randn((rows, width), gen) * torch.exp(0.5 * _randn((rows, 1), gen))
    x[:, :: max(1, width // 7)] *= 12.0
    return x


def _prepare_norm(case, state, gen):
    rows, width, t, a = case["rows"], case["width"], state["type"], TYPES[case["affine"]]
    dev = gen.device
    state |= {"eps": 1e-6, "weight": (1 + 0.2 * _randn((width,), gen)).to(a)}
    stream = _stream_of_rows(rows, width, gen)
    if case["backward"]:
        state |= {"h": stream.to(t), "dy": (1e-2 * _randn((rows, width), gen)).to(t), "dh": (1e-2 * _randn((rows, width), gen)).to(t)}
        # what the forward pass has left
        state["rstd"] = torch.rsqrt(state["h"].float().square().mean(1) + state["eps"])
        state |= {"dx": torch.empty_like(state["h"]), "dweight": torch.empty_like(state["weight"])}
        if own:
            import zero_dp_sharded_amd as zs
            state["space"] = torch.empty(zs.zero_rmsnorm_workspace(rows, width), dtype=torch.uint8, device=dev)
        return
    state |= {"residual": stream.to(t), "x": (0.3 * _randn((rows, width), gen)).to(t)}
    state |= {"h": torch.empty_like(state["x"]), "rstd": torch.empty(rows, device=dev)}
    if case["bytes"]:
        state |= _room(rows, width, False, dev)
        state["values"] = torch.empty(rows, width, dtype=torch.bfloat16, device=dev)
    else:
        state["y"] = torch.empty_like(state["x"])


def _room(rows, width, square, dev):
    """Arrays for codes and exponents."""
    return {"codes": torch.empty(rows, width, dtype=torch.float8_e4m3fn, device=dev),
            "exps": torch.empty(-(-rows // BLOCK) if square else rows, -(-width // BLOCK), dtype=torch.uint8, device=dev)}


def _prepare_pack(case, state, gen):
    rows, width = case["rows"], case["width"]
    # a gradient, rows of different size; or a weight
    x = 0.02 * _randn((rows, width), gen) if case["square"] else 1e-3 * _randn((rows, width), gen) * torch.exp(_randn((rows, 1), gen))
    state["x"] = x.to(state["type"])
    state |= _room(rows, width, case["square"], gen.device)
    # at most 4 significant bits: bf16 has what 8 bits hold as it is
    state["values"] = torch.empty(rows, width, dtype=torch.bfloat16, device=gen.device)
    if case["turned"]:
        state |= {name + "_t": x for name, x in _room(width, rows, case["square"], gen.device).items()}
        state["values_t"] = torch.empty(width, rows, dtype=torch.bfloat16, device=gen.device)


def _prepare_product(case, state, gen):
    m, n, k, t = case["m"], case["n"], case["k"], state["type"]
    # rows scaled as packing leaves them; the other side's squares, or rows of another gradient
    state["a"], state["a_exps"] = _held(_randn((m, k), gen) * torch.exp(0.7 * _randn((m, 1), gen)), False)
    b = 0.02 * _randn((n, k), gen) if case["square"] else _randn((n, k), gen) * torch.exp(0.7 * _randn((n, 1), gen))
    state["b"], state["b_exps"] = _held(b, case["square"])
    state["out"] = torch.empty(m, n, dtype=t, device=gen.device)
    if case["bias"]:
        state["bias"] = (0.1 * _randn((n,), gen)).to(t)
    if own:
        import zero_dp_sharded_amd as zs
        state["space"] = torch.empty(zs.zero_scaled_product_workspace(m, n, k), dtype=torch.uint8, device=gen.device)


def _prepare_logprobs(case, state, gen):
    n, v, d, t = case["tokens"], case["vocab"], case["width"], state["type"]
    dev = gen.device
    # Both sides lie on grids of which 24 bits hold every sum of products: the same logits for every order of adding, and
    # with them the same alternatives, those of equal logits among them.
    grid = lambda x, step, most: (torch.round(x / step) * step).clamp_(-most, most)
    weight = grid(0.02 * _randn((v, d), gen), 2.0 ** -9, 0.25)
    u = _rand((n,), gen)
    tokens = (torch.exp(u * math.log(v)) - 1).long().clamp_(0, v - 1)
    row = weight[tokens]
    # part of the tokens are expected: their hidden states lean towards their row of the weight
    lean = 15.0 * _rand((n, 1), gen) * (_rand((n, 1), gen) < 0.6)
    hidden = grid(_randn((n, d), gen) + lean * row / row.norm(dim=1, keepdim=True).clamp_min(1e-6), 2.0 ** -4, 15.0)
    absent = _rand((n,), gen) < 0.05
    absent[0] = False
    tokens[absent] = -100                # places of a prompt or a filled-up batch
    state |= {"hidden": hidden.to(t), "weight": weight.to(t), "tokens": tokens}
    if case["grad"]:
        logits = _logits(state)
        state["lse"], _, state["entropy"] = _statistics(logits)           # what the forward pass has left
        state["dlogprobs"] = torch.where(absent, 0.0, _randn((n,), gen) * (case["scale"] / n))
        state["dentropy"] = torch.where(absent, 0.0, torch.full((n,), -0.01 * case["scale"] / n, device=dev)) if case["entropy"] else None
        state |= {"dhidden": torch.empty_like(state["hidden"]), "dweight": torch.empty_like(state["weight"])}
    else:
        state |= {"lse": torch.empty(n, device=dev), "logprobs": torch.empty(n, device=dev)}
        state["entropy"] = torch.empty(n, device=dev) if case["entropy"] else None
        top = case["top"]
        state |= {"top_ids": torch.empty(n, top, dtype=torch.int64, device=dev) if top else None,
                  "top_logprobs": torch.empty(n, top, device=dev) if top else None}
    if own:
        import zero_dp_sharded_amd as zs
        state["space"] = torch.empty(zs.zero_token_logprobs_workspace(n, v, d, top=case.get("top", 0), gradient=case["grad"]), dtype=torch.uint8, device=dev)


# ---------------------------------------------------------------- one pass

def run(state):
    return {"norm": _norm, "pack": _pack, "product": _product, "logprobs": _logprobs}[state["op"]](state)


def _blocks(x, square):
    """x in whole blocks, zeros behind its ends: (rows, blocks, 128), or (blocks, 128, blocks, 128)."""
    rows, width = x.shape
    x = torch.nn.functional.pad(x, (0, -width % BLOCK, 0, -rows % BLOCK if square else 0))
    return x.view(-1, BLOCK, x.shape[1] // BLOCK, BLOCK) if square else x.view(rows, -1, BLOCK)


def _encode(x, square):
    """What x is held as in 8 bits (before and after its scale), and the scales' exponents."""
    b = _blocks(x, square)
    over = (1, 3) if square else (2,)
    # the least power of two by which the largest is within e4m3
    frac, e = torch.frexp(b.abs().amax(over))
    e = torch.where(frac > 0, e - 9 + (frac > 0.875), -100).clamp(-100, 127)
    scale = torch.exp2(e.float())
    scale = scale[:, None, :, None] if square else scale[:, :, None]
    y = b / scale
    _, k = torch.frexp(y)
    step = torch.exp2((k - 1).clamp_min(-6).float() - 3)
    y = (torch.round(y / step) * step).clamp(-LARGEST, LARGEST)
    cut = lambda z: z.reshape(b.shape[0] * (BLOCK if square else 1), -1)[:x.shape[0], :x.shape[1]]
    return cut(y), cut(y * scale), (e + 127).to(torch.uint8)


def _held(x, square):
    y, _, e = _encode(x, square)
    return y.to(torch.float8_e4m3fn), e


def _scales(exps, rows, width, square, kind):
    """The scale of every element."""
    s = torch.exp2(exps.to(kind) - 127)
    if square:
        s = s.repeat_interleave(BLOCK, 0)[:rows]
    return s.repeat_interleave(BLOCK, 1)[:, :width]


def _norm(s):
    if "dy" in s:
        if own:
            import zero_dp_sharded_amd as zs
            zs.zero_rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dh"], s["dweight"], s["space"])
        else:
            dy, w, rstd = s["dy"].float(), s["weight"].float(), s["rstd"][:, None]
            xhat = s["h"].float() * rstd
            g = dy * w
            s["dx"].copy_(rstd * (g - xhat * (g * xhat).mean(1, keepdim=True)) + s["dh"].float())
            s["dweight"].copy_((dy * xhat).sum(0))
        return [s["dx"], s["dweight"]]
    held = "codes" in s
    if own:
        import zero_dp_sharded_amd as zs
        zs.zero_rmsnorm_forward(s["x"], s["residual"], s["weight"], s["h"], s.get("y"), s["rstd"], s.get("codes"), s.get("exps"), eps=s["eps"])
        if held:
            zs.zero_scaled_unpack(s["codes"], s["exps"], s["values"])
    else:
        s["h"].copy_(s["x"].float() + s["residual"].float())
        h = s["h"].float()
        rstd = torch.rsqrt(h.square().mean(1) + s["eps"])
        y = h * rstd[:, None] * s["weight"].float()
        s["rstd"].copy_(rstd)
        if held:
            code, value, e = _encode(y, False)
            s["codes"].copy_(code)
            s["exps"].copy_(e)
            s["values"].copy_(value)
        else:
            s["y"].copy_(y)
    return [s["h"], s["rstd"], s["values"] if held else s["y"]]


def _pack(s):
    turned = "codes_t" in s
    if own:
        import zero_dp_sharded_amd as zs
        zs.zero_scaled_pack(s["x"], s["codes"], s["exps"], s.get("codes_t"), s.get("exps_t"))
        zs.zero_scaled_unpack(s["codes"], s["exps"], s["values"])
        if turned:
            zs.zero_scaled_unpack(s["codes_t"], s["exps_t"], s["values_t"])
    else:
        x = s["x"].float()
        for z, end in [(x, "")] + ([(x.t(), "_t")] if turned else []):
            code, value, e = _encode(z, s["case"]["square"])
            s["codes" + end].copy_(code)
            s["exps" + end].copy_(e)
            s["values" + end].copy_(value)
    return [s["values"]] + ([s["values_t"]] if turned else [])


def _product(s):
    if own:
        import zero_dp_sharded_amd as zs
        zs.zero_scaled_product(s["a"], s["a_exps"], s["b"], s["b_exps"], s["out"], s.get("bias"), s["space"])
        return s["out"]
    m, n, k = (s["case"][name] for name in "mnk")
    a = s["a"].float() * _scales(s["a_exps"], m, k, False, torch.float32)
    b = s["b"].float() * _scales(s["b_exps"], n, k, s["case"]["square"], torch.float32)
    out = a @ b.t()
    if "bias" in s:
        out = out + s["bias"].float()
    s["out"].copy_(out)
    return s["out"]


def _logits(s):
    return s["hidden"].float() @ s["weight"].float().t()


def _statistics(logits):
    """lse, the logits less lse, entropy."""
    top = logits.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(1))
    logp = logits - lse[:, None]
    return lse, logp, -(torch.exp(logp) * logp).sum(1)


def _logprobs(s):
    if s["case"]["grad"]:
        if own:
            import zero_dp_sharded_amd as zs
            zs.zero_token_logprobs_backward(s["hidden"], s["weight"], s["tokens"], s["lse"], s["entropy"], s["dlogprobs"], s["dentropy"],
                                            s["dhidden"], s["dweight"], s["space"], ignore_index=-100)
        else:
            given = s["tokens"] != -100
            at = torch.where(given, s["tokens"], 0)[:, None]
            logp = _logits(s) - s["lse"][:, None]
            d = torch.where(given, s["dlogprobs"], 0.0)
            p = torch.exp(logp)
            g = p * -d[:, None]
            if s["dentropy"] is not None:
                g -= s["dentropy"][:, None] * p * (logp + s["entropy"][:, None])
            g.scatter_add_(1, at, d[:, None])
            s["dhidden"].copy_(g @ s["weight"].float())
            s["dweight"].copy_(g.t() @ s["hidden"].float())
        return [s["dhidden"], s["dweight"]]
    if own:
        import zero_dp_sharded_amd as zs
        zs.zero_token_logprobs(s["hidden"], s["weight"], s["tokens"], s["logprobs"], s["lse"], s["entropy"], s["top_ids"], s["top_logprobs"],
                               s["space"], ignore_index=-100)
    else:
        logits = _logits(s)
        lse, logp, entropy = _statistics(logits)
        given = s["tokens"] != -100
        s["lse"].copy_(lse)
        s["logprobs"].copy_(torch.where(given, logp.gather(1, torch.where(given, s["tokens"], 0)[:, None])[:, 0], 0.0))
        if s["entropy"] is not None:
            s["entropy"].copy_(entropy)
        if s["top_ids"] is not None:
            ids = torch.arange(logits.shape[1], device=logits.device)
            for k in range(s["case"]["top"]):       # the largest, the lowest id of those alike, and on without it
                top = logits.amax(1, keepdim=True)
                at = torch.where(logits == top, ids, logits.shape[1]).amin(1)
                s["top_ids"][:, k] = at
                s["top_logprobs"][:, k] = logp.gather(1, at[:, None])[:, 0]
                logits.scatter_(1, at[:, None], -math.inf)
    outs = [s["logprobs"], s["lse"], s["entropy"], s["top_ids"], s["top_logprobs"]]
    return [x for x in outs if x is not None]


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "pack": _exact_pack, "product": _exact_product, "logprobs": _exact_logprobs}[case["op"]](case, s)


def _exact_code(x, square):
    """The values that x is held as: each block on the grid of 4 significant bits under its own power of two."""
    rows, width = x.shape
    out = torch.zeros_like(x)
    for c in range(0, width, BLOCK):
        part = x[:, c:c + BLOCK]
        big = part.abs().amax(1, keepdim=True)
        if square:
            big = torch.cat([big[r:r + BLOCK].amax().expand(min(BLOCK, rows - r), 1) for r in range(0, rows, BLOCK)])
        e = torch.ceil(torch.log2(big.clamp_min(1e-300) / LARGEST))
        e = e + (big > LARGEST * torch.exp2(e)).double() - (big <= LARGEST * torch.exp2(e - 1)).double()
        unit = torch.exp2(e.clamp(-100, 127))
        y = part.abs() / unit
        k = torch.floor(torch.log2(y.clamp_min(1e-300)))
        k = k + (y >= torch.exp2(k + 1)).double() - (y < torch.exp2(k)).double()
        grid = torch.exp2(k.clamp_min(-6.0)) / 8
        out[:, c:c + BLOCK] = torch.sign(part) * torch.round(y / grid) * grid * unit
    return out


def _exact_norm(case, s):
    w = s["weight"].double()
    if case["backward"]:
        # the gradient by the rows' own statistics: d/dh of sum(dy * w * h * rstd), rstd moving with h
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        along = (dy * w * h).sum(1, keepdim=True) / case["width"]
        return [s["dh"].double() + r * dy * w - r ** 3 * along * h, (dy * h * r).sum(0)]
    total = s["x"].double() + s["residual"].double()
    h = total.to(s["type"]).double()
    rstd = 1 / torch.sqrt((h * h).sum(1) / case["width"] + s["eps"])
    y = h * (w * rstd[:, None])
    return [total, rstd, _exact_code(y, False) if case["bytes"] else y]


def _exact_pack(case, s):
    x = s["x"].double()
    return [_exact_code(x, case["square"])] + ([_exact_code(x.t().contiguous(), case["square"])] if case["turned"] else [])


def _exact_product(case, s):
    m, n, k = case["m"], case["n"], case["k"]
    out = torch.zeros(m, n, dtype=torch.float64, device=s["a"].device)
    for c in range(0, k, 16 * BLOCK):          # block by block of the depth
        wide = min(16 * BLOCK, k - c)
        at = slice(c // BLOCK, -(-(c + wide) // BLOCK))
        a = s["a"][:, c:c + wide].double() * _scales(s["a_exps"][:, at], m, wide, False, torch.float64)
        b = s["b"][:, c:c + wide].double() * _scales(s["b_exps"][:, at], n, wide, case["square"], torch.float64)
        out += a @ b.t()
    return out + s["bias"].double() if case["bias"] else out


def _exact_logprobs(case, s):
    h, w, tokens, n = s["hidden"].double(), s["weight"].double(), s["tokens"], case["tokens"]
    given = tokens != -100
    at = torch.where(given, tokens, 0)[:, None]
    parts = []
    dw = torch.zeros_like(w)
    for a in range(0, n, 1024):
        rows = slice(a, min(a + 1024, n))
        z = h[rows] @ w.t()
        if case["grad"]:
            # p is exp(z - lse) by the row's own lse; the token's 1 - p by expm1, which does not cancel
            logp = z - s["lse"][rows].double()[:, None]
            p = torch.exp(logp)
            d = torch.where(given[rows], s["dlogprobs"][rows].double(), 0.0)[:, None]
            g = -d * p
            g.scatter_(1, at[rows], -d * torch.expm1(logp.gather(1, at[rows])))
            if case["entropy"]:
                g -= s["dentropy"][rows].double()[:, None] * p * (logp + s["entropy"][rows].double()[:, None])
            parts.append([g @ w])
            dw += g.t() @ h[rows]
            continue
        lse = torch.logsumexp(z, 1)
        logp = z - lse[:, None]
        row = [torch.where(given[rows], logp.gather(1, at[rows])[:, 0], 0.0), lse]
        if case["entropy"]:
            row.append(-(torch.exp(logp) * logp).sum(1))
        if case["top"]:
            ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["top"]]      # those alike by id
            row += [ids, logp.gather(1, ids)]
        parts.append(row)
    out = [torch.cat(x) for x in zip(*parts)]
    return out + [dw] if case["grad"] else out
