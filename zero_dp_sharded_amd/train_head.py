"""A small next-token model trained with the library's operators (needs a GPU).

    python -m zero_dp_sharded_amd.train_head [--steps 60] [--update adamw|bytes|owner] [--body none|bytes]
            [--vocab 1009] [--width 192] [--tokens 512] [--storage fp16|bf16] [--seed 0]

    x = embed[token] ;  y = layer norm(x) ;  loss = cross entropy(y head^T, next token)

With --body bytes a layer in 8 bits lies between, with root-mean-square norms around it:

    s = x + rms norm(x) body^T ;  y = rms norm(s)

(zero_rmsnorm_forward gives the product its codes, the second one adds the residual; the products of
both directions are zero_scaled_product's, of what zero_scaled_pack gives).  Each step runs zero_layernorm_forward, zero_vocab_loss with both gradients under the
loss scale, zero_layernorm_backward, and the update:
  adamw   zero_adamw_step over the model's tensors, fp32 moments
  bytes   the same with 8-bit moments
  owner   the tensors as one flat shard: zero_step_device with the gradients as its one
          contribution (the owner's step of a rank that holds everything; the same bits
          as adamw, whose arithmetic it is)
The tokens follow a fixed permutation nine times in ten, so the loss falls from log(vocab)
towards the chain's entropy.  At the end the log probabilities of tokens not seen, the rows'
entropy and the alternatives are zero_token_logprobs'.
"""
from __future__ import annotations

import argparse
import math
import sys
from typing import List

STORAGE = ("fp16", "bf16")
BODIES = ("none", "bytes")


class Model:
    """The tensors of the model as views of flat arrays, each beginning at a multiple
    of 256 elements: fp32 masters, 2-byte params and gradients, moments."""

    def __init__(self, vocab: int, width: int, storage: str, device, seed: int, body: str = "none"):
        import torch
        self.dtype = {"fp16": torch.float16, "bf16": torch.bfloat16}[storage]
        shapes = {"embed": (vocab, width), "norm.weight": (width,), "norm.bias": (width,), "head": (vocab, width)}
        if body == "bytes":
            shapes = {"embed": (vocab, width), "norm.weight": (width,), "body": (width, width), "norm2.weight": (width,),
                      "head": (vocab, width)}
        self.spans, at = {}, 0
        for name, shape in shapes.items():
            n = math.prod(shape)
            self.spans[name] = (at, n, shape)
            at += -(-n // 256) * 256
        self.total = at
        g = torch.Generator(device=device).manual_seed(seed)
        self.master = torch.zeros(at, device=device)
        for name, std in (("embed", 1.0), ("head", 0.02), ("body", width ** -0.5)):
            if name in shapes:
                t = self.view(self.master, name)
                t.copy_(std * torch.randn(t.shape, generator=g, device=device))
        for name in ("norm.weight", "norm2.weight"):
            if name in shapes:
                self.view(self.master, name).fill_(1.0)
        self.param = self.master.to(self.dtype)
        self.grad = torch.zeros_like(self.param)

    def view(self, flat, name):
        at, n, shape = self.spans[name]
        return flat[at:at + n].view(shape)

    def part(self, name):
        return self.view(self.param, name)

    def grad_of(self, name):
        return self.view(self.grad, name)


def _handle(model: Model, update: str, hp, ls):
    """(step(), result(), close()) of the chosen update."""
    import torch
    from . import (AdamWTensor, zero_adamw_destroy, zero_adamw_init, zero_adamw_result, zero_adamw_step,
                   zero_device_begin, zero_device_end, zero_shard_destroy, zero_shard_init, zero_step_device)
    if update == "owner":
        m, v = torch.zeros_like(model.master), torch.zeros_like(model.master)
        shard = torch.empty_like(model.grad)
        h = zero_shard_init(model.master, m, v, shard, model.param, psi=model.total, nd=1, rank=0,
                            bucket_elems=model.total, hp=hp, ls=ls)
        zero_device_begin(h)

        def result():
            info = zero_device_end(h)
            zero_device_begin(h)
            return info

        def close(arrays=(m, v, shard)):      # (they must outlive the handle)
            zero_device_end(h)
            zero_shard_destroy(h)

        return lambda: zero_step_device(h, [model.grad]), result, close
    bits = 8 if update == "bytes" else 32
    kind = torch.uint8 if bits == 8 else torch.float32
    state = [torch.zeros(model.total, dtype=kind, device=model.master.device) for _ in range(2)]
    exps = [torch.zeros(model.total // 256, dtype=torch.int8, device=model.master.device) for _ in range(2)]
    tensors = []
    for name, (at, n, _) in model.spans.items():
        blocks = slice(at // 256, at // 256 + -(-n // 256))
        extra = {} if bits == 32 else {"exp_avg_exp": exps[0][blocks], "exp_avg_sq_exp": exps[1][blocks]}
        tensors.append(AdamWTensor(model.grad[at:at + n], model.master[at:at + n], model.param[at:at + n],
                                   state[0][at:at + n], state[1][at:at + n], **extra))
    h = zero_adamw_init(tensors, hp=hp, ls=ls, state_bits=bits, seed=1)
    return lambda: zero_adamw_step(h), lambda: zero_adamw_result(h), lambda: zero_adamw_destroy(h)


class _Plain:
    """y = layer norm(x), and back."""

    def __init__(self, model: Model, tokens: int, width: int, device):
        import torch
        from . import zero_layernorm_workspace
        self.model = model
        self.y = torch.empty(tokens, width, dtype=model.dtype, device=device)
        self.mean, self.rstd = torch.empty(tokens, device=device), torch.empty(tokens, device=device)
        self.space = torch.empty(zero_layernorm_workspace(tokens, width), dtype=torch.uint8, device=device)

    def forward(self, x):
        from . import zero_layernorm_forward
        zero_layernorm_forward(x, self.model.part("norm.weight"), self.model.part("norm.bias"), self.y, self.mean, self.rstd)
        return self.y

    def backward(self, x, dy, dx):
        from . import zero_layernorm_backward
        m = self.model
        zero_layernorm_backward(dy, x, m.part("norm.weight"), self.mean, self.rstd, dx, m.grad_of("norm.weight"), m.grad_of("norm.bias"),
                                self.space)


class _Bytes:
    """s = x + rms norm(x) body^T in 8 bits, y = rms norm(s), and back."""

    def __init__(self, model: Model, tokens: int, width: int, device):
        import torch
        from . import zero_rmsnorm_workspace, zero_scaled_product_workspace
        self.model = model
        new = lambda: torch.empty(tokens, width, dtype=model.dtype, device=device)
        self.y1, self.u, self.s, self.y, self.ds, self.dy1 = (new() for _ in range(6))
        self.rstd = [torch.empty(tokens, device=device) for _ in range(2)]

        def held(rows, columns, square=False):
            blocks = lambda n: -(-n // 128)
            return (torch.empty(rows, columns, dtype=torch.float8_e4m3fn, device=device),
                    torch.empty(blocks(rows) if square else rows, blocks(columns), dtype=torch.uint8, device=device))

        self.y1_held, self.y1_turned = held(tokens, width), held(width, tokens)
        self.w_held, self.w_turned = held(width, width, True), held(width, width, True)
        self.du_held, self.du_turned = held(tokens, width), held(width, tokens)
        self.norm_space = torch.empty(zero_rmsnorm_workspace(tokens, width), dtype=torch.uint8, device=device)
        sizes = [(tokens, width, width), (width, width, tokens)]
        self.space = torch.empty(max(zero_scaled_product_workspace(*n, model.dtype) for n in sizes), dtype=torch.uint8, device=device)

    def forward(self, x):
        from . import zero_rmsnorm_forward, zero_scaled_pack, zero_scaled_product
        m = self.model
        zero_rmsnorm_forward(x, None, m.part("norm.weight"), None, self.y1, self.rstd[0], *self.y1_held)
        zero_scaled_pack(m.part("body"), *self.w_held, *self.w_turned)
        zero_scaled_product(*self.y1_held, *self.w_held, self.u, None, self.space)
        zero_rmsnorm_forward(self.u, x, m.part("norm2.weight"), self.s, self.y, self.rstd[1])
        return self.y

    def backward(self, x, dy, dx):
        from . import zero_rmsnorm_backward, zero_scaled_pack, zero_scaled_product
        m = self.model
        zero_rmsnorm_backward(dy, self.s, m.part("norm2.weight"), self.rstd[1], self.ds, None, m.grad_of("norm2.weight"), self.norm_space)
        zero_scaled_pack(self.ds, *self.du_held, *self.du_turned)
        zero_scaled_pack(self.y1, codes_t=self.y1_turned[0], exps_t=self.y1_turned[1])
        zero_scaled_product(*self.du_turned, *self.y1_turned, m.grad_of("body"), None, self.space)
        zero_scaled_product(*self.du_held, *self.w_turned, self.dy1, None, self.space)
        zero_rmsnorm_backward(self.dy1, x, m.part("norm.weight"), self.rstd[0], dx, self.ds, m.grad_of("norm.weight"), self.norm_space)


def _batch(tokens: int, vocab: int, follow, g, device):
    """Tokens and what follows them: a fixed permutation nine times in ten."""
    import torch
    token = torch.randint(0, vocab, (tokens,), generator=g, device=device)
    stray = torch.rand(tokens, generator=g, device=device) < 0.1
    return token, torch.where(stray, torch.randint(0, vocab, (tokens,), generator=g, device=device), follow[token])


def train(steps: int = 60, update: str = "adamw", vocab: int = 1009, width: int = 192, tokens: int = 512,
          storage: str = "fp16", seed: int = 0, lr: float = 2e-2, log=None, body: str = "none"):
    """Train, and return (losses of all steps, the model, the last step's result)."""
    import torch
    from . import AdamHParams, LossScaleCfg, zero_vocab_loss, zero_vocab_loss_workspace
    if update not in ("adamw", "bytes", "owner"):
        raise ValueError(f"unknown update {update!r}")
    if body not in BODIES:
        raise ValueError(f"unknown body {body!r}")
    dev = torch.device("cuda", torch.cuda.current_device())
    model = Model(vocab, width, storage, dev, seed, body)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    follow = torch.randperm(vocab, generator=g, device=dev)
    ls = LossScaleCfg(init_scale=1024.0 if storage == "fp16" else 1.0, dynamic=1 if storage == "fp16" else 0)
    step, result, close = _handle(model, update, AdamHParams(lr=lr, beta2=0.95), ls)
    layers = (_Bytes if body == "bytes" else _Plain)(model, tokens, width, dev)
    model.layers, model.follow = layers, follow
    x = torch.empty(tokens, width, dtype=model.dtype, device=dev)
    dy, dx = torch.empty_like(x), torch.empty_like(x)
    losses, loss = torch.empty(tokens, device=dev), torch.empty((), device=dev)
    loss_space = torch.empty(zero_vocab_loss_workspace(tokens, vocab, width), dtype=torch.uint8, device=dev)
    table = torch.empty(vocab, width, device=dev)
    scale, seen, info = ls.init_scale, [], None
    try:
        for k in range(steps):
            token, target = _batch(tokens, vocab, follow, g, dev)
            torch.index_select(model.part("embed"), 0, token, out=x)
            y = layers.forward(x)
            zero_vocab_loss(y, model.part("head"), target, losses, None, loss, dy, model.grad_of("head"), loss_space, grad_scale=scale)
            layers.backward(x, dy, dx)
            # rows of the embedding: those of one token added in order
            order = torch.argsort(token, stable=True)
            table.zero_()
            table.index_put_((token[order],), dx.float()[order], accumulate=True)
            model.grad_of("embed").copy_(table)
            step()
            info = result()            # (waits: the next step's loss scale is in it)
            scale = info.scale_next
            seen.append(loss.item())
            if log is not None and (k % 10 == 0 or k == steps - 1):
                log(f"step {k:4d}  loss {seen[-1]:.4f}  norm {info.grad_norm:.4g}  scale {info.scale_used:g}"
                    f"{'  skipped' if info.skipped else ''}")
    finally:
        close()
    return seen, model, info


def evaluate(model: Model, top: int = 5, seed: int = 1):
    """Of as many tokens as a step has, not trained on: (mean log probability of what follows, mean entropy, share of
    those that follow among the `top` alternatives)."""
    import torch
    from . import zero_token_logprobs, zero_token_logprobs_workspace
    layers, head = model.layers, model.part("head")
    vocab, width = head.shape
    tokens, dev = layers.y.shape[0], head.device
    g = torch.Generator(device=dev).manual_seed(1000003 + seed)
    token, target = _batch(tokens, vocab, model.follow, g, dev)
    y = layers.forward(model.part("embed")[token])
    logp, lse, entropy = (torch.empty(tokens, device=dev) for _ in range(3))
    ids, scores = torch.empty(tokens, top, dtype=torch.int64, device=dev), torch.empty(tokens, top, device=dev)
    space = torch.empty(zero_token_logprobs_workspace(tokens, vocab, width, top=top), dtype=torch.uint8, device=dev)
    zero_token_logprobs(y, head, target, logp, lse, entropy, ids, scores, space)
    return logp.mean().item(), entropy.mean().item(), (ids == target[:, None]).any(1).float().mean().item()


def main(argv: List[str] = None) -> int:
    ap = argparse.ArgumentParser(prog="python -m zero_dp_sharded_amd.train_head",
                                 description="a small next-token model on the library's operators")
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--update", choices=("adamw", "bytes", "owner"), default="adamw")
    ap.add_argument("--body", choices=BODIES, default="none")
    ap.add_argument("--vocab", type=int, default=1009)
    ap.add_argument("--width", type=int, default=192)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--storage", choices=STORAGE, default="fp16")
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    seen, model, _ = train(a.steps, a.update, a.vocab, a.width, a.tokens, a.storage, a.seed, log=print, body=a.body)
    entropy = -(0.9 * math.log(0.9 + 0.1 / a.vocab) + 0.1 * math.log(0.1 / a.vocab))
    print(f"loss {seen[0]:.4f} -> {seen[-1]:.4f} (log vocab {math.log(a.vocab):.4f}, the chain's entropy {entropy:.4f})")
    logp, spread, among = evaluate(model, top=min(5, a.vocab))
    print(f"not seen: log probability {logp:.4f}, entropy {spread:.4f}, among 5 alternatives {100 * among:.1f}%")
    return 0


if __name__ == "__main__":
    sys.exit(main())
