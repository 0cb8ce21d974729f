"""A small next-token model trained with the library's operators (needs a GPU).

    python -m zero_dp_sharded_amd.train_head [--steps 60] [--update adamw|bytes|owner]
            [--vocab 1009] [--width 192] [--tokens 512] [--storage fp16|bf16] [--seed 0]

    x = embed[token] ;  y = layer norm(x) ;  loss = cross entropy(y head^T, next token)

Each step runs zero_layernorm_forward, zero_vocab_loss with both gradients under the
loss scale, zero_layernorm_backward, and the update:
  adamw   zero_adamw_step over the model's tensors, fp32 moments
  bytes   the same with 8-bit moments
  owner   the tensors as one flat shard: zero_step_device with the gradients as its one
          contribution (the owner's step of a rank that holds everything; the same bits
          as adamw, whose arithmetic it is)
The tokens follow a fixed permutation nine times in ten, so the loss falls from log(vocab)
towards the chain's entropy.
"""
from __future__ import annotations

import argparse
import math
import sys
from typing import List

STORAGE = ("fp16", "bf16")


class Model:
    """The tensors of the model as views of flat arrays, each beginning at a multiple
    of 256 elements: fp32 masters, 2-byte params and gradients, moments."""

    def __init__(self, vocab: int, width: int, storage: str, device, seed: int):
        import torch
        self.dtype = {"fp16": torch.float16, "bf16": torch.bfloat16}[storage]
        shapes = {"embed": (vocab, width), "norm.weight": (width,), "norm.bias": (width,), "head": (vocab, width)}
        self.spans, at = {}, 0
        for name, shape in shapes.items():
            n = math.prod(shape)
            self.spans[name] = (at, n, shape)
            at += -(-n // 256) * 256
        self.total = at
        g = torch.Generator(device=device).manual_seed(seed)
        self.master = torch.zeros(at, device=device)
        for name, std in (("embed", 1.0), ("head", 0.02)):
            t = self.view(self.master, name)
            t.copy_(std * torch.randn(t.shape, generator=g, device=device))
        self.view(self.master, "norm.weight").fill_(1.0)
        self.param = self.master.to(self.dtype)
        self.grad = torch.zeros_like(self.param)

    def view(self, flat, name):
        at, n, shape = self.spans[name]
        return flat[at:at + n].view(shape)


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


def train(steps: int = 60, update: str = "adamw", vocab: int = 1009, width: int = 192, tokens: int = 512,
          storage: str = "fp16", seed: int = 0, lr: float = 2e-2, log=None):
    """Train, and return (losses of all steps, the model, the last step's result)."""
    import torch
    from . import (AdamHParams, LossScaleCfg, zero_layernorm_backward, zero_layernorm_forward,
                   zero_layernorm_workspace, zero_vocab_loss, zero_vocab_loss_workspace)
    if update not in ("adamw", "bytes", "owner"):
        raise ValueError(f"unknown update {update!r}")
    dev = torch.device("cuda", torch.cuda.current_device())
    model = Model(vocab, width, storage, dev, seed)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    follow = torch.randperm(vocab, generator=g, device=dev)
    ls = LossScaleCfg(init_scale=1024.0 if storage == "fp16" else 1.0, dynamic=1 if storage == "fp16" else 0)
    step, result, close = _handle(model, update, AdamHParams(lr=lr, beta2=0.95), ls)
    x = torch.empty(tokens, width, dtype=model.dtype, device=dev)
    y, dy, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(tokens, device=dev), torch.empty(tokens, device=dev)
    losses, loss = torch.empty(tokens, device=dev), torch.empty((), device=dev)
    norm_space = torch.empty(zero_layernorm_workspace(tokens, width), dtype=torch.uint8, device=dev)
    loss_space = torch.empty(zero_vocab_loss_workspace(tokens, vocab, width), dtype=torch.uint8, device=dev)
    part = lambda name: model.view(model.param, name)
    grad = lambda name: model.view(model.grad, name)
    table = torch.empty(vocab, width, device=dev)
    scale, seen, info = ls.init_scale, [], None
    try:
        for k in range(steps):
            token = torch.randint(0, vocab, (tokens,), generator=g, device=dev)
            stray = torch.rand(tokens, generator=g, device=dev) < 0.1
            target = torch.where(stray, torch.randint(0, vocab, (tokens,), generator=g, device=dev), follow[token])
            torch.index_select(part("embed"), 0, token, out=x)
            zero_layernorm_forward(x, part("norm.weight"), part("norm.bias"), y, mean, rstd)
            zero_vocab_loss(y, part("head"), target, losses, None, loss, dy, grad("head"), loss_space, grad_scale=scale)
            zero_layernorm_backward(dy, x, part("norm.weight"), mean, rstd, dx, grad("norm.weight"), grad("norm.bias"),
                                    norm_space)
            # rows of the embedding: those of one token added in order
            order = torch.argsort(token, stable=True)
            table.zero_()
            table.index_put_((token[order],), dx.float()[order], accumulate=True)
            grad("embed").copy_(table)
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


def main(argv: List[str] = None) -> int:
    ap = argparse.ArgumentParser(prog="python -m zero_dp_sharded_amd.train_head",
                                 description="a small next-token model on the library's operators")
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--update", choices=("adamw", "bytes", "owner"), default="adamw")
    ap.add_argument("--vocab", type=int, default=1009)
    ap.add_argument("--width", type=int, default=192)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--storage", choices=STORAGE, default="fp16")
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    seen, _, _ = train(a.steps, a.update, a.vocab, a.width, a.tokens, a.storage, a.seed, log=print)
    entropy = -(0.9 * math.log(0.9 + 0.1 / a.vocab) + 0.1 * math.log(0.1 / a.vocab))
    print(f"loss {seen[0]:.4f} -> {seen[-1]:.4f} (log vocab {math.log(a.vocab):.4f}, the chain's entropy {entropy:.4f})")
    return 0


if __name__ == "__main__":
    sys.exit(main())
