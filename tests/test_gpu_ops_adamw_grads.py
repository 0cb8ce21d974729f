"""Other gradients for an AdamW handle: what is refused, and how long the old ones live."""
import pytest
import torch

import zero_dp_sharded_amd as zs
from test_gpu_ops_adamw import DEV, HP, SIZES, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_overlap_what_the_step_writes_are_refused(bits):
    model = make(SIZES, ["fp32", "bf16"], bits, seed=4)
    n = len(SIZES)
    h = zs.zero_adamw_init(model.tensors, hp=HP, ls=zs.LossScaleCfg(dynamic=0), state_bits=bits)
    try:
        before = [a.clone() for a in model.arrays()]
        refused = []
        for k, x in enumerate(model.tensors):
            size = x.grad.numel()
            if size < 8:
                continue
            base = x.master if x.grad.dtype == torch.float32 else x.param
            refused.append((k, base))                                            # the array itself
            other = next(j for j in range(n - 1, -1, -1) if model.tensors[j].grad.dtype == x.grad.dtype and SIZES[j] > size) if size < 12289 else None
            if other is not None:                                                # inside another's
                y = model.tensors[other]
                refused.append((k, (y.master if x.grad.dtype == torch.float32 else y.param)[SIZES[other] - size:]))
        for k, grad in refused:
            grads = list(model.grads)
            grads[k] = grad
            with pytest.raises(zs.ZeroError, match="overlaps"):
                zs.zero_adamw_set_grads(h, grads)
        # nothing was taken: the step is the one of the first gradients
        zs.zero_adamw_set_grads(h, model.grads)
        zs.zero_adamw_step(h)
        assert not zs.zero_adamw_result(h).skipped
        again = make(SIZES, ["fp32", "bf16"], bits, seed=4)
        assert all(torch.equal(a, b) for a, b in zip(before, again.arrays()))
        k = zs.zero_adamw_init(again.tensors, hp=HP, ls=zs.LossScaleCfg(dynamic=0), state_bits=bits)
        zs.zero_adamw_step(k)
        torch.cuda.synchronize()
        zs.zero_adamw_destroy(k)
        assert all(torch.equal(a, b) for a, b in zip(model.arrays(), again.arrays()))
    finally:
        zs.zero_adamw_destroy(h)


def test_old_gradients_outlive_a_step_that_still_waits():
    """A step is enqueued on a stream that is busy, the handle gets other gradients, the old
    ones are let go, and their memory is asked for again on their own stream."""
    sizes = [70001, 4096, 300000]
    model, want = make(sizes, ["fp32"], 32, seed=9), make(sizes, ["fp32"], 32, seed=9)
    kw = dict(hp=HP, ls=zs.LossScaleCfg(dynamic=0))
    h, k = zs.zero_adamw_init(model.tensors, **kw), zs.zero_adamw_init(want.tensors, **kw)
    try:
        zs.zero_adamw_step(k)
        torch.cuda.synchronize()
        mine = [g.clone() for g in model.grads]
        zs.zero_adamw_set_grads(h, mine)
        places = {g.data_ptr() for g in mine}
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)
        zs.zero_adamw_step(h, stream=s)
        zs.zero_adamw_set_grads(h, model.grads, stream=s)
        del mine
        others = [torch.full((n,), float("nan"), device=DEV) for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        assert not places & {g.data_ptr() for g in others}
        assert all(torch.equal(a, b) for a, b in zip(model.arrays(), want.arrays()))
    finally:
        zs.zero_adamw_destroy(h)
        zs.zero_adamw_destroy(k)
