"""Clipping and the guard against gradients that are not finite, for every max_norm.

An infinite max_norm asks for the norm and the guard without clipping.
"""

import numpy as np
import pytest
import torch

from gpu_helpers import U32, announce, f64, needs_gpu
from test_gpu_adamw import B1, B2, BF, EPS, F32, LR, WD, Mirror, params_of

pytestmark = [pytest.mark.gpu, needs_gpu]

INF = float("inf")


def two_calls(moe, opt, grads):
    """moet_grad_norm and moet_adamw with its factor, on the buffers of `opt`."""
    for e, g in zip(opt._entries, grads):
        moe.set_grad(e, g, 0)
    moe.moet_grad_norm(opt._list, opt.max_norm, opt.norm, opt.scale, opt._ws)
    moe.moet_adamw(opt._list, moe.AdamWOptions(opt.lr, *opt.betas, opt.eps, opt.seed), opt.counter, None, opt.scale)


def everything(params, o):
    return [t for t in (*params, *o.master, *o.m, *o.v, *o.m_scale, *o.v_scale, o.counter) if t is not None]


@pytest.mark.parametrize("max_norm", [1.0, 1e300, INF])
@pytest.mark.parametrize("bad", [float("nan"), INF, -INF])
@pytest.mark.parametrize("calls", [1, 2])
def test_no_max_norm_takes_a_step_of_them(moe, bad, max_norm, calls):
    announce(f"adamw skips {bad} max_norm={max_norm} calls={calls}")
    params, grads = params_of([(5000, BF, BF), (33, F32, F32)], 4)
    opt = moe.AdamW(params, bits=[8, 32], max_norm=max_norm)
    step = opt.step if calls == 1 else lambda g: two_calls(moe, opt, g)
    step(grads)
    before = [t.clone() for t in everything(params, opt)]
    grads[0][4321] = bad
    step(grads)
    torch.cuda.synchronize()
    assert torch.isnan(opt.scale).item() and not torch.isfinite(opt.norm).item()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(everything(params, opt), before))
    grads[0][4321] = 0.0
    step(grads)
    assert opt.counter.tolist() == [2, 0] and float(opt.scale) == (1.0 if max_norm > 1 else opt.scale.item())


def test_norm_past_float32_without_clipping(moe):
    """A norm that float32 does not hold is finite all the same: its factor is 1 and the step is taken."""
    announce("grad norm of 3e39, max_norm inf")
    p, g = torch.full((100,), 2.0, device="cuda"), torch.full((100,), 3e38, device="cuda")
    opt = moe.AdamW([p], lr=LR, weight_decay=0.0, max_norm=INF)
    norm = opt.step([g])
    torch.cuda.synchronize()
    assert torch.isinf(norm).item() and float(opt.scale) == 1.0 and opt.counter.tolist() == [1, 0]
    # v is past float32: a move by nothing
    assert bool((p == 2.0).all()) and torch.isfinite(opt.m[0]).all()


@pytest.mark.parametrize("max_norm,clips", [(0.5, True), (1e6, False), (INF, False)])
@pytest.mark.parametrize("calls", [1, 2])
def test_factor_is_one_or_the_ratio(moe, max_norm, clips, calls):
    announce(f"adamw factor of max_norm={max_norm} calls={calls}")
    params, grads = params_of([(5000, BF, BF), (33, F32, F32)], 3)
    total = np.sqrt(sum(np.sum(f64(g) ** 2) for g in grads))
    assert (total > max_norm) == clips
    opt = moe.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, bits=8, max_norm=max_norm)
    ref = Mirror(opt)
    ref.before()
    if calls == 1:
        opt.step(grads)
    else:
        for d, e in zip((WD, WD), opt._entries):
            assert e.weight_decay == d
        two_calls(moe, opt, grads)
    torch.cuda.synchronize()
    want = max_norm / total if clips else 1.0
    # the sum of squares in 64 bits and one rounding to float32
    assert abs(float(opt.scale) - want) <= (2 * U32 * want if clips else 0.0)
    ref.check(grads, scale=np.float32(opt.scale.item()))
