"""What the optimizer's constructor refuses, before a step finds it."""

import pytest
import torch

from gpu_helpers import needs_gpu
from test_gpu_adamw import BF, F32, params_of

pytestmark = [pytest.mark.gpu, needs_gpu]


def test_factors(moe):
    params, grads = params_of([(300, F32, F32), (500, BF, BF)], 51)
    for bad in (-1.0, float("nan"), float("inf"), -1e-300):
        with pytest.raises(ValueError, match="parameter 0"):
            moe.AdamW(params, weight_decay=bad)
        with pytest.raises(ValueError, match="parameter 1"):
            moe.AdamW(params, lr_factor=[0.0, bad])
    opt = moe.AdamW(params, lr_factor=[0.0, 2.0], weight_decay=[0, 0.1])
    opt.step(grads)
    assert opt.counter.tolist() == [1, 0]


def test_alignment(moe):
    params, _ = params_of([(304, F32, F32), (512, BF, BF)], 52)
    with pytest.raises(moe.MoEError, match="parameter 1"):
        moe.AdamW([params[0], params[1][1:]])
    state = moe.AdamW(params).state
    wide = torch.zeros(308, device="cuda")
    for shift in (1, 2, 3):
        with pytest.raises(moe.MoEError, match="parameter 0"):
            moe.AdamW(params, state={**state, "v": [wide[shift:shift + 304], state["v"][1]]})
    opt = moe.AdamW([params[0][4:], params[1][8:]])
    assert opt.counter.tolist() == [0, 0]
    with pytest.raises(ValueError, match="expected 512"):
        moe.AdamW(params, state={**state, "v": [state["v"][0], wide]})


def test_state_that_is_no_tensor(moe):
    params, _ = params_of([(304, F32, F32), (512, BF, BF)], 53)
    state = moe.AdamW(params).state
    for name in ("m", "v"):
        for bad in ([0.0] * 304, 1.0):
            with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
                moe.AdamW(params, state={**state, name: [bad, state[name][1]]})
        with pytest.raises(ValueError, match=f"{name} is required"):
            moe.AdamW(params, state={**state, name: [None, state[name][1]]})
        with pytest.raises(ValueError, match="GPU"):
            moe.AdamW(params, state={**state, name: [state[name][0].cpu(), state[name][1]]})
