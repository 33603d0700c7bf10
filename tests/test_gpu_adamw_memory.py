"""The optimizer's hold on the memory that it updates."""

import pytest
import torch

from gpu_helpers import announce, needs_gpu
from test_gpu_adamw import BF, F32, LR, params_of

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("bits", [8, 32])
def test_parameters_that_moved_are_refused(moe, bits):
    """A parameter with other memory than at the start: the step would write where something else may lie by now."""
    announce(f"adamw parameter with new memory bits={bits}")
    params, grads = params_of([(5000, BF, BF), (300, F32, F32)], 41)
    opt = moe.AdamW(params, lr=LR, bits=[bits, bits], max_norm=1.0)
    opt.step(grads)
    for i in (0, 1):
        old = params[i].data
        before = [t.clone() for t in (*params, *opt.m, *opt.v, opt.counter)]
        params[i].data = old.clone()
        with pytest.raises(RuntimeError, match="memory"):
            opt.step(grads)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((*params, *opt.m, *opt.v, opt.counter), before))
        params[i].data = old
    opt.step(grads)
    assert opt.counter.tolist() == [2, 0]


def test_moments_outlive_their_names(moe):
    """The buffers that a step writes stay the object's, whatever its attributes are made to name."""
    announce("adamw buffers kept")
    params, grads = params_of([(70000, BF, BF)], 42)
    opt = moe.AdamW(params, lr=LR, bits=8)
    with pytest.raises(TypeError):
        opt.m[0] = torch.zeros(70000, device="cuda")
    opt.step(grads)
    torch.cuda.synchronize()
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for k in ("master", "m", "m_scale", "v", "v_scale")
             for t in getattr(opt, k)]
    for k in ("master", "m", "m_scale", "v", "v_scale"):
        setattr(opt, k, ())
    fresh = [torch.empty(b - a, dtype=torch.uint8, device="cuda") for a, b in spans * 2]
    for t in fresh:
        assert all(t.data_ptr() + t.numel() <= lo or hi <= t.data_ptr() for lo, hi in spans)
    opt.step(grads)
    torch.cuda.synchronize()
    assert opt.counter.tolist() == [2, 0] and torch.isfinite(params[0].float()).all()


def test_steps_go_on_with_parameters_of_a_module(moe):
    """Parameters changed in place, or shared with a module, keep their memory and go on."""
    announce("adamw module parameters")
    m = torch.nn.Linear(64, 32, bias=False, device="cuda", dtype=F32)
    opt = moe.AdamW([m.weight], lr=LR)
    for _ in range(2):
        m.weight.grad = None
        m(torch.ones(4, 64, device="cuda")).sum().backward()
        opt.step([m.weight.grad])
        with torch.no_grad():
            m.weight.mul_(0.5)
    torch.cuda.synchronize()
    assert opt.counter.tolist() == [2, 0] and torch.isfinite(m.weight).all()
