"""MoETrainBlock: a step of norm, routed and dense experts, gradients and the optimizer,
against the same mathematics by float32 autograd, and as it is used (captured, on other
streams, without the dense expert)."""

import numpy as np
import pytest
import torch

from ext_helpers import HALF, randn
from gpu_helpers import announce, needs_gpu
from harness import make_inputs, scaled_config

pytestmark = [pytest.mark.gpu, needs_gpu]

BF, F32 = torch.bfloat16, torch.float32
T, D, E, K, DE, DD = 192, 256, 8, 2, 128, 320
EPS, COEF = 1e-6, 0.02


def make(moe, dense=True, bias=True, seed=1, **kw):
    cfg = scaled_config("fine_grained", T=T, d_model=D, E=E, k=K, d_expert=DE, suffix="train_block")
    inp = make_inputs(cfg, seed=seed, device="cuda")
    params = {"gain": (1 + 0.1 * randn((D,), 1.0, F32, seed)).to(BF), "w_router": randn((D, E), D ** -0.5, BF, seed + 5),
              "W1": inp["W1"], "W2": inp["W2"]}
    if bias:
        params["router_bias"] = randn((E,), 0.3, F32, seed + 6)
    if dense:
        params.update(V1=randn((D, DD), D ** -0.5, BF, seed + 7), c1=randn((DD,), 0.3, BF, seed + 8),
                      V2=randn((DD, D), DD ** -0.5, BF, seed + 9), c2=randn((D,), 0.3, BF, seed + 10))
    return params, moe.MoETrainBlock(T, D, E, K, DE, params, coef=COEF, eps=EPS, **kw)


@pytest.fixture(scope="module")
def data():
    return [randn((T, D), 1.0, BF, s) for s in (20, 21, 22, 23)]  # x, residual, dy, dh


def reference(params, x, res, dy, dh, block):
    """Gradients by autograd in float32 of the formulas, with the block's own routing."""
    leaves = {n: p.float().requires_grad_() for n, p in params.items()}
    xr = x.float().requires_grad_()
    h = xr + res.float()
    h.data.copy_(block.h.float())  # the rounded stream, as the norm takes it
    n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * leaves["gain"]
    logits = n @ leaves["w_router"] + (leaves["router_bias"] if "router_bias" in leaves else 0)
    prob = torch.softmax(logits, 1)
    idx = logits.topk(K, dim=1).indices
    y = 0
    for j in range(K):
        w1, w2 = leaves["W1"][idx[:, j]], leaves["W2"][idx[:, j]]
        a = torch.nn.functional.gelu((n[:, :, None] * w1).sum(1), approximate="tanh")
        y = y + prob.gather(1, idx[:, j:j + 1]) * (a[:, :, None] * w2).sum(1)
    if "V1" in leaves:
        y = y + torch.nn.functional.gelu(n @ leaves["V1"] + leaves["c1"], approximate="tanh") @ leaves["V2"] + leaves["c2"]
    counts = torch.zeros(E, device="cuda").index_add(0, idx.reshape(-1), torch.ones(T * K, device="cuda"))
    loss = COEF * E * (counts / (T * K) * prob.mean(0)).sum()
    ((y * dy.float()).sum() + (h * dh.float()).sum() + loss).backward()
    return y.detach(), xr.grad, {k: v.grad for k, v in leaves.items()}, float(loss), counts


@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_gradients_against_autograd(moe, data, dense, bias):
    """Rows are rounded to bfloat16 between the parts: n, u, a, the experts' rows, dU and dn each by half a step,
    2^-8 of a value, so a result after up to eight of them is within eight half steps in the norm."""
    announce(f"train block dense={dense} bias={bias}")
    params, block = make(moe, dense, bias)
    x, res, dy, dh = data
    y, h = block.forward(x, res)
    assert h is block.h and torch.equal(h, (x.float() + res.float()).to(BF))
    dx = block.backward(dy, dh)
    torch.cuda.synchronize()
    ry, rdx, rg, rloss, counts = reference(params, x, res, dy, dh, block)
    assert torch.equal(block.counts.float(), counts)
    for name, a, b in (("y", y, ry), ("dx", dx, rdx), *((n, block.grads[n], rg[n]) for n in params)):
        err = float((a.float().reshape(b.shape) - b).norm() / b.norm())
        assert err < 8 * HALF[BF], (name, err)
    assert abs(float(block.loss) - rloss) < 1e-3 * rloss


def test_steps_are_the_optimizers(moe, data):
    """step() is AdamW's on the block's gradients, matrices with decay and vectors without."""
    announce("train block step")
    params, block = make(moe, lr=1e-3, weight_decay=0.1, max_norm=0.5, bits=8, seed=3)
    copies = {n: p.clone() for n, p in params.items()}
    other = moe.AdamW([copies[n] for n in block.names], lr=1e-3, max_norm=0.5, bits=8,
                      weight_decay=[0.1 if copies[n].dim() > 1 else 0.0 for n in block.names])
    x, res, dy, dh = data
    for _ in range(3):
        block.forward(x, res)
        block.backward(dy, dh)
        norm = block.step()
        other.step([block.grads[n] for n in block.names])
        torch.cuda.synchronize()
        assert all(torch.equal(params[n], copies[n]) for n in params) and float(norm) == float(other.norm)
    assert block.optimizer.counter.tolist() == [3, 0]
    assert not torch.equal(params["W1"], make_inputs(scaled_config("fine_grained", T=T, d_model=D, E=E, k=K, d_expert=DE,
                                                                   suffix="train_block"), seed=1, device="cuda")["W1"])


def test_without_residual_and_masked(moe, data):
    announce("train block without residual, masked")
    _, block = make(moe, seed=4)
    x, _, dy, _ = data
    mask = (torch.arange(T, device="cuda") % 3 > 0).to(torch.uint8)
    y, h = block.forward(x)
    assert h is x
    dx = block.backward(dy, None, mask)
    torch.cuda.synchronize()
    assert torch.isfinite(y.float()).all() and torch.isfinite(dx.float()).all()
    assert int(block.counts.sum()) == int(mask.sum()) * K


def test_captured_steps(moe, data):
    """A captured step replayed gives the bits of eager steps."""
    announce("train block captured")
    x, res, dy, dh = data
    (pa, a), (pb, b) = (make(moe, lr=1e-3, max_norm=1.0, bits=8, seed=5) for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.forward(x, res)
        a.backward(dy, dh)
        a.step()
    for _ in range(4):
        g.replay()
        b.forward(x, res)
        b.backward(dy, dh)
        b.step()
        torch.cuda.synchronize()
        torch.randn(1000, device="cuda").sum().item()
        assert torch.equal(a.y, b.y) and torch.equal(a.dx, b.dx) and torch.equal(a.loss, b.loss)
        assert all(torch.equal(pa[n], pb[n]) and torch.equal(a.grads[n], b.grads[n]) for n in pa)


@pytest.mark.parametrize("how", ["argument", "handle", "current"])
def test_other_streams(moe, data, how):
    announce(f"train block on a side stream ({how})")
    x, res, dy, dh = data
    (pa, a), (pb, b) = (make(moe, lr=1e-3, max_norm=1.0, seed=6) for _ in range(2))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
        if how == "current":
            b.forward(x, res)
            b.backward(dy, dh)
            b.step()
    if how != "current":
        st = s if how == "argument" else s.cuda_stream
        b.forward(x, res, st)
        b.backward(dy, dh, None, st)
        b.step(st)
    assert not s.query()  # nothing of it waited
    a.forward(x, res)
    a.backward(dy, dh)
    a.step()
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a.y, b.y) and all(torch.equal(pa[n], pb[n]) for n in pa)


def test_memory_outlives_the_object(moe, data):
    """Dropped while a side stream's step is in flight: nothing else gets its memory before the step ends."""
    announce("train block dropped in flight")
    x, res, dy, dh = data
    params, block = make(moe, lr=1e-3, max_norm=1.0, bits=8, seed=7)
    o = block.optimizer
    mine = [t for t in (*vars(block).values(), *block.grads.values(), o.counter, o.lr_scale, o.norm, o.scale, o._ws, *o.master,
                        *o.m, *o.v, *o.m_scale, *o.v_scale) if isinstance(t, torch.Tensor)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in mine]
    sizes = [b - a for a, b in spans]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(500_000_000)
    block.forward(x, res, side)
    block.backward(dy, dh, None, side)
    block.step(side)
    del block, mine, o
    fresh = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes * 3]
    assert not side.query()
    for t in fresh:
        a, b = t.data_ptr(), t.data_ptr() + t.numel()
        assert all(b <= lo or hi <= a for lo, hi in spans)
    side.synchronize()


def test_refusals(moe, data):
    params, block = make(moe, seed=8)
    with pytest.raises(RuntimeError, match="without a forward"):
        block.backward(data[2])
    with pytest.raises(ValueError, match="unknown"):
        moe.MoETrainBlock(T, D, E, K, DE, {**params, "W3": params["W1"]})
    with pytest.raises(ValueError, match="W1 holds"):
        moe.MoETrainBlock(T, D, E, K, 2 * DE, params)
    with pytest.raises(TypeError):
        moe.MoETrainBlock(T, D, E, K, DE, {**params, "gain": params["gain"].float()})
    with pytest.raises(ValueError):
        block.forward(data[0][:10])
    with pytest.raises(moe.MoEError):
        block.forward(data[0], block.h)  # the residual stream over itself
