"""MoEBlockFP8 on streams other than the one it was made on."""

import pytest
import torch

from ext_helpers import randn
from gpu_helpers import announce, needs_gpu
from harness import make_inputs, scaled_config

pytestmark = [pytest.mark.gpu, needs_gpu]

BF = torch.bfloat16
T, D, E, K, DE = 70, 320, 8, 2, 448
DELAY = 500_000_000  # cycles of a kernel that only waits, 0.2 s: far longer than a constructor or a call takes


@pytest.fixture(scope="module")
def inputs():
    cfg = scaled_config("fine_grained", T=T, d_model=D, E=E, k=K, d_expert=DE, suffix="streams")
    inp = make_inputs(cfg, seed=3, device="cuda")
    return {"w": (randn((D,), 1.0, BF, 1), inp["w_router"], inp["W1"], inp["W2"]),
            "x": randn((T, D), 1.0, BF, 2), "res": randn((T, D), 1.0, BF, 3)}


@pytest.fixture(scope="module")
def want(moe, inputs):
    y, h = moe.MoEBlockFP8(T, D, E, K, DE, *inputs["w"])(inputs["x"], inputs["res"])
    torch.cuda.synchronize()
    return y.clone(), h.clone()


def made(moe, inputs, stream=None):
    return moe.MoEBlockFP8(T, D, E, K, DE, *inputs["w"], stream=stream)


@pytest.mark.parametrize("how", ["argument", "handle", "current"])
def test_ready_for_any_stream(moe, inputs, want, how):
    """The weights are quantised when the constructor returns, whatever its stream was busy with."""
    announce(f"block made on a busy stream ({how})")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    a.wait_stream(torch.cuda.current_stream())
    b.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(a):
        torch.cuda._sleep(DELAY)
        if how == "current":
            block = made(moe, inputs)
    if how != "current":
        block = made(moe, inputs, a if how == "argument" else a.cuda_stream)
    assert a.query()
    y, h = block(inputs["x"], inputs["res"], b)
    b.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("how", ["argument", "current"])
def test_memory_outlives_the_object(moe, inputs, how):
    """Dropped while a side stream's call is in flight: nothing else gets its memory before the call ends."""
    announce(f"block dropped in flight ({how})")
    side = torch.cuda.Stream()
    block = made(moe, inputs)
    mine = [block.ws, block.y, block.h, block.normed, block.x8, block.x_scale, *block.experts]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in mine]
    sizes = [b - a for a, b in spans]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
        if how == "current":
            block(inputs["x"], inputs["res"])
    if how == "argument":
        block(inputs["x"], inputs["res"], side)
    del block, mine
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes * 4]
    assert not side.query()  # the call was still waiting
    for t in new:
        a, b = t.data_ptr(), t.data_ptr() + t.numel()
        assert all(b <= lo or hi <= a for lo, hi in spans)
    side.synchronize()


def test_zero_handle_is_the_default_stream(moe, inputs, want):
    announce("block on handle 0")
    y, h = made(moe, inputs, 0)(inputs["x"], inputs["res"], 0)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])


def test_captured_call_replays(moe, inputs, want):
    """Captured on another stream than the constructor's, replayed on new inputs."""
    announce("block captured")
    block, eager = made(moe, inputs), made(moe, inputs)
    x, res = inputs["x"].clone(), inputs["res"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = block(x, res)
    for seed in (10, 20, 30):
        x.copy_(randn((T, D), 1.0, BF, seed))
        res.copy_(randn((T, D), 1.0, BF, seed + 1))
        graph.replay()
        torch.cuda.synchronize()
        ye, he = eager(x, res)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(h, he)


def test_refusals_come_first(moe, inputs):
    w = list(inputs["w"])
    w[2] = w[2].cpu()
    with pytest.raises(ValueError, match="GPU"):
        moe.MoEBlockFP8(T, D, E, K, DE, *w)


def test_made_inside_a_capture(moe, inputs, want):
    """Then the graph lays the weights out again at every replay."""
    announce("block made in a capture")
    gain, wr, W1, W2 = inputs["w"]
    w1, w2 = W1.clone(), W2.clone()
    made(moe, inputs)(inputs["x"], inputs["res"])  # kernels loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = moe.MoEBlockFP8(T, D, E, K, DE, gain, wr, w1, w2)(inputs["x"], inputs["res"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    w2.mul_(2)  # exact in 8 bits too: the scales double, and so does every product
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.float(), 2 * want[0].float())
    w2.copy_(W2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])
