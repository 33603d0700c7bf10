"""MoETrainBlock's backward pass called again for the same forward call."""

import pytest
import torch

from ext_helpers import randn
from gpu_helpers import announce, needs_gpu
from test_gpu_train_block import BF, D, T, make

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("captured", [True, False])
def test_backward_again_with_another_gradient(moe, dense, captured):
    """Each backward call gives the bits of one that is the first after its forward call."""
    announce(f"train block: two backward calls, dense={dense} captured={captured}")
    x, res, dy, dh, dy2, dh2 = (randn((T, D), 1.0, BF, s) for s in range(71, 77))
    (pa, a), (_, b) = (make(moe, dense, seed=9) for _ in range(2))
    mask = (torch.arange(T, device="cuda") % 5 > 0).to(torch.uint8)

    def outputs(block):
        return [t.clone() for t in (block.dx, block.loss, block.counts, *block.grads.values())]

    want = []
    for g, h, m in ((dy, dh, None), (dy2, dh2, mask), (dy, dh, None)):
        b.forward(x, res)
        b.backward(g, h, m)
        want.append(outputs(b))
    a.forward(x, res)
    if captured:
        graphs = []
        for g, h, m in ((dy, dh, None), (dy2, dh2, mask)):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                a.backward(g, h, m)
        runs = [graphs[0].replay, graphs[1].replay, graphs[0].replay]
    else:
        runs = [lambda: a.backward(dy, dh), lambda: a.backward(dy2, dh2, mask), lambda: a.backward(dy, dh)]
    for run, w in zip(runs, want):
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outputs(a), w))
    assert not torch.equal(want[0][0], want[1][0]) and torch.equal(want[0][0], want[2][0])
