"""What the gradients of the dense projection are rounded to on the way: dU between the products, and
each result once; and that calls repeat their bits."""

import numpy as np
import pytest
import torch

from gpu_helpers import announce, f64, needs_gpu
from oracle import train_ops as to
from test_gpu_linear import Linear

pytestmark = [pytest.mark.gpu, needs_gpu]

# A bfloat16 value of one binade is rounded by at most 2^-8 of the binade's beginning either way, evenly spread:
# 2^-8 / sqrt(3) of the value in the mean square where all lie at its beginning, less elsewhere.
ONE = 2.0 ** -8 / 3 ** 0.5


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("T,K,N", [(777, 320, 448), (600, 512, 1024)])
def test_two_roundings(moe, T, K, N, act):
    announce(f"linear rounding T={T} K={K} N={N} {act}")
    c = Linear(moe, T, K, N, 131)
    runs = []
    for fill in (0x00, 0xFF, 0x5A):
        for n in ("ws", "wsb"):
            c.o[n].view(torch.uint8).fill_(fill)
        c.forward(act, True, True, True)
        c.backward(act)
        torch.cuda.synchronize()
        runs.append({n: c.o[n].clone() for n in ("u", "y", "dx", "dW", "db")})
    assert all(torch.equal(runs[0][n], r[n]) for r in runs[1:] for n in r)
    du = f64(c.dy) * to.act_slope(f64(c.o["u"]), act)
    rounded = f64(torch.from_numpy(du).to(torch.bfloat16))
    for name, product in (("dx", lambda v: v @ f64(c.W).T), ("dW", lambda v: f64(c.x).T @ v)):
        exact, inner = product(du), product(rounded)
        got = f64(c.o[name])
        off = lambda ref: np.linalg.norm(got - ref) / np.linalg.norm(ref)  # noqa: E731
        # from the exact product of the rounded dU: its own rounding alone, sums in float32 being far below it
        assert off(inner) < ONE, (name, off(inner))
        # from the formula: that and dU's, which are independent
        assert off(exact) < (off(inner) ** 2 + ONE ** 2) ** 0.5 * 1.02, (name, off(exact))
