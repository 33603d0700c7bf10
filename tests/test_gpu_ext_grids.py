"""Batches whose launches need more threads than one grid dimension holds (2^32)."""

import pytest
import torch

from ext_helpers import randn
from gpu_helpers import announce, needs_gpu
from oracle import block_ops as ob

pytestmark = [pytest.mark.gpu, needs_gpu]

BF, F32 = torch.bfloat16, torch.float32


def test_norm_of_more_rows_than_one_grid_dimension_holds(moe):
    """2^26 rows of 64 and a few: each is the row of a small batch, bit for bit."""
    announce("norm 2^26 rows")
    T, d, n = (1 << 26) + 7, 64, 1009
    x, res, gain = randn((n, d), 1.0, BF, 1), randn((n, d), 1.0, BF, 2), randn((d,), 1.0, BF, 3)
    row = torch.arange(T, device="cuda") % n

    def run(x, res):
        p = moe.make_problem(x.shape[0], d, 1, 1, 64, BF)
        o = {"h": torch.empty_like(x), "y": torch.empty_like(x),
             "y8": torch.empty((p.T, ob.code_pitch(d)), dtype=torch.uint8, device="cuda"),
             "scale": torch.empty((p.T, ob.scale_pitch(d)), dtype=torch.uint8, device="cuda"),
             "r": torch.empty(p.T, dtype=F32, device="cuda")}
        moe.moex_add_rmsnorm(p, x, res, gain, 1e-5, o["h"], o["y"], o["y8"], o["scale"], o["r"])
        return o

    small, big = run(x, res), run(x[row], res[row])
    torch.cuda.synchronize()
    for key in small:
        step = 1 << 24  # in pieces: the expected rows take as much memory as the result
        for t in range(0, T, step):
            assert torch.equal(big[key][t:t + step], small[key][row[t:t + step]]), key
