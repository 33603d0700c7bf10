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


def test_experts_of_more_pieces_than_one_grid_dimension_holds(moe, monkeypatch):
    """Narrow experts, wide rows: the second product has 2^23 pieces of 512 threads and a
    few. Each row is that of its token and expert in a small call, bit for bit."""
    announce("experts 2^23 pieces")
    monkeypatch.setenv("MOE_FP8_TILES", "0")
    T, d, E, k, de, n = 262000, 8192, 64, 8, 128, 37
    W1, W2 = randn((E, d, de), d ** -0.5, BF, 4), randn((E, de, d), de ** -0.5, BF, 5)
    p = moe.make_problem(T, d, E, k, de, BF)
    q = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in moe.expert_shapes(p)]
    moe.moex_quantize_experts(p, W1, W2, *q)
    x = randn((n, d), 1.0, BF, 6)
    x8 = torch.empty((n, ob.code_pitch(d)), dtype=torch.uint8, device="cuda")
    xs = torch.empty((n, ob.scale_pitch(d)), dtype=torch.uint8, device="cuda")
    moe.moex_quantize_rows(moe.make_problem(n, d, 1, 1, 64, BF), x, x8, xs)

    def run(p, x8, xs, perm, off):
        y = torch.empty((p.T * p.k, d), dtype=BF, device="cuda")
        ws = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_FFN_FP8), dtype=torch.uint8, device="cuda")
        moe.moex_grouped_ffn_fp8(p, x8, xs, perm, off, *q, y, ws)
        return y

    R = T * k
    row = torch.arange(T, device="cuda") % n
    # 41 rows of every expert but the last, which has all others: its last rows are the launch's last
    off = torch.tensor([41 * e for e in range(E)] + [R], dtype=torch.int32, device="cuda")
    perm = (torch.arange(R, device="cuda") * 7 % T).to(torch.int32)
    big = run(p, x8[row], xs[row], perm, off)
    small = run(moe.make_problem(n, d, E, E, de, BF), x8, xs,
                (torch.arange(n * E, device="cuda") % n).to(torch.int32),
                torch.arange(E + 1, device="cuda", dtype=torch.int32) * n)
    torch.cuda.synchronize()
    e = torch.searchsorted(off[1:].contiguous(), torch.arange(R, device="cuda", dtype=torch.int32), right=True)
    want = e * n + row[perm.long()]
    for r in range(0, R, 1 << 17):
        assert torch.equal(big[r:r + (1 << 17)], small[want[r:r + (1 << 17)]])
