"""The 8-bit experts where tiles of a last round are cut over the workgroups: against
float64, and the parts' places in the workspace."""

import numpy as np
import pytest
import torch

import fp8_tiles_replica as fr
from ext_helpers import assert_within, f64, ffn_bound, quantized, randn
from gpu_helpers import announce, needs_gpu
from oracle import block_ops as ob
from test_gpu_ffn_fp8 import experts, groups

pytestmark = [pytest.mark.gpu, needs_gpu]

BF = torch.bfloat16
SLOT = fr.TILE * fr.TILE  # float32 of a part


@pytest.mark.parametrize("name,counts,d,de", fr.CASES, ids=[c[0] for c in fr.CASES])
def test_cut_tiles_against_float64(moe, monkeypatch, name, counts, d, de):
    announce(f"ffn fp8 cuts {name}")
    monkeypatch.setenv("MOE_FP8_TILES", "1")
    E, R = len(counts), sum(counts)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    cuts = fr.cuts(counts, de, d, cus)
    assert cuts
    p = moe.make_problem(R, d, E, 1, de, BF)
    n = min(R, 1500)  # rows are drawn from so many
    src = torch.arange(R, device="cuda") * 37 % n
    x8, xs, dec = quantized(moe, randn((n, d), 1.0, BF, 30))
    W1, W2 = randn((E, d, de), d ** -0.5, BF, 31), randn((E, de, d), de ** -0.5, BF, 32)
    q = experts(moe, p, W1, W2)
    off = groups(counts)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = torch.full((moe.moex_workspace_size(p, moe.MOEX_STAGE_FFN_FP8),), 0x7F, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0  # the workspace is laid out from here on
    y = [torch.full((R, d), float("nan"), dtype=BF, device="cuda") for _ in range(2)]
    for out in y:
        moe.moex_grouped_ffn_fp8(p, x8[src], xs[src], None, offsets, *q, out, ws)
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1])

    # exactly the parts of the cut tiles have gone through the workspace (its last region)
    slots = 2 * fr.workgroups(R, d, E, cus)
    part = ws[ws.numel() - 256 - slots * SLOT * 4:ws.numel() - 256].view(torch.int32).view(slots, SLOT)
    used = {p_.workgroup * 2 + p_.slot for c in cuts for p_ in c.parts}
    assert set(torch.nonzero((part != 0x7F7F7F7F).any(dim=1)).reshape(-1).tolist()) == used

    # rows: of every cut tile the first and last of each 32, and some of all others
    rows = {r for c in cuts for b in range(0, c.rows, 32)
            for r in (c.row0 + b, c.row0 + min(b + 31, c.rows - 1), c.row0 + min(b + 13, c.rows - 1))}
    rows |= set(np.random.default_rng(1).integers(0, R, 200).tolist()) | {o - 1 for o in off[1:] if o}
    rows = np.array(sorted(rows))
    few = np.searchsorted(rows, off)  # the groups of these rows alone
    w1, w2 = ob.weight_layout(f64(W1))[2], ob.weight_layout(f64(W2))[2]
    ref, bound = ffn_bound(dec[src.cpu().numpy()[rows]], few.tolist(), w1[:, :dec.shape[1]], w2, de)
    assert_within(name, f64(y[0])[rows], ref, bound)
    assert torch.isfinite(y[0]).all()
    # and every row, roughly: the other form's product of hidden rows that differ in codes at a border
    monkeypatch.setenv("MOE_FP8_TILES", "0")
    other = torch.empty_like(y[0])
    moe.moex_grouped_ffn_fp8(p, x8[src], xs[src], None, offsets, *q, other, ws)
    torch.cuda.synchronize()
    a, b = y[0].double(), other.double()
    assert bool(((a - b).norm(dim=1) <= 2.0 ** -6 * b.norm(dim=1)).all())
