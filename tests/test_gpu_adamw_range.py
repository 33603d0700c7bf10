"""Moments at the ends of their types' ranges, and factors beta next to 1, against float64."""

import numpy as np
import pytest
import torch

from ext_helpers import assert_within, gen
from gpu_helpers import U32, announce, f64, needs_gpu
from oracle import train_ops as to
from test_gpu_adamw import B1, B2, BF, EPS, F32, LR

pytestmark = [pytest.mark.gpu, needs_gpu]

# Largest second moment of each block of 128. Float32 ends at 3.4e38; the codes, 57344 2^120, at 7.62e40.
TOPS = [1e36, 3.3e38, 3.5e38, 5.9e38, 6.0e38, 1e39, 3.3e39, 1e40, 4.1e40, 7.5e40, 8e40, 1e42]


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("gt", [F32, BF])
def test_second_moments_past_float32(moe, gt):
    announce(f"adamw second moments past float32 {gt}")
    n = 128 * len(TOPS)
    spread = torch.exp2(-12 * torch.rand((len(TOPS), 128), generator=gen(31), device="cuda"))
    spread[:, 17] = 1.0
    g = (spread * torch.tensor([(v / (1 - B2)) ** 0.5 for v in TOPS], device="cuda")[:, None]).reshape(-1).to(gt)
    p = torch.full((n,), 2.0, device="cuda")
    opt = moe.AdamW([p], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.0, bits=[8], seed=5)
    opt.step([g])
    torch.cuda.synchronize()
    x = f64(g)
    m, v = (1 - B1) * x, ((1 - B2) * x) * x
    r = to.draws(n, 5, 1, 0)
    for name, val, rr, c, s, tab in (("m", m, r & 0xFFFF, opt.m[0], opt.m_scale[0], to.E4M3_POS),
                                     ("v", v, r >> 16, opt.v[0], opt.v_scale[0], to.E5M2_POS)):
        want, e = to.round_stochastic(val, rr, tab, name == "v")
        assert np.array_equal(s.cpu().numpy().astype(np.int64) - 127, e), name
        assert np.array_equal(codes(c), want), name
    held = v <= 57344 * 2.0 ** 120
    assert held[:128 * 10].all() and not held[-128 * 2:].all()
    assert np.array_equal(codes(opt.v[0]) != 0x7F, held)
    # the move is made in float32, which does not hold the larger ones: such a value moves by nothing
    far = torch.from_numpy(v > 3.5e38).cuda()
    assert bool((p[far] == 2.0).all()) and torch.isfinite(p).all()
    opt.step([torch.zeros_like(g)])
    torch.cuda.synchronize()
    assert torch.equal(torch.isfinite(p), torch.from_numpy(held).cuda())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_blocks_with_what_is_not_finite(moe, bad):
    """A NaN is left out of its block's scale, an infinity gives its block the largest one; each becomes a NaN code."""
    announce(f"adamw scale of a block with {bad}")
    n = 384
    g = torch.randn(n, generator=gen(32), device="cuda")
    g[5], g[130] = bad, bad
    p = torch.zeros(n, device="cuda")
    opt = moe.AdamW([p], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.0, bits=[8], seed=6)
    opt.step([g])
    torch.cuda.synchronize()
    x = f64(g)
    r = to.draws(n, 6, 1, 0)
    lost = ~np.isfinite(x)
    for name, val, rr, c, s, tab in (("m", (1 - B1) * x, r & 0xFFFF, opt.m[0], opt.m_scale[0], to.E4M3_POS),
                                     ("v", ((1 - B2) * x) * x, r >> 16, opt.v[0], opt.v_scale[0], to.E5M2_POS)):
        want, e = to.round_stochastic(val, rr, tab, name == "v")
        assert np.array_equal(s.cpu().numpy().astype(np.int64) - 127, e), name
        assert np.isnan(bad) or e.tolist() == [120, 120, e[2]]
        assert np.array_equal(codes(c)[~lost], want[~lost]) and (codes(c)[lost] & 0x7F == 0x7F).all(), name
    assert np.array_equal(np.isfinite(f64(p)), ~lost)


@pytest.mark.parametrize("betas", [(1 - 1e-9, 1 - 1e-12), (1 - 2.0 ** -53, 1 - 2.0 ** -53), (1 - 1e-6, 1 - 1e-8),
                                   (0.0, 1 - 1e-10), (0.999999, 0.0)])
@pytest.mark.parametrize("taken", [0, 1, 12345])
def test_factors_next_to_one(moe, betas, taken):
    """The corrections 1 - beta^t are good to float32 for every beta below 1 and every step."""
    announce(f"adamw betas={betas} after {taken} steps")
    n = 1000
    g = torch.randn(n, generator=gen(33), device="cuda")
    p = torch.randn(n, generator=gen(34), device="cuda")
    opt = moe.AdamW([p], lr=LR, betas=betas, eps=EPS, weight_decay=0.0)
    opt.counter[0] = taken
    # the moments that as many steps of unit gradients would have left, so that a move is about lr
    for t, b in ((opt.m[0], betas[0]), (opt.v[0], betas[1])):
        t.fill_(-np.expm1(taken * np.log(b)) if b and taken else 0.0)
    before, m, v = f64(p), f64(opt.m[0]), f64(opt.v[0])
    opt.step([g])
    torch.cuda.synchronize()
    want = to.adamw(before, f64(g), m, v, taken + 1, LR, *betas, EPS, 0.0)[0]
    move = np.abs(want - before)
    assert np.isfinite(want).all() and move.max() > 0.1 * LR
    # a move from roots and reciprocals of a unit each, float32 moments and four roundings; the parameter rounded twice
    assert_within("param", f64(p), want, 2.0 ** -20 * move + 2 * U32 * (np.abs(want) + np.abs(before)))
