"""The expert FFN with 8-bit rows, hidden activations and weights against float64."""

import numpy as np
import pytest
import torch

from ext_helpers import assert_within, f64, ffn_bound, gen, quantized, randn
from gpu_helpers import announce, needs_gpu
from oracle import block_ops as ob

pytestmark = [pytest.mark.gpu, needs_gpu]

BF = torch.bfloat16


def experts(moe, p, W1, W2):
    s1, c1, s2, c2 = moe.expert_shapes(p)
    q = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in (s1, c1, s2, c2)]
    moe.moex_quantize_experts(p, W1, W2, *q)
    return q


def groups(counts):
    return [0] + np.cumsum(counts).tolist()


def ffn(moe, p, x8, xs, perm, off, q, fill=float("nan"), stream=None):
    y = torch.full((p.T * p.k, p.d_model), fill, dtype=BF, device="cuda")
    ws = torch.empty(moe.moex_workspace_size(p, moe.MOEX_STAGE_FFN_FP8), dtype=torch.uint8, device="cuda")
    ws.fill_(0x7F)  # NaN codes: nothing may be read that was not written
    moe.moex_grouped_ffn_fp8(p, x8, xs, perm, torch.tensor(off, dtype=torch.int32, device="cuda"), *q, y, ws, stream)
    return y


@pytest.mark.parametrize("E,d,de", [(1, 64, 64), (3, 320, 448), (2, 128, 2112), (5, 192, 128)])
def test_quantize_experts(moe, E, d, de):
    announce(f"quantize experts E={E} d={d} de={de}")
    p = moe.make_problem(1, d, E, 1, de, BF)
    W1, W2 = randn((E, d, de), 0.1, BF, 1), randn((E, de, d), 3.0, BF, 2)
    W1[0, :, 0] = 0
    q = experts(moe, p, W1, W2)
    torch.cuda.synchronize()
    for w, codes, scale in ((W1, q[0], q[1]), (W2, q[2], q[3])):
        rq, rs, _ = ob.weight_layout(f64(w))
        assert np.array_equal(rq, codes.cpu().numpy()) and np.array_equal(rs, scale.cpu().numpy())


CASES = [  # name, d, de, rows per expert, tokens or None (rows already permuted)
    ("one_row", 64, 64, [1], None),
    ("one_token", 256, 128, [0, 1, 0, 0, 1, 0, 0, 0], 1),
    ("empty_ends", 128, 192, [0, 3, 0, 5, 0], 4),
    ("ragged", 320, 448, [17, 0, 33, 64, 1, 31, 95, 2, 0, 128, 63, 32], 140),
    ("half_blocks", 576, 320, [40, 65, 3], 70),
    ("wide", 2112, 192, [5, 33], 20),
    ("deep", 192, 2112, [5, 33], 20),
    ("tall", 128, 64, [700, 300], None),
    ("tiles", 512, 256, [256, 257, 255, 1], 300),
    ("uneven", 256, 640, [600, 3, 0, 90], 200),
    ("long", 64, 4224, [300, 5, 0, 129], None),
    ("odd_steps", 192, 1920, [40, 260], 150),
]


@pytest.mark.parametrize("tiles", ["0", "1"], ids=["small", "tiles"])
@pytest.mark.parametrize("name,d,de,counts,T", CASES, ids=[c[0] for c in CASES])
def test_against_float64(moe, monkeypatch, name, d, de, counts, T, tiles):
    announce(f"ffn fp8 {name} d={d} de={de} counts={counts} tiles={tiles}")
    monkeypatch.setenv("MOE_FP8_TILES", tiles)
    E, R = len(counts), sum(counts)
    rows = R if T is None else T
    x = randn((rows, d), 1.0, BF, 3)
    W1, W2 = randn((E, d, de), d ** -0.5, BF, 4), randn((E, de, d), de ** -0.5, BF, 5)
    x8, xs, dec = quantized(moe, x)
    perm = None
    if T is None:
        p = moe.make_problem(R, d, E, 1, de, BF)
    else:
        k = R // T if R % T == 0 else -(-R // T)
        p = moe.make_problem(T, d, max(E, k), k, de, BF)
        if max(E, k) != E:
            pytest.skip("rows per token exceed the experts")
        perm = torch.full((T * k,), 1 << 30, dtype=torch.int32, device="cuda")  # rows past the groups: never read
        perm[:R] = torch.randint(0, T, (R,), generator=gen(6), device="cuda", dtype=torch.int32)
        dec = dec[perm[:R].cpu().numpy()]
    q = experts(moe, p, W1, W2)
    off = groups(counts)
    y = ffn(moe, p, x8, xs, perm, off, q)
    y2 = ffn(moe, p, x8, xs, perm, off, q)
    torch.cuda.synchronize()
    w1, w2 = ob.weight_layout(f64(W1))[2], ob.weight_layout(f64(W2))[2]
    w1 = w1[:, :dec.shape[1]]
    ref, bound = ffn_bound(dec, off, w1, w2, de)
    got = f64(y)
    assert np.isnan(got[R:]).all()  # rows behind the last group keep what they held
    assert_within(name, got[:R], ref, bound)
    assert torch.equal(y[:R], y2[:R])


@pytest.mark.parametrize("counts", [[256] * 33, [2560, 40, 0, 256, 3000], [256 * 31 + 77]],
                         ids=["one_over", "mixed", "one_expert"])
def test_cut_tiles_are_joined(moe, monkeypatch, counts):
    """A contraction long enough that a last round's tiles are cut over the
    workgroups: the same as the uncut product to float32's rounding of the parts,
    the same bits twice, and the same in either place of a workspace."""
    announce(f"ffn fp8 cut tiles {counts}")
    E, R, d, de = len(counts), sum(counts), 256, 2560
    p = moe.make_problem(R, d, E, 1, de, BF)
    x8, xs, _ = quantized(moe, randn((R, d), 1.0, BF, 20))
    q = experts(moe, p, randn((E, d, de), d ** -0.5, BF, 21), randn((E, de, d), de ** -0.5, BF, 22))
    off = groups(counts)
    monkeypatch.setenv("MOE_FP8_TILES", "1")
    a, b = ffn(moe, p, x8, xs, None, off, q), ffn(moe, p, x8, xs, None, off, q)
    monkeypatch.setenv("MOE_FP8_TILES", "0")
    c = ffn(moe, p, x8, xs, None, off, q)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    ya, yc = f64(a), f64(c)
    assert np.isfinite(ya).all()
    # both round the same hidden rows but for codes at a border (a step of 2^-3 of one of 2560 terms) and
    # round once to bf16: far apart only where a part was lost or added twice
    norm = np.linalg.norm(yc, axis=1)
    assert np.all(np.linalg.norm(ya - yc, axis=1) <= 2.0 ** -6 * norm)


def test_row_order_and_batch_do_not_change_a_row(moe):
    """A row's result depends on the row alone: with and without the permutation."""
    announce("ffn fp8 perm against permuted rows")
    T, d, E, k, de = 90, 256, 6, 2, 192
    p = moe.make_problem(T, d, E, k, de, BF)
    x = randn((T, d), 1.0, BF, 7)
    W1, W2 = randn((E, d, de), d ** -0.5, BF, 8), randn((E, de, d), de ** -0.5, BF, 9)
    q = experts(moe, p, W1, W2)
    x8, xs, _ = quantized(moe, x)
    perm = torch.randint(0, T, (T * k,), generator=gen(10), device="cuda", dtype=torch.int32)
    off = groups([30, 0, 61, 9, 70, 10])
    a = ffn(moe, p, x8, xs, perm, off, q)
    b = ffn(moe, p, x8[perm.long()].contiguous(), xs[perm.long()].contiguous(), None, off, q)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_non_finite_rows_stay_in_their_rows(moe):
    announce("ffn fp8 NaN rows")
    T, d, E, de = 40, 128, 2, 256
    p = moe.make_problem(T, d, E, 1, de, BF)
    x = randn((T, d), 1.0, BF, 11)
    q = experts(moe, p, randn((E, d, de), d ** -0.5, BF, 12), randn((E, de, d), de ** -0.5, BF, 13))
    off = groups([23, 17])
    clean = ffn(moe, p, *quantized(moe, x)[:2], None, off, q)
    x[5, 77], x[30, 0] = float("nan"), float("inf")
    dirty = ffn(moe, p, *quantized(moe, x)[:2], None, off, q)
    torch.cuda.synchronize()
    assert torch.isnan(dirty[5]).all() and torch.isnan(dirty[30]).all()
    keep = [r for r in range(T) if r not in (5, 30)]
    assert torch.equal(clean[keep], dirty[keep])


def test_foreign_rows_of_the_permutation_are_not_followed(moe):
    """A row index outside [0, T) is against the contract; it must not leave x8."""
    announce("ffn fp8 foreign rows")
    T, d, E, de = 64, 128, 2, 128
    p = moe.make_problem(T, d, E, 1, de, BF)
    x8, xs, _ = quantized(moe, randn((T, d), 1.0, BF, 14))
    q = experts(moe, p, randn((E, d, de), d ** -0.5, BF, 15), randn((E, de, d), de ** -0.5, BF, 16))
    perm = torch.arange(T, dtype=torch.int32, device="cuda")
    good = ffn(moe, p, x8, xs, perm, groups([32, 32]), q)
    perm[3], perm[40] = -5, 1 << 28
    bad = ffn(moe, p, x8, xs, perm, groups([32, 32]), q)
    torch.cuda.synchronize()
    keep = [r for r in range(T) if r not in (3, 40)]
    assert torch.equal(good[keep], bad[keep])
