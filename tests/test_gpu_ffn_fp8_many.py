"""The 8-bit experts with more experts than a wave has lanes, and at the widest rows
of the workloads: the products and the whole layer against float64."""

import numpy as np
import pytest
import torch

from ext_helpers import assert_within, f64, ffn_bound, gen, quantized, randn
from gpu_helpers import announce, needs_gpu
from oracle import block_ops as ob
from test_gpu_block_run import test_block_against_float64 as block_against_float64
from test_gpu_ffn_fp8 import experts, ffn, groups

pytestmark = [pytest.mark.gpu, needs_gpu]

BF = torch.bfloat16


def spread(E, rows, seed):
    """Rows per expert: groups of `rows` sizes at random experts, the first and last among them."""
    rng = np.random.default_rng(seed)
    counts = np.zeros(E, int)
    counts[[0, E - 1]] = rows[:2]
    counts[1 + rng.permutation(E - 2)[:len(rows) - 2]] = rows[2:]
    return counts.tolist()


CASES = [  # experts past 1, 2, 3 and 4 waves of lanes; every expert with a row; all rows at the last one
    ("65", 192, 128, spread(65, [33, 260, 1, 1, 129, 64, 31, 300, 2], 1)),
    ("130", 128, 320, spread(130, [1, 1] + [3] * 60 + [257], 2)),
    ("200", 320, 192, spread(200, [257, 129, 40, 1, 77, 32, 256], 3)),
    ("256", 256, 256, spread(256, [5, 140] + [1, 2, 33, 4] * 40, 4)),
    ("256_each", 192, 192, [1 + e % 3 for e in range(256)]),
    ("256_last", 256, 192, [0] * 255 + [600]),
    ("7168", 7168, 128, [3, 0, 40]),
    ("7168_deep", 128, 7168, [3, 0, 40]),
]


@pytest.mark.parametrize("tiles", ["0", "1"], ids=["small", "tiles"])
@pytest.mark.parametrize("name,d,de,counts", CASES, ids=[c[0] for c in CASES])
def test_against_float64(moe, monkeypatch, name, d, de, counts, tiles):
    announce(f"ffn fp8 many {name} tiles={tiles}")
    monkeypatch.setenv("MOE_FP8_TILES", tiles)
    E, R, T = len(counts), sum(counts), 50
    k = -(-R // T) if -(-R // T) <= E else 1
    T = T if k > 1 else R
    p = moe.make_problem(T, d, E, k, de, BF)
    x8, xs, dec = quantized(moe, randn((T, d), 1.0, BF, 3))
    W1, W2 = randn((E, d, de), d ** -0.5, BF, 4), randn((E, de, d), de ** -0.5, BF, 5)
    q = experts(moe, p, W1, W2)
    perm = torch.randint(0, T, (T * k,), generator=gen(6), device="cuda", dtype=torch.int32)
    y = ffn(moe, p, x8, xs, perm, groups(counts), q)
    torch.cuda.synchronize()
    w1, w2 = ob.weight_layout(f64(W1))[2], ob.weight_layout(f64(W2))[2]
    ref, bound = ffn_bound(dec[perm[:R].cpu().numpy()], groups(counts), w1[:, :dec.shape[1]], w2, de)
    got = f64(y)
    assert np.isnan(got[R:]).all()
    assert_within(name, got[:R], ref, bound)


@pytest.mark.parametrize("T,d,E,k,de", [(40, 256, 96, 6, 128), (300, 192, 256, 8, 192), (3, 320, 256, 8, 64)])
def test_layer(moe, T, d, E, k, de):
    block_against_float64(moe, T, d, E, k, de)
