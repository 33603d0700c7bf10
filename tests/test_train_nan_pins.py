"""The float64 form of the moments' codes where a block holds NaN or infinity (CPU only)."""

import numpy as np
import pytest

from oracle import train_ops as to


@pytest.mark.parametrize("table,keep", [(to.E4M3_POS, False), (to.E5M2_POS, True)], ids=["m", "v"])
def test_nan_is_left_out_of_a_blocks_scale(table, keep):
    x = np.abs(np.random.default_rng(0).normal(size=256))
    clean, e = to.round_stochastic(x, np.full(256, 1234), table, keep)
    y = x.copy()
    at = int(np.argmin(x[:128]))  # not the block's largest
    y[at] = np.nan
    codes, f = to.round_stochastic(y, np.full(256, 1234), table, keep)
    assert np.array_equal(e, f) and codes[at] & 127 == 127
    assert np.array_equal(np.delete(codes, at), np.delete(clean, at))
    y[at] = np.inf  # an infinity is the largest: the block gets the largest scale
    codes, f = to.round_stochastic(y, np.full(256, 1234), table, keep)
    assert codes[at] & 127 == 127 and f.tolist() == [120, e[1]]
    y[:128] = np.nan  # nothing else: the smallest
    assert to.round_stochastic(y, np.full(256, 1234), table, keep)[1].tolist() == [-120, e[1]]
