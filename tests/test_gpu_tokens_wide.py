"""A few tokens with rows of one to many parts: index and rows in one launch, and in three, on
both sides of the rule that chooses (compares of a selection with all others, for each part)."""

import pytest
import torch

from gpu_helpers import announce, needs_gpu
from test_gpu_tokens import BF, F32, Tokens

pytestmark = [pytest.mark.gpu, needs_gpu]

# 2^21 compares: 724 tokens of 4 with rows of one part, 512 of two, 362 of four
SHAPES = [(T, d, k) for d in (2048, 2112, 4096, 4160, 7168) for T, k in ((360, 4), (365, 4), (513, 4), (725, 4))]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d,k", SHAPES)
def test_wide_rows(moe, T, d, k, dtype):
    announce(f"tokens wide T={T} d={d} k={k} {dtype}")
    t = Tokens(moe, T, d, 12, k, dtype, 110, 0.1, repeats=T % 2 == 1, guarded=True)
    t.run(True, False)
    t.check(True, False)
    assert all(g.intact() for g in t.out.values())


def test_very_wide_rows(moe):
    """Three tokens take one launch: 2^18 values are 128 parts of a float32 row."""
    announce("tokens: 3 tokens, rows of 2^18")
    t = Tokens(moe, 3, 1 << 18, 4, 4, F32, 111, 0.2, guarded=True)
    t.run(False, True)
    t.check(False, True)
