"""The cases of the cut tiles do cut tiles, in every way that the kernels distinguish."""

import os
import re

import fp8_tiles_replica as fr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_constants_are_the_kernels():
    src = open(os.path.join(ROOT, "sparse_mixture_experts_route_amd", "csrc", "ffn_fp8.hip")).read()
    assert int(re.search(r"constexpr int kFp8SplitPairs = (\d+);", src).group(1)) == fr.MIN_PAIRS
    assert re.search(r"constexpr int L_BM = (\d+), L_BN = (\d+),", src).groups() == (str(fr.TILE),) * 2


def test_cases_cover_the_ways_to_cut():
    """On 256 compute units."""
    by = {name: fr.cuts(counts, de, d, 256) for name, counts, d, de in fr.CASES}
    assert all(by.values())
    every = [c for cs in by.values() for c in cs]
    assert max(sum(1 for z in cs if z.xcd == c.xcd) for cs in by.values() for c in cs) >= 2  # several on one XCD
    assert any(p.slot == 1 for c in every for p in c.parts)            # a workgroup with parts of two tiles
    # one and more rounds of the join
    assert any(len(c.parts) <= 4 for c in every) and any(len(c.parts) > 4 for c in every)
    assert {c.rows for c in every} >= {fr.TILE, 1} and any(1 < c.rows < 128 for c in every)
    assert any(c.cols < fr.TILE for c in every) and any(c.cols == fr.TILE for c in every)
    # after whole rounds
    assert any(c.place >= fr.workgroups(sum(n), d, len(n), 256) // 8 for name, n, d, _ in fr.CASES for c in by[name])
    assert {fr.ceil_div(de, 128) % 2 for _, _, _, de in fr.CASES} == {0, 1}
    assert any(p.blocks % 2 for c in every for p in c.parts)           # a part that ends in an odd block
