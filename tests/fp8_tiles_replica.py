"""Host replica of how the 256 x 256 form of the 8-bit experts deals tiles to
workgroups and cuts those of a last round (not collected as a test)."""

from __future__ import annotations

import collections

TILE = 256      # rows and columns
MIN_PAIRS = 6   # pairs of steps that a cut has to save

Part = collections.namedtuple("Part", "workgroup slot blocks")
Cut = collections.namedtuple("Cut", "xcd place row0 rows cols parts")  # a tile that is cut


def ceil_div(a, b):
    return -(-a // b)


def workgroups(R, N, E, cus):
    m = min(R, (R + E * (TILE - 1)) // TILE)
    return max(8, min(ceil_div(m * ceil_div(N, TILE), 8) * 8, cus // 8 * 8))


def tiles_of(counts, N):
    """(whole tiles, tails) in list order, (first row, rows, columns) of each; up to 8
    whole row tiles a group, whose order inside it is column by column."""
    cols = [min(N - c, TILE) for c in range(0, N, TILE)]
    full, tail, first = [], [], 0
    for r in counts:
        mt = r // TILE + (1 if r % TILE > TILE // 2 else 0)
        assert mt <= 8 or len(cols) == 1
        full += [(first + m * TILE, min(r - m * TILE, TILE), c) for c in cols for m in range(mt)]
        left = r - mt * TILE
        tail += [(first + mt * TILE, left, c) for c in cols] if left > 0 else []
        first += r
    return full, tail


def cuts(counts, K, N, cus, R=None):
    """Every tile that is cut, by the product of contraction K and N columns."""
    KB, nb = ceil_div(K, 128), workgroups(R or sum(counts), N, len(counts), cus) // 8
    pairs, out = KB // 2, []
    full, tail = tiles_of(counts, N)
    if pairs <= MIN_PAIRS:
        return out
    for x in range(8):
        mine = full[len(full) * x // 8:len(full) * (x + 1) // 8] + tail[len(tail) * x // 8:len(tail) * (x + 1) // 8]
        rounds, rem = divmod(len(mine), nb)
        if rem == 0 or pairs * (nb - rem) < MIN_PAIRS * nb:
            continue
        W = rem * pairs
        for r in range(rem):
            parts = []
            for j in range(nb):
                s0, s1 = W * j // nb, W * (j + 1) // nb
                lo, hi = max(s0, r * pairs), min(s1, (r + 1) * pairs)
                if lo < hi:
                    end = KB if hi == (r + 1) * pairs else 2 * (hi - r * pairs)
                    parts.append(Part(8 * j + x, r - s0 // pairs, end - 2 * (lo - r * pairs)))
            assert sum(p.blocks for p in parts) == KB
            if len(parts) > 1:
                out.append(Cut(x, rounds * nb + r, *mine[rounds * nb + r], parts))
    return out


# name, rows per expert, d_model (columns of the second product), d_expert (its contraction)
SOME = [256, 0, 300, 40, 0, 1, 129, 0, 0, 0, 77, 0, 256, 0, 0, 200, 0, 0, 5] + [0] * 13
CASES = [
    ("some_experts", SOME, 320, 2688),
    ("few_parts", SOME, 256, 2560),
    ("many_parts", [300, 128, 1, 256] + [0] * 60, 320, 4224),
    ("after_whole_rounds", [TILE * 150 + 200, TILE * 100 + 77, 0, TILE * 30], 64, 2496),
]
