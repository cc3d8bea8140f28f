"""The order in which the attention's many-row tiles start, restated in Python and checked on the CPU.

find_long_tile gives the workgroup of each rank one tile of the batch, longest context first.  A mistake there
reads and writes rows outside a sequence.  The test restates its arithmetic as the kernel source computes it (the
two must be changed together), in int32 where the source does, and checks that the ranks of a batch are its
tiles, each once -- with contexts of none, past the table, and at the ends of int32 side by side.
"""
import random

import numpy as np
import pytest

R = 128
I32 = 2 ** 31 - 1


def _fits(x):
    assert -I32 - 1 <= x <= I32, x
    return x


def long_tiles(lens, ctx, g, positions):
    """(sequence, tile) of every rank; `positions` is what a row of the tables holds."""
    n = len(lens)
    tiles = [(m * g + R - 1) // R for m in lens] + [0] * (64 - n)
    past = [_fits(min(max(c, 0), positions) - m) for c, m in zip(ctx, lens)] + [0] * (64 - n)

    def count(s, x):  # of the sequence's tiles that are ranked by x or more
        k1 = ((x - past[s]) * g + R - 1) >> 7
        return tiles[s] - min(max(k1 - 1, 0), tiles[s])

    lo0 = min(p if t else I32 for p, t in zip(past, tiles))
    span = 0
    for p, t in zip(past, tiles):
        if t:
            span = max(span, min(p - lo0 + R * t // g + 1, I32))
    out = []
    for rank in range(sum(tiles)):
        lo, hi = lo0, lo0 + span
        while hi - lo > 1:
            mid = (lo + hi) >> 1
            if sum(count(s, mid) for s in range(64)) > rank:
                lo = mid
            else:
                hi = mid
        start = [count(s, lo) for s in range(64)]
        longer = [count(s, hi) for s in range(64)]
        same = [a - b for a, b in zip(start, longer)]
        up = list(np.cumsum(same))
        j = rank - sum(longer)
        s = sum(u <= j for u in up)
        out.append((s, tiles[s] - start[s] + j - (up[s] - same[s])))
    return out, past


def check(lens, ctx, g, positions):
    got, past = long_tiles(lens, ctx, g, positions)
    want = [(s, k) for s, m in enumerate(lens) for k in range(-(-m * g // R))]
    assert sorted(got) == want, (lens, ctx, g)
    ends = [past[s] + R * (k + 1) // g for s, k in got]
    assert ends == sorted(ends, reverse=True)


@pytest.mark.parametrize("g", [1, 3, 4, 64])
@pytest.mark.parametrize("far", [0, 17, 1 << 27, I32 - 1, I32])
def test_ranks_with_lengths_past_the_table(g, far):
    for positions in (16, 4096, 1 << 27):
        check([40, 300, 0, 1, 77], [far, 0, 5, far, 90], g, positions)
        check([300, 1], [0, far], g, positions)
        check([1, 300], [far, 0], g, positions)
        check([130] * 5, [-1, -I32 - 1, far, 0, far], g, positions)


def test_ranks_of_random_batches():
    r = random.Random(5)
    for _ in range(60):
        n = r.randrange(1, 65)
        lens = [r.choice([0, 1, r.randrange(200), r.randrange(900)]) for _ in range(n)]
        ctx = [r.choice([m, max(0, m - r.randrange(50)), m + r.randrange(5000), 0, I32]) for m in lens]
        check(lens, ctx, r.choice([1, 2, 3, 5, 8]), r.choice([64, 1000, 1 << 20]))
