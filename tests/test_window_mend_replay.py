"""Replay on the CPU of how mend_rows (csrc/window_tc.cu) cuts the keys that a warp's rows see: what all of
them see is read once, the rest for each row, and together that is each row's keys, every index inside
[0, row] and what is read for a row alone a few dozen keys."""
import random

import pytest


def ranges(n, s, W, g, q0, quarter, rows):
    """(common ranges, {row: (position, its own ranges)}, the ranges that finite_keys reads)."""
    P = 128 // g
    place = {i: q0 + (quarter * 32 + i) % P for i in rows}
    first, last, back = min(place.values()), max(place.values()), W - 1
    s1 = min(s, first + 1)
    w0 = max(s1, last - back)
    common = [(0, s1), (w0, first + 1)]
    own = {i: (p, [(max(s1, p - back), min(w0, p + 1)), (max(first + 1, p - back), p + 1), (s1, min(s, p + 1))])
           for i, p in place.items()}
    return common, own, [(0, min(s, last + 1)), (max(0, first - back), last + 1)]


def visited(parts):
    """Indices that a loop of eight reads, the last one again past the end."""
    seen = set()
    for a, b in parts:
        for j in range(a, b, 8):
            seen |= {min(j + i, b - 1) for i in range(8)}
    return seen


@pytest.mark.parametrize("seed", range(400, 410))
def test_every_key_seen(seed):
    rng = random.Random(seed)
    for _ in range(40):
        every_key_seen(rng)


def every_key_seen(rng):
    n = rng.choice([1, 2, 17, 64, 129, 300, 700])
    g = rng.choice([1, 2, 4, 8])
    s = min(n, rng.choice([0, 1, 4, 37, 128, rng.randint(0, n), n]))
    W = min(n, rng.choice([1, 2, 17, 31, 64, 100, rng.randint(1, n), n]))
    P = 128 // g
    q0 = rng.randrange(0, n, P)
    quarter = rng.randrange(4)
    live = [i for i in range(32) if q0 + (quarter * 32 + i) % P < n]
    if not live:
        return
    rows = rng.sample(live, rng.randint(1, len(live)))
    common, own, keys = ranges(n, s, W, g, q0, quarter, rows)
    shared, asked = visited(common), visited(keys)
    for pos, mine in own.values():
        want = {j for j in range(pos + 1) if j < s or pos - j < W}
        assert shared | visited(mine) == want
        assert want <= asked <= set(range(n))
        assert sum(max(0, b - a) for a, b in mine) <= 3 * 31


def again(n, s, W, g, q0, quarter, rows):
    """rows_again over the lowest three rows: per row, the keys it takes in order, and every key read."""
    P = 128 // g
    place = [q0 + (quarter * 32 + i) % P for i in sorted(rows)[:3]]
    lo, hi = min(place), max(place)
    s1 = min(s, hi + 1)
    w0 = max(s1, lo - (W - 1))
    taken, read = [[] for _ in place], set()
    for start, end in ((0, s1), (w0, hi + 1)):
        for j0 in range(start, end, 32):
            read |= {min(j0 + lane, end - 1) for lane in range(32)}
            for i0 in range(0, min(32, end - j0), 8):
                read |= {min(j0 + i0 + i, end - 1) for i in range(8)}
                for i in range(8):
                    j = j0 + i0 + i
                    for r, p in enumerate(place):
                        if j < end and j <= p and (j < s or p - j < W):
                            taken[r].append(j)
    return place, taken, read


@pytest.mark.parametrize("seed", range(5))
def test_rows_formed_again(seed):
    rng = random.Random(1000 + seed)
    for _ in range(40):
        rows_formed_again(rng)


def rows_formed_again(rng):
    n = rng.choice([1, 2, 17, 64, 129, 300, 700])
    g = rng.choice([1, 2, 4, 8])
    s = min(n, rng.choice([0, 1, 4, 37, rng.randint(0, n), n]))
    W = min(n, rng.choice([1, 2, 17, 64, rng.randint(1, n), n]))
    q0, quarter = rng.randrange(0, n, 128 // g), rng.randrange(4)
    live = [i for i in range(32) if q0 + (quarter * 32 + i) % (128 // g) < n]
    if not live:
        return
    place, taken, read = again(n, s, W, g, q0, quarter, rng.sample(live, rng.randint(1, len(live))))
    assert read <= set(range(n))
    for p, keys in zip(place, taken):
        assert keys == [j for j in range(p + 1) if j < s or p - j < W]
