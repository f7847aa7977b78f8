"""CPU replays of the drafted-tree attention launch (tree.cu): index arithmetic and order of
events only, no attention arithmetic.

Work: the tiles of all segments (layer, unit, row tile) are laid end to end and cut into one
contiguous range per CTA. Checked over many layouts, segments of a single tile among them (a
layer that holds no token has the drafted tile alone):

  * every tile is held by one CTA, and the stepped cursor equals a direct lookup;
  * every segment is put out once, by the CTA that holds it whole or by the last of its holders;
  * a CTA's partial states (two slots) are written once each, each merge reads those of its
    segment's holders, and every ticket is back at zero.

Order: the roles of a CTA (copies, products, keys, values, softmax) are restated as events with
the waits between them, and what must not be overwritten early is looked up in the graph that
they form: X is safe before Y if every order of events that the waits allow has X before Y.
Checked for the ancestor sets of drafted tiles (as many as tree.cu keeps), the query sets and
their scales and marks, the buffers of weights and the outputs, and for every wait on a barrier's phase that
the phase after it cannot pass before the wait is over."""
import os
import random
import re

import pytest

from test_decode_split_replay import Split

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..",
                      "kv_cache_compression_snapkv_gb300", "csrc", "tree.cu")


def ancestor_sets():
    with open(SOURCE) as f:
        return int(re.search(r"constexpr int kTrAnc = (\d+);", f.read()).group(1))


# ------------------------------------------------------------------------------- the work
def tree_grid(tps, units, row_tiles, n_sm):
    total = sum(units * row_tiles * t for t in tps)
    segs = len(tps) * units * row_tiles
    if segs <= n_sm and all(t == tps[0] for t in tps):
        t = tps[0]
        s = min(n_sm // segs, (t + 1) // 2 if t > 8 else (t if t > 3 else 1))
        if (t + s - 1) // s <= (total + n_sm - 1) // n_sm + 6:
            return segs * s
    return min(n_sm, total)


def replay(tps, units, row_tiles, n_sm):
    """tps: tiles per segment of each layer. Returns each CTA's segments as (layer, unit, row
    tile, first tile, end, tiles of the segment)."""
    begins, total = [], 0
    for t in tps:
        begins.append(total)
        total += units * row_tiles * t
    grid = tree_grid(tps, units, row_tiles, n_sm)
    assert 1 <= grid <= min(n_sm, total)
    cs = Split(total, grid, 0)

    def locate(c):
        li = 0
        while li + 1 < len(tps) and c >= begins[li + 1]:
            li += 1
        seg, j = divmod(c - begins[li], tps[li])
        unit, rt = divmod(seg, row_tiles)
        return li, unit, rt, j

    held, written, partial, tickets, merges, ctas = [0] * total, {}, {}, {}, [], []
    for b in range(grid):
        C0, C1 = cs.first(b), cs.first(b + 1)
        assert C1 > C0, "every CTA holds a tile"
        li, unit, rt, j = locate(C0)
        c, mine = C0, []
        while c < C1:
            assert (li, unit, rt, j) == locate(c), "the stepped cursor equals a direct lookup"
            end = min(tps[li], j + C1 - c)
            for k in range(c, c + end - j):
                held[k] += 1
            mine.append((li, unit, rt, j, end, tps[li]))
            c += end - j
            key, sbeg = (li, unit, rt), c - end
            send = sbeg + tps[li]
            if sbeg >= C0 and send <= C1:
                assert key not in written
                written[key] = "whole"
            else:
                slot = (b, 0 if max(sbeg, C0) == C0 else 1)
                assert slot not in partial, "a partial slot written twice"
                partial[slot] = key
                ca, cb = cs.owner(sbeg), cs.owner(send - 1)
                assert ca <= b <= cb
                tickets[key] = tickets.get(key, 0) + 1
                if tickets[key] == cb - ca + 1:
                    late = cs.first(ca) < sbeg
                    merges.append((key, [(ca + k, 1 if k == 0 and late else 0)
                                         for k in range(cb - ca + 1)]))
                    assert key not in written
                    written[key] = "merged"
                    tickets[key] = 0
            li, unit, rt, j = locate(c) if c < total else (0, 0, 0, 0)
        ctas.append(mine)
    assert held == [1] * total
    assert len(written) == len(tps) * units * row_tiles
    assert not any(tickets.values())
    for key, read in merges:
        assert [partial.get(s) for s in read] == [key] * len(read), "a merge reads its holders"
    return ctas


def random_layout(rng):
    tps = [rng.choice([1, 1, 2, 3, 4, 5, 9, 10, 33, rng.randint(1, 300)])
           for _ in range(rng.choice([1, 1, 2, 3, 8]))]
    if rng.random() < 0.5:
        tps = [tps[0]] * len(tps)
    return tps, rng.choice([1, 2, 3, 8, 40, 160, 301]), rng.choice([1, 1, 2, 8]), \
        rng.choice([1, 2, 3, 19, 148, 152])


@pytest.mark.parametrize("seed", range(6))
def test_work_is_cut_into_whole_ranges(seed):
    rng = random.Random(seed)
    for _ in range(60):
        replay(*random_layout(rng))


def test_layouts_of_the_cases():
    assert len(replay([5 + 1], 8, 2, 152)) == 96              # 544 tokens: one tile a CTA
    assert len(replay([1024 + 1], 8, 4, 152)) in (128, 152)   # 131,072 tokens, 256 rows
    assert len(replay([257], 160, 1, 152)) == 152
    assert len(replay([1], 1, 1, 152)) == 1                   # nothing cached, one unit
    assert len(replay([1], 301, 1, 152)) == 152


# ------------------------------------------------------------------------------- the order
class Graph:
    def __init__(self):
        self.before = {}

    def add(self, event, *after):
        """event comes after all of `after` (those that are not None)."""
        self.before.setdefault(event, set()).update(x for x in after if x is not None)
        return event

    def ordered(self, first, then):
        seen, todo = set(), [then]
        while todo:
            for x in self.before.get(todo.pop(), ()):
                if x == first:
                    return True
                if x not in seen:
                    seen.add(x)
                    todo.append(x)
        return False


def roles(d, n, segments, n_anc):
    """The events of one CTA for head dimension d and n columns. segments: (packed tiles, window
    tiles, drafted tile or not) of each of its segments, in order. Returns what is not safe."""
    NP = 1 if n == 64 else 2
    G, NB = NP, 2 if n == 64 else 3
    apart = NB != 2
    RS = (4 if d == 128 else 8) // G
    tiles, sets, drafts = [], [], []          # (kind, segment); set -> its tiles; drafted tiles
    first_of_set, seg_tiles = {}, []
    for s, (p, w, draft) in enumerate(segments):
        kinds = ["p"] * p + ["w"] * w + ["d"] * draft
        assert kinds
        seg_tiles.append(list(range(len(tiles), len(tiles) + len(kinds))))
        for part in (seg_tiles[-1][:p], seg_tiles[-1][p:]):
            if part:
                first_of_set[part[0]] = len(sets)
                sets.append(part)
        tiles += [(k, s) for k in kinds]
        if draft:
            drafts.append(len(tiles) - 1)
    N, g = len(tiles), Graph()
    nd = {i: k for k, i in enumerate(drafts)}
    group = [i % 2 if G == 2 else 0 for i in range(N)]
    need = []                                  # (event, later event, what)

    # copies: ring items of each group, the ancestor set before its drafted tile's
    items, it, last = {}, [0] * G, None
    for i, (kind, _) in enumerate(tiles):
        if kind == "d":
            last = g.add(("set", nd[i]), last)
        items[i] = []
        for _ in range(1 if kind == "p" else 2):
            r = (group[i], it[group[i]])
            it[group[i]] += 1
            old = (r[0], r[1] - RS)
            last = g.add(("copy", r), last, *([("give", old, "K"), ("give", old, "V")] if old[1] >= 0 else []))
            g.add(("landed", r), last)
            items[i].append(r)

    # keys and values (one chain each per group)
    for gr in range(G):
        for side in "KV":
            done = "QK" if side == "K" else "PV"
            prev = None
            for i, (kind, _) in enumerate(tiles):
                if group[i] != gr:
                    continue
                prev = g.add(("free" + side, i), prev, (done, i - NB) if i >= NB else None)
                if i >= NB:
                    need.append((prev, (done, i), "a buffer's phase"))
                if i in first_of_set:
                    s = first_of_set[i]
                    if apart or side == "V":
                        prev = g.add(("qwait" + side, i), prev, ("QK", i - 2) if i >= 2 else None)
                        if i >= 2:
                            need.append((prev, ("QK", i), "a phase of the first products"))
                    prev = g.add(("queries" + side, s), prev)
                    if s >= 2:
                        need.append((("QK", sets[s - 2][-1]), prev, "a query set"))
                    if s >= 8:
                        need.append((("P", sets[s - 8][-1]), prev, "a query set's scales"))
                        need.append((("out", tiles[sets[s - 8][-1]][1]), prev, "a query set's mark"))
                    if s >= 2:      # the wait for set s - 2 is over before its phase passes again
                        need.append((("qk", sets[s - 2][0]), prev, "a query set's phase"))
                r = items[i]
                if kind == "p":
                    prev = g.add(("give", r[0], side), g.add(("read" + side, i), prev, ("landed", r[0])))
                    prev = g.add((side + "ready", i), prev)
                elif side == "K":
                    prev = g.add(("give", r[0], side), g.add(("readK", i), prev, ("landed", r[0])))
                    prev = g.add(("Kready", i), prev)
                    prev = g.add(("give", r[1], side), prev, ("landed", r[1]))
                else:
                    prev = g.add(("give", r[0], side), prev, ("landed", r[0]))
                    prev = g.add(("readV", i), prev, ("landed", r[1]), ("set", nd[i]) if kind == "d" else None)
                    prev = g.add(("Vready", i), prev)
                    prev = g.add(("give", r[1], side), prev)

    # products; a completion covers what its warp has issued before
    def qk(i, prev):
        s = first_of_set.get(i)
        e = g.add(("qk", i), prev, ("Kready", i), ("sfree", i - 2) if i >= 2 else None,
                  *([] if s is None else [("queriesK", s), ("queriesV", s)]))
        g.add(("QK", i), e)
        return e

    def pv(i, prev):
        e = g.add(("pv", i), prev, ("Vready", i), ("P", i))
        g.add(("PV", i), e)
        return e
    if NP == 2:
        a = b = None
        for i in range(N):
            a, b = qk(i, a), pv(i, b)
            if i:
                g.add(("QK", i), ("QK", i - 1))
                g.add(("PV", i), ("PV", i - 1))
    else:
        a, done = qk(0, None), ("QK", 0)
        for i in range(N):
            if i + 1 < N:
                a = qk(i + 1, a)
                g.add(("QK", i + 1), done)
                done = ("QK", i + 1)
            a = pv(i, a)
            g.add(("PV", i), done)
            done = ("PV", i)

    # softmax and output
    prev = [None] * NP
    for s, mine in enumerate(seg_tiles):
        for i in mine:
            p = i % NP
            e = g.add(("softmax", i), prev[p], ("QK", i), ("set", nd[i]) if i in nd else None)
            need.append((e, ("QK", i + 2), "a phase of the first products"))
            e = g.add(("sfree", i), e)
            if NP == 2 and i >= 2:
                e = g.add(("pfree", i), e, ("PV", i - 2))
                need.append((e, ("PV", i), "a phase of the second products"))
            if i >= 2:
                need.append((("PV", i - 2), ("P", i), "a buffer of weights"))
            prev[p] = g.add(("P", i), e)
        end = g.add(("end", s), *prev, ("set", nd[mine[-1]]) if mine[-1] in nd else None,
                    ("PV", mine[-1]), ("PV", mine[-2]) if len(mine) > 1 else None)
        for x in mine[-2:]:
            need.append((end, ("PV", x + 2), "a phase of the second products"))
        out = g.add(("out", s), end)
        prev = [out] * NP
        for i in seg_tiles[s + 1][:NP] if s + 1 < len(seg_tiles) else []:
            need.append((out, ("pv", i), "an output"))
    # ancestor sets: the output of a segment and the values of its drafted tile read its set
    for k, i in enumerate(drafts):
        if k >= n_anc:
            need.append((("out", tiles[drafts[k - n_anc]][1]), ("set", k), "an ancestor set"))
            need.append((("readV", drafts[k - n_anc]), ("set", k), "an ancestor set"))
    return sorted({what for first, then, what in need
                   if then in g.before and not g.ordered(first, then)})


FORMS = [(d, n) for d in (64, 128) for n in (16, 32, 64)]


@pytest.mark.parametrize("d,n", FORMS)
def test_nothing_is_overwritten_early(d, n):
    A = ancestor_sets()
    short = [(0, 0, 1), (0, 1, 1), (1, 0, 1), (1, 1, 1), (2, 1, 1), (3, 0, 1), (5, 2, 1), (0, 3, 1)]
    for s in short:
        assert roles(d, n, [s] * 24, A) == [], s
        assert roles(d, n, [(3, 0, 0)] + [s] * 22, A) == [], s     # (the CTA's first is a part)
    rng = random.Random(d + n)
    for _ in range(6):
        few = [rng.choice(short) for _ in range(3)]
        layout = [rng.choice(few) for _ in range(22)]
        layout[0] = rng.choice([(0, 0, 1), (2, 1, 1), (7, 0, 1)])
        layout[-1] = rng.choice([(4, 0, 0), (2, 1, 0), (0, 0, 1)])
        assert roles(d, n, layout, A) == [], layout


def test_the_replay_finds_what_is_too_few():
    """With eight ancestor sets, segments of a lone drafted tile could lose theirs at head
    dimension 64 and up to 32 columns; with four, segments of two tiles as well."""
    for n in (16, 32):
        assert roles(64, n, [(0, 0, 1)] * 24, 8) == ["an ancestor set"]
        assert roles(64, n, [(1, 0, 1)] * 24, 8) == []
        assert roles(64, n, [(1, 0, 1)] * 24, 4) == ["an ancestor set"]
    assert roles(64, 16, [(0, 0, 1)] * 24, 9) == []
