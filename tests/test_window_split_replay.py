"""CPU replays of the windowed prompt attention launch (window_tc.cu): index arithmetic and order of
events only, no attention arithmetic.

Work: an item is a unit and 2 P consecutive positions in two row tiles; its key tiles are those of the
sinks in front of the first row's window, then those from that window's first key on. Checked over
many shapes: every key that a row sees lies in exactly one tile that its row tile takes part in,
at a place that the mask leaves, no other place is left by the masks, and no tile begins outside the
prompt.

Order: the roles of a CTA (copies, products of scores and of outputs, groups) are restated as
processes that wait on barriers by the parity of a phase, as the kernel does, run in random order
with copies and products that end late. Checked: they all come to an end; a wait is over exactly when
its phase is (never a phase early, nor blocked because the barrier is a phase ahead); and nothing is
overwritten before its last reader is done: stages of keys and values, queries, buffers of scores and
weights, outputs, references."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..",
                      "kv_cache_compression_snapkv_gb300", "csrc", "window_tc.cu")
KEYS = 64


class Item:
    def __init__(self, block, n, s, W, P, two=True):
        self.p0 = block * P * (2 if two else 1)
        end = min(self.p0 + P * (2 if two else 1), n)
        self.j0 = max(0, self.p0 - (W - 1))
        self.s0 = min(s, self.j0)
        self.ts = (self.s0 + KEYS - 1) // KEYS
        self.T = self.ts + (end - 1 - self.j0) // KEYS + 1
        self.lo, self.hi = [], []
        for x in range(2):
            q0 = self.p0 + x * P
            first = self.j0 if s > self.j0 else max(self.j0, q0 - (W - 1))
            self.lo.append(self.ts + (first - self.j0) // KEYS)
            self.hi.append(self.ts + (min(q0 + P, end) - 1 - self.j0) // KEYS + 1 if q0 < end else 0)

    def key0(self, t):
        return t * KEYS if t < self.ts else self.j0 + (t - self.ts) * KEYS

    def active(self, x, t):
        return t < self.hi[x] and (t < self.ts or t >= self.lo[x])

    def tiles(self, x):
        """As the groups step: from the first on, over the tiles left out."""
        t, out = 0 if self.ts else self.lo[x], []
        while t < self.hi[x]:
            out.append(t)
            t = self.lo[x] if t + 1 == self.ts else t + 1
        return out


def below(k):
    return 0 if k <= 0 else (1 << min(k, 32)) - 1


def left(item, x, t, pos, n, s, W, P):
    """Columns that the kernel leaves of tile t for the row at `pos`."""
    key0, q0 = item.key0(t), item.p0 + x * P
    q1 = q0 + P - 1
    bits = (1 << KEYS) - 1
    sinks = t < item.ts
    if (key0 + KEYS > item.s0) if sinks else (key0 + KEYS - 1 > q0 or key0 < q1 - (W - 1)):
        bits = 0
        for h in range(2):
            k = key0 + 32 * h
            word = below(item.s0 - k) if sinks else \
                below(pos + 1 - k) & (~below(pos - (W - 1) - k) | below(s - k))
            bits |= (word & 0xffffffff) << (32 * h)
    return bits


SHAPES = [(n, s, W, g) for n in (1, 2, 63, 64, 65, 200, 333) for s in (0, 1, 5, 64, 70, 400)
          for W in (1, 2, 63, 64, 65, 130, 333) for g in (1, 2, 4, 8)]


def test_every_seen_key_once():
    for n, s, W, g in random.Random(1).sample(SHAPES, 260) + [(700, 4, 128, 1), (700, 150, 90, 2), (1000, 37, 300, 8)]:
        s, W, P = min(s, n), min(W, n), 128 // g
        rows, two = set(), n % 3 > 0
        for block in range(-(-n // (P * (2 if two else 1)))):
            it = Item(block, n, s, W, P, two)
            for t in range(it.T):
                assert 0 <= it.key0(t) < n
            for x in range(2):
                assert it.tiles(x) == [t for t in range(it.T) if it.active(x, t)]
                for dp in range(P):
                    pos = it.p0 + x * P + dp
                    if pos >= n or not it.hi[x]:
                        continue
                    assert pos not in rows
                    rows.add(pos)
                    found = []
                    for t in it.tiles(x):
                        bits = left(it, x, t, pos, n, s, W, P)
                        found += [it.key0(t) + c for c in range(KEYS) if bits >> c & 1]
                    assert sorted(found) == [j for j in range(pos + 1) if j < s or pos - j < W], (n, s, W, g, pos)
        assert rows == set(range(n))


# ------------------------------------------------------------------------------------ order of events
class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.phases = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phases = 0, self.phases + 1

    def over(self, phase):
        assert self.phases <= phase + 1, "a phase ahead of its waiter: the wait would block"
        passed = self.phases % 2 != phase % 2          # as try_wait.parity answers
        assert passed == (self.phases == phase + 1), "a wait that is over before its phase is"
        return passed


class Cta:
    def __init__(self, items, SB, NB, KS, VS, rng):
        self.items, self.SB, self.NB, self.rng = items, SB, NB, rng
        self.rings = {"k": (KS, [Barrier(1) for _ in range(KS)], [Barrier(2) for _ in range(KS)]),
                      "v": (VS, [Barrier(1) for _ in range(VS)], [Barrier(2) for _ in range(VS)])}
        rows = lambda k, c=1: [[Barrier(c) for _ in range(k)] for _ in range(2)]  # noqa: E731
        self.qfull, self.qempty = rows(NB), rows(NB)
        self.sfull, self.pfull, self.pvdone = rows(SB), rows(SB), rows(SB)
        self.oread, self.ofull = [Barrier(2), Barrier(2)], [Barrier(1), Barrier(1)]
        self.pair = [Barrier(2), Barrier(2)]
        self.late = {}                                  # queues of what ends late, in order of issue
        self.stage = {}                                 # (ring, stage) -> (tile, users left)
        self.queries = {}                               # (x, buffer) -> (item, users left)
        self.scores = {}                                # (x, buffer) -> (tile, state)
        self.outputs = {0: None, 1: None}               # x -> (item, readers left)
        self.ref = {}                                   # (x, item & 1) -> (item, tile)

    def later(self, queue, f):
        self.late.setdefault(queue, []).append(f)

    # ---- processes: generators that yield (barrier, phase) or a condition
    def copies(self):
        nq = [0, 0]
        tiles = [(i, t) for i, it in enumerate(self.items) for t in range(it.T)]

        def load(ring, j):
            S, full, empty = self.rings[ring]
            s, rnd = j % S, j // S
            if rnd:
                yield empty[s], rnd - 1
            assert self.stage.get((ring, s), (0, 0))[1] == 0, "a stage that is still read"

            def landed():
                self.stage[ring, s] = (j, 2)
                full[s].arrive()
            self.later(("load", ring, s), landed)

        def keys(j):
            if j >= len(tiles):
                return
            i, t = tiles[j]
            if t == 0:
                for x in range(2):
                    if not self.items[i].hi[x]:
                        continue
                    b, rnd = nq[x] % self.NB, nq[x] // self.NB
                    if rnd:
                        yield self.qempty[x][b], rnd - 1
                    users = len(self.items[i].tiles(x))
                    assert self.queries.get((x, b), (0, 0))[1] == 0, "queries that are still read"

                    def landed(x=x, b=b, item=nq[x], users=users):
                        self.queries[x, b] = (item, users)
                        self.qfull[x][b].arrive()
                    self.later(("q", x, b), landed)
                    nq[x] += 1
            yield from load("k", j)
        yield from keys(0)
        yield from keys(1)
        for j in range(len(tiles)):
            yield from load("v", j)
            yield from keys(j + 2)

    def use(self, ring, s, tile):
        have, users = self.stage[ring, s]
        assert have == tile and users > 0, "another tile's stage"
        self.stage[ring, s] = (have, users - 1)
        self.rings[ring][2][s].arrive()

    def products(self, x, ring):
        S, full, _ = self.rings[ring]
        j = n = no = 0
        for it in self.items:
            mine = it.tiles(x)
            for t in range(it.T):
                s = j % S
                yield full[s], j // S
                if not it.active(x, t):
                    self.use(ring, s, j)
                else:
                    b, r = n % self.SB, n // self.SB
                    begin, end = t == mine[0], t == mine[-1]
                    if ring == "k":
                        if begin:
                            qb = no % self.NB
                            yield self.qfull[x][qb], no // self.NB
                            no += 1
                        if r:
                            yield self.pvdone[x][b], r - 1
                        assert self.scores.get((x, b), (0, "used"))[1] == "used", "scores or weights still read"
                        self.scores[x, b] = (n, "forming")

                        def done(b=b, n=n, s=s, j=j, end=end, qb=qb, item=no - 1):
                            have, users = self.queries[x, qb]
                            assert have == item and users > 0
                            self.queries[x, qb] = (have, users - 1)
                            self.scores[x, b] = (n, "scores")
                            self.sfull[x][b].arrive()
                            self.use("k", s, j)
                            if end:
                                assert self.queries[x, qb][1] == 0
                                self.qempty[x][qb].arrive()
                    else:
                        if begin:
                            if no:
                                yield self.oread[x], no - 1
                            assert self.outputs[x] is None or self.outputs[x][1] == 0, "outputs not read yet"
                            self.outputs[x] = (no, 2)
                            no += 1
                        yield self.pfull[x][b], r
                        assert self.scores[x, b] == (n, "weights")

                        def done(b=b, n=n, s=s, j=j, end=end):
                            assert self.scores[x, b] == (n, "weights")
                            self.scores[x, b] = (n, "used")
                            self.pvdone[x][b].arrive()
                            self.use("v", s, j)
                            if end:
                                self.ofull[x].arrive()
                    self.later((ring, x), done)
                    n += 1
                j += 1

    def group(self, x, buf):
        n = no = 0
        for it in self.items:
            if not it.hi[x]:
                continue
            mine = it.tiles(x)
            for t in mine:
                if n % 2 == buf:
                    b, r = n % self.SB, n // self.SB
                    yield self.sfull[x][b], r
                    assert self.scores[x, b] == (n, "scores")
                    if t != mine[0]:
                        yield lambda n=n, no=no: self.ref.get((x, no & 1)) == (no, n - 1)
                        if self.rng.random() < 0.3:     # the reference is raised: outputs are rescaled
                            m = n - 1
                            yield self.pvdone[x][m % self.SB], m // self.SB
                            assert self.outputs[x][0] == no
                            assert not [q for q in self.late.get(("v", x), [])], "a product of outputs under way"
                    self.ref[x, no & 1] = (no, n)
                    self.scores[x, b] = (n, "weights")
                    self.pfull[x][b].arrive()
                n += 1
            yield lambda n=n, no=no: self.ref.get((x, no & 1)) == (no, n - 1)
            p = self.pair[x].phases
            self.pair[x].arrive()
            yield self.pair[x], p
            yield self.ofull[x], no
            have, readers = self.outputs[x]
            assert have == no and readers > 0
            self.outputs[x] = (have, readers - 1)
            self.oread[x].arrive()
            no += 1

    def run(self):
        todo = {}
        for name, g in [("copies", self.copies())] + [((r, x), self.products(x, r)) for r in "kv" for x in range(2)] + \
                       [(("group", x, b), self.group(x, b)) for x in range(2) for b in range(2)]:
            todo[name] = [g, None]
        slow = self.rng.choice([None] + list(todo))     # one role may be far behind
        while todo:
            ready = []
            for name, (g, wait) in todo.items():
                if wait is None or (wait() if callable(wait) else wait[0].over(wait[1])):
                    ready.append(name)
            late = [q for q, fs in self.late.items() if fs]
            assert ready or late, "no role can go on: %s" % list(todo)
            pick = self.rng.choice([(0, r) for r in ready if r != slow or self.rng.random() < 0.1 or len(ready) == 1 and not late] +
                                   [(1, q) for q in late] or [(0, r) for r in ready])
            if pick[0]:
                self.late[pick[1]].pop(0)()
                continue
            name = pick[1]
            try:
                todo[name][1] = next(todo[name][0])
            except StopIteration:
                del todo[name]
        for fs in self.late.values():
            while fs:
                fs.pop(0)()
        assert all(state == "used" for _, state in self.scores.values())


def test_buffers_are_the_kernels():
    text = open(SOURCE).read()
    assert re.search(r"SB = D == 64 \? 3 : 2;", text) and re.search(r"NB = D == 64 \? 2 : 1;", text)
    smem = int(re.search(r"kWnSmemLimit = (\d+);", text).group(1))
    rest = int(re.search(r"FIT = \(kWnSmemLimit - 2 \* NB \* TQ - (\d+)\) / TB;", text).group(1))
    for d, NB, stages in ((64, 2, (8, 8)), (128, 1, (4, 5))):
        fit = (smem - 2 * NB * 128 * d * 2 - rest) // (KEYS * d * 2)
        assert ((8, 8) if fit > 16 else (fit // 2, fit - fit // 2)) == stages


@pytest.mark.parametrize("SB,NB,KS,VS", [(3, 2, 8, 8), (2, 1, 4, 5)])
def test_order(SB, NB, KS, VS):
    rng = random.Random(7)
    for _ in range(160):
        g = rng.choice([1, 2, 4, 8])
        n, s, W = rng.randint(1, 900), rng.choice([0, 0, 3, 70, 200]), rng.choice([1, 2, 40, 64, 130, 400])
        P, s, W = 128 // g, min(s, n), min(W, n)
        two = rng.random() < 0.7
        blocks = -(-n // (P * (2 if two else 1)))
        items = [Item(rng.randrange(blocks), n, s, W, P, two) for _ in range(rng.randint(1, 7))]
        Cta(items, SB, NB, KS, VS, rng).run()
