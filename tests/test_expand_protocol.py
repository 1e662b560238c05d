"""Protocol model of the expansion kernel (csrc/expand.cu), without a GPU.

A cluster's agents: the TMA thread of each of its two CTAs, the leader's warp
that issues the pair's MMAs, and four storing warps a CTA.  The barriers that the
MMAs wait on are the leader's, and both CTAs' loads count on them; the others are
each CTA's own, reached by commits that go to both, each at its own time.  TMA
landings, the two halves of a commit and the reads of stores from shared memory
come in any order; MMAs and commits run in the order in which they were issued.
mbarriers follow the hardware's rules (arrivals, transaction bytes, phases told
apart by their parity alone), every wait says which phase it means, and every
read is checked for the tile it expects, every write for readers that are not
done.  Random interleavings must end without deadlock; planted mistakes must not.

The order in which clusters take units (Walk) is restated and checked: every
unit once, latents loaded where they change.
"""

import random

import pytest

from .test_prefill_protocol import Bar, Fault, check

WARPS = 4          # storing warps of a CTA
PIECES = 4         # 64-column pieces of an accumulator


class Walk:
    """The units of cluster c of n, as (tile pair, group, head pair), and whether the unit after has other latents."""

    def __init__(self, c, n, tiles, groups, pairs):
        all_pairs, each = (tiles + 1) // 2, groups * pairs
        rounds = all_pairs // n
        left = (all_pairs - rounds * n) * each
        lo, hi = left * c // n, left * (c + 1) // n
        self.whole, self.end, self.first = rounds * each, rounds * each + hi - lo, rounds * n * each + lo
        self.n, self.groups, self.pairs = n, groups, pairs
        self.unit, self.at = 0, [c, 0, 0]
        if rounds == 0:
            self.rest()

    def rest(self):
        self.at = [self.first // self.pairs // self.groups, self.first // self.pairs % self.groups, self.first % self.pairs]

    def units(self):
        out = []
        while self.unit < self.end:
            last = self.at[2] + 1 == self.pairs or self.unit + 1 == self.end
            out.append((tuple(self.at), last))
            self.unit += 1
            if self.unit == self.whole:
                self.rest()
                continue
            self.at[2] += 1
            if self.at[2] == self.pairs:
                self.at[2] = 0
                self.at[1] += 1
                if self.at[1] == self.groups:
                    self.at[1] = 0
                    self.at[0] += self.n if self.unit < self.whole else 1
        return out


class Model:
    def __init__(self, units, tiles, chunks, stages, rng, broken=None):
        self.units, self.tiles, self.chunks, self.stages, self.rng, self.broken = units, tiles, chunks, stages, rng, broken
        self.lead = dict(a_full=[Bar(1) for _ in range(chunks)], b_full=[Bar(1) for _ in range(stages)],
                         d_empty=[Bar(2 * WARPS) for _ in range(2)])
        self.own = [dict(a_empty=[Bar(1)], b_empty=[Bar(1) for _ in range(stages)], d_full=[Bar(1), Bar(1)], done=[Bar(1)])
                    for _ in range(2)]
        self.A = [[None] * chunks for _ in range(2)]
        self.W = [[None] * stages for _ in range(2)]
        self.D = [None, None]
        self.d_left = [0, 0]                            # storing warps that have the accumulator still to read
        self.readers = {}
        self.pipe, self.landings, self.halves = [], [], []
        self.box = {}                                   # (rank, warp) -> [tags of the two boxes]
        self.stores = {}                                # (rank, warp) -> stores that have not read their box: (box, tag)
        self.stored = []

    def ready(self, w):
        if callable(w):
            return w()
        bar, phase = w
        if not bar.passes(phase & 1):
            return False
        check(bar.done > phase, "a wait passed before its phase")
        return True

    def load(self, mem, cell, at, tag, bar):
        check(self.readers.get((cell, at), 0) == 0, f"{cell} loaded while it is read")
        mem[at] = None
        self.landings.append((mem, at, tag, bar))

    def commit(self, name, at):
        self.pipe.append(("commit", name, at))

    def has_tile(self, pair, rank):
        return 2 * pair + rank < self.tiles

    # ----------------------------------------------------------------- agents
    def tma(self, rank):
        nb = na = 0
        fresh = True
        for (pair, group, heads), last in self.units:
            if fresh:
                if na > 0 and self.broken != "a_empty":
                    yield (self.own[rank]["a_empty"][0], na - 1)
                na += 1
                for c in range(self.chunks):
                    if rank == 0:
                        self.lead["a_full"][c].arrive(tx=1 + self.has_tile(pair, 1))
                    if self.has_tile(pair, rank):
                        self.load(self.A[rank], ("A", rank), c, (pair, group, c), self.lead["a_full"][c])
                    yield None
            fresh = last
            for kind in range(2):
                for c in range(self.chunks):
                    st = nb % self.stages
                    if nb >= self.stages and self.broken != "b_empty":
                        yield (self.own[rank]["b_empty"][st], nb // self.stages - 1)
                    if rank == 0:
                        self.lead["b_full"][st].arrive(tx=2)
                    self.load(self.W[rank], ("W", rank), st, (group, heads, kind, c), self.lead["b_full"][st])
                    nb += 1
                    yield None

    def mma(self):
        nb = na = nd = 0
        fresh = True
        for (pair, group, heads), last in self.units:
            na += fresh
            for kind in range(2):
                buf = nd & 1
                if nd >= 2 and self.broken != "d_empty":
                    yield (self.lead["d_empty"][buf], (nd >> 1) - 1)
                if self.broken == "early":
                    self.commit("d_full", buf)
                for c in range(self.chunks):
                    st = nb % self.stages
                    if fresh and kind == 0 and self.broken != "a_full":
                        yield (self.lead["a_full"][c], na - 1)
                    yield (self.lead["b_full"][st], nb // self.stages)
                    for r in range(2):
                        for cell in ((("A", r), c), (("W", r), st)):
                            self.readers[cell] = self.readers.get(cell, 0) + 1
                    self.pipe.append(("mma", buf, c, st, (pair, group, heads, kind)))
                    self.commit("b_empty", st)
                    nb += 1
                if self.broken != "early":
                    self.commit("d_full", buf)
                nd += 1
            if last:
                self.commit("a_empty", 0)
            fresh = last
        self.commit("done", 0)

    def wait_done(self, rank):
        yield (self.own[rank]["done"][0], 0)

    def store(self, rank, w):
        nd = no = 0
        key = (rank, w)
        self.box[key], self.stores[key] = [None, None], []
        for (pair, group, heads), _ in self.units:
            for kind in range(2):
                buf, tag = nd & 1, (pair, group, heads, kind)
                yield (self.own[rank]["d_full"][buf], nd >> 1)
                for piece in range(PIECES):
                    check(self.D[buf] == (tag, self.chunks), "another accumulator stored")
                    yield None
                    check(self.D[buf] == (tag, self.chunks) and self.d_left[buf] > 0, "the accumulator changed while it was read")
                    if piece == (0 if self.broken == "release" else PIECES - 1):
                        self.d_left[buf] -= 1
                        self.lead["d_empty"][buf].arrive()
                    if not self.has_tile(pair, rank):
                        continue
                    b = no & 1
                    no += 1
                    if self.broken != "box":
                        yield lambda: len(self.stores[key]) <= 1
                    check(all(x != b for x, _ in self.stores[key]), "a box overwritten before its store read it")
                    self.box[key][b] = (tag, piece)
                    self.stores[key].append((b, (tag, piece)))
                nd += 1
        yield lambda: not self.stores[key]

    def run_pipe(self):
        op = self.pipe.pop(0)
        if op[0] == "commit":
            self.halves += [self.own[r][op[1]][op[2]] for r in range(2)]
            return
        _, buf, c, st, (pair, group, heads, kind) = op
        for r in range(2):
            if self.has_tile(pair, r):
                check(self.A[r][c] == (pair, group, c), "MMA of other latents")
            check(self.W[r][st] == (group, heads, kind, c), "MMA of other weights")
            self.readers[(("A", r), c)] -= 1
            self.readers[(("W", r), st)] -= 1
        tag = (pair, group, heads, kind)
        if c == 0:
            check(self.d_left[buf] == 0, "accumulator overwritten before it was stored")
        else:
            check(self.D[buf] == (tag, c), "MMAs out of order")
        self.D[buf] = (tag, c + 1)
        if c + 1 == self.chunks:
            self.d_left[buf] = 2 * WARPS

    def run(self):
        agents = [self.tma(0), self.tma(1), self.mma(), self.wait_done(0), self.wait_done(1)]
        agents += [self.store(r, w) for r in range(2) for w in range(WARPS)]
        waits, live = [None] * len(agents), set(range(len(agents)))
        lag = self.rng.choice([0.0, 0.8, 0.97])
        for _ in range(400000):
            moves = [("agent", a) for a in live if waits[a] is None or self.ready(waits[a])]
            if self.pipe:
                moves.append(("pipe", 0))
            moves += [("land", k) for k in range(len(self.landings))]
            moves += [("half", k) for k in range(len(self.halves))]
            moves += [("read", k) for k, v in self.stores.items() if v]
            if not moves or not live:
                check(not live, "deadlock")
                # the cluster's last barrier: nothing may still be on its way to either CTA
                check(not self.pipe and not self.landings and not any(self.stores.values()), "work in flight at the end")
                want = [(r, w, (p, g, h, k), x) for (p, g, h), _ in self.units for k in range(2) for r in range(2)
                        if self.has_tile(p, r) for w in range(WARPS) for x in range(PIECES)]
                check(sorted(self.stored) == sorted(want), "an output was lost")
                return
            kind, x = self.rng.choice(moves)
            if kind == "land" and self.rng.random() < lag:
                continue                                # memory is slow in some runs
            if kind == "pipe":
                self.run_pipe()
            elif kind == "land":
                mem, at, tag, bar = self.landings.pop(x)
                mem[at] = tag
                bar.land(1)
            elif kind == "half":
                self.halves.pop(x).arrive()
            elif kind == "read":
                b, tag = self.stores[x].pop(0)
                check(self.box[x][b] == tag, "a store read another piece")
                self.stored.append((x[0], x[1], tag[0], tag[1]))
            else:
                try:
                    waits[x] = next(agents[x])
                except StopIteration:
                    live.discard(x)
        raise Fault("does not end")


@pytest.mark.parametrize("clusters", [1, 2, 3, 7, 74])
def test_walk_takes_every_unit_once(clusters):
    rng = random.Random(clusters)
    for _ in range(200):
        tiles, groups, pairs = rng.randint(1, 12 * clusters), rng.choice([1, 2, 4]), rng.choice([1, 3, 8])
        n = min(clusters, (tiles + 1) // 2 * groups * pairs)
        seen = []
        for c in range(n):
            units = Walk(c, n, tiles, groups, pairs).units()
            for (a, last), (b, _) in zip(units, units[1:]):
                assert last == (a[:2] != b[:2])             # (the pair that starts over is a tile pair's or a group's end)
            if units:
                assert units[-1][1]
            seen += [u for u, _ in units]
        assert sorted(seen) == [(t, g, p) for t in range((tiles + 1) // 2) for g in range(groups) for p in range(pairs)]


def some_units(rng):
    tiles, groups, pairs, n = rng.randint(1, 9), rng.choice([1, 2]), rng.choice([1, 2, 3]), rng.randint(1, 3)
    n = min(n, (tiles + 1) // 2 * groups * pairs)
    return Walk(rng.randrange(n), n, tiles, groups, pairs).units()[:8], tiles


@pytest.mark.parametrize("seed", range(10))
def test_random_interleavings_end_well(seed):
    rng = random.Random(seed)
    for _ in range(8):
        units, tiles = some_units(rng)
        if units and not units[-1][1]:
            units[-1] = (units[-1][0], True)
        Model(units, tiles, rng.choice([1, 2, 3]), rng.choice([2, 3, 4]), rng).run()


@pytest.mark.parametrize("tiles,groups,pairs,chunks,stages", [(1, 1, 1, 1, 2), (3, 1, 2, 2, 3), (4, 2, 1, 3, 2), (2, 1, 4, 2, 4)])
def test_chosen_shapes_end_well(tiles, groups, pairs, chunks, stages):
    for seed in range(6):
        Model(Walk(0, 1, tiles, groups, pairs).units(), tiles, chunks, stages, random.Random(seed)).run()


@pytest.mark.parametrize("broken", ["a_empty", "b_empty", "a_full", "d_empty", "early", "release", "box"])
def test_planted_mistakes_are_caught(broken):
    caught = 0
    for seed in range(20):
        try:
            Model(Walk(0, 1, 6, 1, 2).units(), 6, 2, 3, random.Random(seed), broken).run()
        except Fault:
            caught += 1
    assert caught > 0
