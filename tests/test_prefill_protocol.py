"""Protocol model of the prefill kernel (csrc/prefill.cu), without a GPU.

The agents are the kernel's: the TMA thread, the warp that issues the scores'
MMAs, the one that issues P.V, the guard, and the softmax warps of both query tiles.  TMA
landings come in any order; each issuing warp's MMAs and commits run in order,
the two warps' in any interleaving.  mbarriers follow the hardware's rules
(arrivals, transaction bytes, phases told apart by their parity alone), and
every wait says which phase it means: one that passes early is an error.  Every
read is checked for the tile it expects, every write for readers that are not
done.  Random interleavings of small items (several, of different lengths, with
query tiles without keys) must end without deadlock; planted mistakes must not.

Values of tiles that some row does not attend whole (the last ones of an item)
land on a barrier of the guard warp, which looks them over before P.V may.
"""

import random

import pytest

ITEMS = 4          # places for items handed out
WARPS = 4          # softmax warps of a query tile


class Fault(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.done = count, count, 0, 0

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.done += 1
            self.pending = self.count

    def arrive(self, tx=0):
        if self.pending == 0:
            raise Fault("more arrivals than the phase takes")
        self.pending -= 1
        self.tx += tx
        self._turn()

    def land(self, tx):
        self.tx -= tx
        self._turn()

    def passes(self, parity):
        return (self.done & 1) != parity


def check(cond, what):
    if not cond:
        raise Fault(what)


class Model:
    def __init__(self, items, rng, broken=None):
        self.items, self.rng, self.broken = items, rng, broken
        B = Bar
        self.bar = dict(item_full=[B(1) for _ in range(ITEMS)], item_empty=[B(3 + 2 * WARPS) for _ in range(ITEMS)], edge_full=[B(1), B(1)],
                        k_full=[B(1), B(1)], k_empty=[B(1), B(1)], v_full=[B(1), B(1)], v_empty=[B(1), B(1)],
                        q_full=[B(1), B(1)], q_empty=[B(1), B(1)], s_full=[B(1), B(1)], s_free=[B(WARPS), B(WARPS)],
                        p_full=[B(WARPS), B(WARPS)], p_free=[B(1), B(1)], o_full=[B(1), B(1)])
        self.slot = [None] * ITEMS
        self.Q, self.K, self.V, self.S = [None] * 2, [None] * 2, [None] * 2, [None] * 2
        self.readers = {}                               # cell -> reads issued and not done
        self.s_left = [0, 0]                            # softmax warps that have the scores still to read
        self.P = [None] * WARPS
        self.O = [None] * 2
        self.o_left = [0, 0]                            # softmax warps that have the output still to read
        self.pipes = {"s": [], "v": []}
        self.landings = []
        self.stored = 0

    # a wait names a barrier, the parity the kernel computes and the phase it means
    def ready(self, w):
        name, at, parity, phase = w
        b = self.bar[name][at]
        if not b.passes(parity & 1):
            return False
        check(b.done > phase, f"{name}[{at}] passed before phase {phase}")
        return True

    def load(self, cell, at, tag, full):
        mem = getattr(self, cell)
        check(self.readers.get((cell, at), 0) == 0, f"{cell}[{at}] loaded while it is read")
        mem[at] = None
        full.arrive(tx=1)
        self.landings.append((mem, at, tag, full))

    def run_pipe(self, which):
        op = self.pipes[which].pop(0)
        if op[0] == "commit":
            op[1].arrive()
        elif op[0] == "s":
            _, i, it, j, st = op
            check(self.Q[i] == it and self.K[st] == (it, j), "scores of the wrong tiles")
            check(self.s_left[i] == 0, "scores overwritten before they were read")
            self.S[i], self.s_left[i] = (it, j), WARPS
            self.readers[("Q", i)] -= 1
            self.readers[("K", st)] -= 1
        else:
            _, i, it, j, st = op
            check(all(p == (i, it, j) for p in self.P), "P.V of other probabilities")
            check(self.V[st] == (it, j), "P.V of the wrong values")
            if j == 0:
                check(self.o_left[i] == 0, "output overwritten before it was stored")
            else:
                check(self.O[i] == (it, j - 1), "P.V out of order")
            self.O[i] = (it, j)
            if j + 1 == self.items[it][i]:
                self.o_left[i] = WARPS
            self.readers[("V", st)] -= 1
            self.readers[("P", 0)] -= 1
            self.readers[("O", i)] -= 1

    def read(self, cell, at):
        self.readers[(cell, at)] = self.readers.get((cell, at), 0) + 1

    # ----------------------------------------------------------------- agents
    def tma(self):
        bar, kn, vn, qn = self.bar, 0, 0, [0, 0]
        for given in range(len(self.items) + 1):
            slot = given % ITEMS
            if given >= ITEMS:
                yield ("item_empty", slot, given // ITEMS - 1, given // ITEMS - 1)
            self.slot[slot] = given if given < len(self.items) else -1
            bar["item_full"][slot].arrive()
            if given == len(self.items):
                return
            n0, n1 = self.items[given]
            n = max(n0, n1)

            def load_q(i):
                if qn[i] > 0 and self.broken != "q_empty":
                    yield ("q_empty", i, qn[i] - 1, qn[i] - 1)
                qn[i] += 1
                self.load("Q", i, given, bar["q_full"][i])

            def load_k(j):
                nonlocal kn
                st = kn & 1
                if kn >= 2 and self.broken != "k_empty":
                    yield ("k_empty", st, (kn >> 1) - 1, (kn >> 1) - 1)
                kn += 1
                self.load("K", st, (given, j), bar["k_full"][st])

            def load_v(j):
                nonlocal vn
                st = vn & 1
                if vn >= 2:
                    yield ("v_empty", st, (vn >> 1) - 1, (vn >> 1) - 1)
                vn += 1
                edge = j >= self.edge(given)
                self.load("V", st, (given, j, "raw") if edge else (given, j), bar["edge_full" if edge else "v_full"][st])
            if n == 0:
                continue
            if n0:
                yield from load_q(0)
            yield from load_k(0)
            if n1:
                yield from load_q(1)
            for j in range(n):
                if j + 1 < n:
                    yield from load_k(j + 1)
                yield from load_v(j)

    def edge(self, it):
        """The first tile of the item that some row does not attend whole."""
        n0, n1 = self.items[it]
        return max((n0 if n0 else n1) - 2, 0)

    def guard(self):
        bar, t, taken, e = self.bar, 0, 0, [0, 0]
        while True:
            it = yield from self.take(taken)
            if it < 0:
                return
            n = max(self.items[it])
            for j in range(self.edge(it), n):
                st = (t + j) & 1
                if self.broken != "guard":
                    yield ("edge_full", st, e[st], e[st])
                e[st] += 1
                check(self.V[st] == (it, j, "raw"), "the guard looks over another tile")
                yield None
                check(self.V[st] == (it, j, "raw") and self.readers.get(("V", st), 0) == 0, "values looked over while they are read")
                self.V[st] = (it, j)
                bar["v_full"][st].arrive()
            t += n
            bar["item_empty"][taken % ITEMS].arrive()
            taken += 1

    def take(self, taken):
        yield ("item_full", taken % ITEMS, taken // ITEMS, taken // ITEMS)
        return self.slot[taken % ITEMS]

    def scores(self):
        bar, t, taken, q, f = self.bar, 0, 0, [0, 0], [0, 0]
        while True:
            it = yield from self.take(taken)
            if it < 0:
                return
            nn = self.items[it]
            bar["item_empty"][taken % ITEMS].arrive()
            taken += 1
            n = max(nn)
            for x in range(2 * n):
                j, i = x >> 1, x & 1
                mine, other = nn[i], nn[i ^ 1]
                if j >= mine:
                    continue
                st = (t + j) & 1
                if i == 0 or j >= other:
                    yield ("k_full", st, (t + j) >> 1, (t + j) >> 1)
                if j == 0:
                    yield ("q_full", i, q[i], q[i])
                    q[i] += 1
                if self.broken != "s_free":
                    yield ("s_free", i, f[i] + 1, f[i] - 1)
                f[i] += 1
                self.read("Q", i)
                self.read("K", st)
                pipe = self.pipes["s"]
                pipe.append(("s", i, it, j, st))
                pipe.append(("commit", bar["s_full"][i]))
                if i == 1 or j >= other:
                    pipe.append(("commit", bar["k_empty"][st]))
                if j + 1 == mine:
                    pipe.append(("commit", bar["q_empty"][i]))
            t += n

    def pv(self):
        bar, t, taken, p = self.bar, 0, 0, [0, 0]
        while True:
            it = yield from self.take(taken)
            if it < 0:
                return
            nn = self.items[it]
            bar["item_empty"][taken % ITEMS].arrive()
            taken += 1
            n = max(nn)
            pipe = self.pipes["v"]
            if n:
                pipe.append(("commit", bar["p_free"][0 if nn[0] else 1]))
            for x in range(2 * n):
                j, i = x >> 1, x & 1
                mine, other = nn[i], nn[i ^ 1]
                if j >= mine:
                    continue
                st = (t + j) & 1
                if i == 0 or j >= other:
                    yield ("v_full", st, (t + j) >> 1, (t + j) >> 1)
                yield ("p_full", i, p[i], p[i])
                p[i] += 1
                self.read("V", st)
                self.read("P", 0)
                self.read("O", i)
                pipe.append(("v", i, it, j, st))
                nxt = (i ^ 1) if j + i < other else (i if j + 1 < mine else -1)
                if self.broken == "next":
                    nxt = i ^ 1 if other else i
                if nxt >= 0:
                    pipe.append(("commit", bar["p_free"][nxt]))
                if i == 1 or j >= other:
                    pipe.append(("commit", bar["v_empty"][st]))
                if j + 1 == mine:
                    pipe.append(("commit", bar["o_full"][i]))
            t += n

    def softmax(self, i, w):
        bar, taken, sn, on = self.bar, 0, 0, 0
        while True:
            it = yield from self.take(taken)
            if it < 0:
                return
            n = self.items[it][i]
            for j in range(n):
                yield ("s_full", i, sn, sn)
                sn += 1
                check(self.S[i] == (it, j), "softmax of other scores")
                yield None
                check(self.S[i] == (it, j) and self.s_left[i] > 0, "scores changed while they were read")
                self.s_left[i] -= 1
                bar["s_free"][i].arrive()
                yield None
                if self.broken != "p_free":
                    yield ("p_free", i, sn - 1, sn - 1)
                if j and self.rng.random() < 0.3:           # a rescale of the output
                    check(self.readers.get(("O", i), 0) == 0 and self.O[i] == (it, j - 1), "rescaled during a P.V")
                check(self.readers.get(("P", 0), 0) == 0, "probabilities overwritten during a P.V")
                self.P[w] = (i, it, j)
                yield None
                bar["p_full"][i].arrive()
            if n:
                if self.broken != "o_full":
                    yield ("o_full", i, on, on)
                on += 1
                check(self.O[i] == (it, n - 1) and self.readers.get(("O", i), 0) == 0, "output stored before its last P.V")
                yield None
                self.o_left[i] -= 1
            self.stored += 1
            bar["item_empty"][taken % ITEMS].arrive()
            taken += 1

    def run(self):
        agents = [self.tma(), self.scores(), self.pv(), self.guard()] + [self.softmax(i, w) for i in range(2) for w in range(WARPS)]
        waits = [None] * len(agents)
        live = set(range(len(agents)))
        for _ in range(200000):
            moves = [("agent", a) for a in live if waits[a] is None or self.ready(waits[a])]
            moves += [("pipe", k) for k in self.pipes if self.pipes[k]]
            moves += [("land", k) for k in range(len(self.landings))]
            if not moves:
                check(not live, "deadlock")
                check(self.stored == 2 * WARPS * len(self.items), "an item was lost")
                return
            kind, x = self.rng.choice(moves)
            if kind == "pipe":
                self.run_pipe(x)
            elif kind == "land":
                mem, at, tag, full = self.landings.pop(x)
                mem[at] = tag
                full.land(1)
            else:
                try:
                    waits[x] = next(agents[x])
                except StopIteration:
                    live.discard(x)
        raise Fault("does not end")


def random_items(rng):
    items = []
    for _ in range(rng.randint(1, 7)):
        n0 = rng.randint(0, 4)
        items.append(rng.choice([(n0, 0), (n0, n0), (n0, n0 + 1), (n0, n0 + 2)]))
    return items


@pytest.mark.parametrize("seed", range(12))
def test_random_interleavings_end_well(seed):
    rng = random.Random(seed)
    for _ in range(25):
        Model(random_items(rng), rng).run()


@pytest.mark.parametrize("items", [[(0, 0)], [(1, 0)] * 9, [(0, 2), (0, 0), (3, 0), (0, 1), (2, 2)], [(5, 5)], [(1, 3)] * 4])
def test_chosen_items_end_well(items):
    for seed in range(20):
        Model(items, random.Random(seed)).run()


@pytest.mark.parametrize("broken", ["q_empty", "k_empty", "s_free", "p_free", "next", "o_full", "guard"])
def test_planted_mistakes_are_caught(broken):
    caught = 0
    for seed in range(30):
        rng = random.Random(seed)
        try:
            Model([(2, 3), (3, 4), (2, 2), (1, 0), (3, 3)], rng, broken).run()
        except Fault:
            caught += 1
    assert caught > 0
