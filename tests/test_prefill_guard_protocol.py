"""Protocol model of the guard's notes in the prefill kernel (csrc/prefill.cu),
without a GPU: which tokens of an item's last value tiles are not finite, noted
by the guard warp and read by the softmax warps when they store.

The notes of an item (one word a tile here) are reset when the guard takes the
item and written tile by tile, before the guard lets P.V have the tile.  A
softmax warp may read the notes of the tiles that its own query tile works off:
its last P.V is done, so the guard is done with them.  Of the others it knows
nothing: an item without such tiles may be stored before the guard has taken it,
and the other query tile's may still be written.
"""

import random

import pytest

from .test_prefill_protocol import ITEMS, Fault, Model, check


class Noted(Model):
    """edges: for every item the first tile that some row does not attend whole (no less than its tiles: none)."""

    def __init__(self, items, edges, rng, broken=None):
        super().__init__(items, rng, broken)
        self.edges = edges
        self.notes = [[None] * 5 for _ in range(ITEMS)]

    def edge(self, it):
        return self.edges[it]

    def guard(self):
        bar, t, taken, e = self.bar, 0, 0, [0, 0]
        while True:
            it = yield from self.take(taken)
            if it < 0:
                return
            mine = self.notes[taken % ITEMS]
            yield None
            for x in range(5):
                mine[x] = None
            for j in range(self.edge(it), max(self.items[it])):
                st = (t + j) & 1
                yield ("edge_full", st, e[st], e[st])
                e[st] += 1
                yield None
                if self.broken != "late":
                    mine[j - self.edge(it)] = (it, j)
                self.V[st] = (it, j)
                bar["v_full"][st].arrive()
                if self.broken == "late":
                    for _ in range(60):
                        yield None
                    mine[j - self.edge(it)] = (it, j)
            t += max(self.items[it])
            bar["item_empty"][taken % ITEMS].arrive()
            taken += 1

    def softmax(self, i, w):
        bar, taken, sn, on = self.bar, 0, 0, 0
        while True:
            it = yield from self.take(taken)
            if it < 0:
                return
            n, slot = self.items[it][i], taken % ITEMS
            for j in range(n):
                yield ("s_full", i, sn, sn)
                sn += 1
                self.s_left[i] -= 1
                bar["s_free"][i].arrive()
                yield ("p_free", i, sn - 1, sn - 1)
                self.P[w] = (i, it, j)
                yield None
                bar["p_full"][i].arrive()
            if n:
                yield ("o_full", i, on, on)
                on += 1
            tiles = range(5) if self.broken == "all" else range(max(n - self.edge(it), 0) if n else 0)
            for x in tiles:
                yield None
                check(self.notes[slot][x] == (it, self.edge(it) + x), "notes read that the guard has not written")
            if n:
                self.o_left[i] -= 1
            self.stored += 1
            bar["item_empty"][slot].arrive()
            taken += 1


def random_items(rng):
    """Query tiles of an item with their key tiles, and its first edge tile: none, or in front of both tiles' ends."""
    items, edges = [], []
    for _ in range(rng.randint(1, 7)):
        n0, more, both = rng.randint(0, 4), rng.randint(0, 2), rng.random() < 0.7
        n1 = n0 + more if both else 0
        first = min(x for x in (n0, n1) if x) if n0 or n1 else 0
        items.append((n0, n1))
        if n0 == n1 or not n0 or not n1:
            edges.append(rng.choice([max(n0, n1), max(first - 1, 0), max(first - 3, 0)]))
        else:
            edges.append(max(first - rng.randint(1, 2), 0))
    return items, edges


@pytest.mark.parametrize("seed", range(12))
def test_notes_are_read_after_the_guard_wrote_them(seed):
    rng = random.Random(seed)
    for _ in range(25):
        Noted(*random_items(rng), rng).run()


@pytest.mark.parametrize("items,edges", [([(2, 2)] * 6, [2] * 6), ([(0, 0)] * 9, [0] * 9), ([(1, 3)] * 5, [0] * 5), ([(4, 5), (3, 0)] * 3, [2, 3] * 3)])
def test_chosen_items(items, edges):
    for seed in range(20):
        Noted(items, edges, random.Random(seed)).run()


@pytest.mark.parametrize("broken,items,edges", [
    ("all", [(2, 2)] * 6, [2] * 6),          # every note of an item that has none
    ("all", [(1, 3)] * 5, [0] * 5),          # the other query tile's notes too
    ("late", [(2, 3)] * 5, [0] * 5),         # notes written after P.V has the tile
])
def test_planted_mistakes_are_caught(broken, items, edges):
    caught = 0
    for seed in range(30):
        try:
            Noted(items, edges, random.Random(seed), broken).run()
        except Fault as e:
            caught += "notes read" in str(e)
    assert caught > 0
