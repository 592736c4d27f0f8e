"""The shared-prefix kernel's barrier protocol, simulated on the CPU.

Persistent CTAs (csrc/prefix.cu): a producer claims items, publishes them
through a two-slot mailbox and streams their tiles into a ring that runs on
across items.  Four compute warps form 1, 2 or 4 row groups and 4, 2 or 1 key
groups; a stage belongs to one key group, whose warps release it for all four
(the others do not wait on it), and the warps of an item with several key groups
meet at a barrier of their own to join them.
tests/protocol_sim.py checks for deadlocks and for parity waits that pass early
or alias; here also that a stage is refilled only after all warps read it and
that a mailbox slot still holds its item.  Planted mistakes must fail.
"""
import random

import pytest

from tests.protocol_sim import Bar, Engine, ProtocolError


class Persistent:
    def __init__(self, items, NS, rng, plant=None):
        self.items, self.NS, self.plant = items, NS, plant      # (tiles, row groups)
        self.engine = Engine(rng)
        self.full = [Bar("full%d" % i, 1) for i in range(NS)]
        self.empty = [Bar("empty%d" % i, 3 if plant == "three_readers" else 4) for i in range(NS)]
        self.item_full = [Bar("item_full%d" % i, 1) for i in range(2)]
        self.item_empty = [Bar("item_empty%d" % i, 4) for i in range(2)]
        self.join = Bar("join", 4)
        self.mailbox = [None, None]
        self.read = {}
        self.nloads = 0

    def producer(self):
        g = kf = 0
        for u in list(range(len(self.items))) + [-1]:
            if u >= 0 and self.items[u][0] == 0:
                continue
            slot = kf & 1
            if kf >= 2 and self.plant != "mailbox_ungated":
                yield ("wait", self.item_empty[slot], (kf >> 1) - 1)
            self.mailbox[slot] = (kf, u)
            self.item_full[slot].arrive()
            kf += 1
            if u < 0:
                break
            for _ in range(self.items[u][0]):
                st = g % self.NS
                if g >= self.NS:
                    yield ("wait", self.empty[st], g // self.NS - 1)
                    if self.read.get(g - self.NS, 0) != 4:
                        raise ProtocolError("tile %d refilled before every warp read it" % (g - self.NS))
                self.nloads += 1
                self.engine.later(("tma", self.nloads), self.full[st])
                g += 1
        for j in range(max(0, g - self.NS), g):
            yield ("wait", self.full[j % self.NS], j // self.NS)

    def warp(self, w):
        g = kc = nj = 0
        while True:
            yield ("wait", self.item_full[kc & 1], kc >> 1)
            k, u = self.mailbox[kc & 1]
            if k != kc:
                raise ProtocolError("mailbox slot of item %d overwritten" % kc)
            self.item_empty[kc & 1].arrive()
            kc += 1
            if u < 0:
                return
            for _ in range(self.items[u][0]):
                rgs = self.items[u][1]
                kgs = 4 // rgs
                mine = g % self.NS % kgs == w // rgs
                if mine or self.plant == "waits_for_all":
                    yield ("wait", self.full[g % self.NS], g // self.NS)
                if mine:
                    for _ in range(kgs):
                        self.read[g] = self.read.get(g, 0) + 1
                        self.empty[g % self.NS].arrive()
                g += 1
            half = 2
            while half >= self.items[u][1] and self.plant != "no_join":
                for _ in range(2):
                    self.join.arrive()
                    yield ("wait", self.join, nj)
                    nj += 1
                half //= 2

    def run(self):
        roles = {"P": self.producer()}
        roles.update({"W%d" % w: self.warp(w) for w in range(4)})
        self.engine.run(roles)


def _items(rng):
    return [(rng.choice([0, 1, 1, 2, 4, 7, 9]), rng.choice([1, 2, 4])) for _ in range(rng.randrange(0, 12))]


@pytest.mark.parametrize("NS", [4, 8])
def test_persistent_protocol(NS):
    rng = random.Random(NS)
    for _ in range(300):
        Persistent(_items(rng), NS, random.Random(rng.random())).run()


@pytest.mark.parametrize("plant", ["three_readers", "mailbox_ungated", "waits_for_all", "no_join"])
def test_planted_mistakes_are_caught(plant):
    rng = random.Random(5)
    for _ in range(400):
        try:
            Persistent(_items(rng), 4, random.Random(rng.random()), plant=plant).run()
        except ProtocolError:
            return
    pytest.fail("not caught")


class TensorMemory:
    """csrc/prefix_tc.cu: one item a CTA.  Two slots share the ring's tiles, or
    (folded) own its even and odd stages and work at key ranges of their own."""

    def __init__(self, tiles, fold, NS, rng, plant=None):
        self.tiles, self.fold, self.NS, self.plant = tiles, fold, NS, plant
        self.nact = len(tiles)
        self.engine = Engine(rng)
        users = self.nact if not fold or plant == "both_release" else 1
        bars = lambda name, count: [Bar("%s%d" % (name, i), count) for i in range(NS)]
        self.k_full, self.v_full = bars("k_full", 1), bars("v_full", 1)
        self.k_empty, self.v_empty = bars("k_empty", users), bars("v_empty", users)
        self.s_full = [Bar("s_full%d" % x, 1) for x in range(2)]
        self.s_free = [Bar("s_free%d" % x, 1) for x in range(2)]
        self.p_full = [[Bar("p_full%d%d" % (x, j), 1) for j in range(2)] for x in range(2)]
        self.pv_done = [[Bar("pv_done%d%d" % (x, j), 1) for j in range(2)] for x in range(2)]
        self.loads = 0

    def place(self, s, x):
        return 2 * s + x if self.fold else s

    def load(self, bar):
        self.loads += 1
        self.engine.later(("tma", self.loads), bar)

    def producer(self):
        NS = self.NS
        for s in range(self.tiles[0]):
            for x in range(self.nact if self.fold else 1):
                if s >= self.tiles[x]:
                    continue
                g = self.place(s, x)
                for full, empty in ((self.k_full, self.k_empty), (self.v_full, self.v_empty)):
                    if g >= NS:
                        yield ("wait", empty[g % NS], g // NS - 1)
                    self.load(full[g % NS])
        own = NS // 2 if self.fold else NS
        for x in range(self.nact if self.fold else 1):
            for full in (self.k_full, self.v_full):
                for s in range(max(0, self.tiles[x] - own), self.tiles[x]):
                    yield ("wait", full[self.place(s, x) % NS], self.place(s, x) // NS)

    def s_issuer(self, x):
        for s in range(self.tiles[x]):
            g = self.place(s, x)
            yield ("wait", self.k_full[g % self.NS], g // self.NS)
            for j in range(2):
                if s + j > 0 and self.plant != "no_s_free":
                    yield ("wait", self.s_free[x], 2 * s + j - 1)
                if s > 0:
                    yield ("wait", self.pv_done[x][j], s - 1)
                self.engine.later("S%d" % x, self.s_full[x])
            self.engine.later("S%d" % x, self.k_empty[g % self.NS])

    def pv_issuer(self, x):
        for s in range(self.tiles[x]):
            g = self.place(s, x)
            yield ("wait", self.v_full[g % self.NS], g // self.NS)
            for j in range(2):
                yield ("wait", self.p_full[x][j], s)
                self.engine.later("PV%d" % x, self.pv_done[x][j])
            self.engine.later("PV%d" % x, self.v_empty[g % self.NS])

    def softmax(self, x):
        for s in range(self.tiles[x]):
            for j in range(2):
                yield ("wait", self.s_full[x], 2 * s + j)
                self.s_free[x].arrive()
                if s + j > 0:
                    yield ("wait", self.pv_done[x][j ^ 1], s if j else s - 1)
                self.p_full[x][j].arrive()
        yield ("wait", self.pv_done[x][1], self.tiles[x] - 1)

    def run(self):
        roles = {"P": self.producer()}
        for x in range(self.nact):
            roles.update({"S%d" % x: self.s_issuer(x), "PV%d" % x: self.pv_issuer(x), "W%d" % x: self.softmax(x)})
        self.engine.run(roles)


def _slots(rng, fold):
    n = rng.randrange(1, 9)
    return rng.choice([(n,), (n, rng.randrange(1, n + 1) if fold else n)])


@pytest.mark.parametrize("fold,NS", [(False, 2), (False, 4), (False, 5), (True, 2), (True, 4)])
def test_tensor_memory_protocol(fold, NS):
    rng = random.Random(NS)
    for _ in range(300):
        TensorMemory(_slots(rng, fold), fold, NS, random.Random(rng.random())).run()


@pytest.mark.parametrize("plant,NS", [("both_release", 4), ("no_s_free", 4), ("odd_ring", 5)])
def test_planted_mistakes_are_caught_in_tensor_memory(plant, NS):
    rng = random.Random(6)
    for _ in range(400):
        try:
            TensorMemory(_slots(rng, True), True, NS, random.Random(rng.random()), plant=plant).run()
        except ProtocolError:
            return
    pytest.fail("not caught")
