"""The differential-attention kernels' barrier protocols, simulated on the CPU.

Forward (csrc/diff_fwd.cu): persistent CTAs, an item is one query tile with two
score maps.  A stage holds the K tiles of both maps (released by the S issuer)
and one V tile (released by both P V issuers); a stage's first use skips the
empty waits; a tile is worked in two halves h: S(h) waits until the softmax has
read S(h-1) and the product of half h - 2 is done, which frees P(h)'s place, O is rescaled after
that of half h - 1; the two softmax groups meet before and after they read both accumulators.

Backward (csrc/diff_bwd.cu): the roles of the d = 128 backward with a two-stage
Q / dO ring, K double-buffered per item and one V buffer, and W^T over S_1^T: the
S issuer waits for dV(g-1) before S_1(g), the compute warps do not wait for it.

tests/protocol_sim.py checks for deadlocks and for parity waits that pass early
or alias; here also that nothing reads a buffer that is being refilled.
Planted mistakes must fail.
"""
import random

import pytest

from tests.protocol_sim import Bar, Engine, ProtocolError

NS = 2


class Forward:
    """items: key tiles of each work item."""

    def __init__(self, items, rng, plant=None):
        self.items, self.plant = items, plant
        self.engine = Engine(rng)
        B = Bar
        self.item_full = [B("item_full%d" % i, 1) for i in range(2)]
        self.item_empty = [B("item_empty%d" % i, 5) for i in range(2)]      # S, two P V issuers, two softmax groups
        self.q_full, self.q_empty = B("q_full", 1), B("q_empty", 1)
        self.s_full, self.s_free = ([B("%s%d" % (n, x), 1) for x in range(2)] for n in ("s_full", "s_free"))
        self.p_full, self.pv_done = ([[B("%s%d%d" % (n, x, j), 1) for j in range(2)] for x in range(2)]
                                     for n in ("p_full", "pv_done"))
        self.k_full, self.v_full, self.k_empty = ([B("%s%d" % (n, i), 1) for i in range(NS)]
                                                  for n in ("k_full", "v_full", "k_empty"))
        self.v_empty = [B("v_empty%d" % i, 1 if plant == "v_one_reader" else 2) for i in range(NS)]
        self.meet = B("meet", 2)
        self.seed, self.issued = rng.randrange(1 << 30), [0, 0]
        self.mailbox = [None, None]
        self.reading = [False, False]      # a softmax group is reading both accumulators
        self.nloads = 0

    def load(self, bar):
        self.nloads += 1
        self.engine.later(("tma", self.nloads), bar)

    def producer(self):
        g = ni = 0
        for kf, u in enumerate(list(range(len(self.items))) + [-1]):
            slot = kf & 1
            if kf >= 2:
                yield ("wait", self.item_empty[slot], (kf >> 1) - 1)
            self.mailbox[slot] = (kf, u)
            self.item_full[slot].arrive()
            if u < 0:
                break
            if self.items[u] == 0:
                continue
            if ni >= 1:
                yield ("wait", self.q_empty, ni - 1)
            self.load(self.q_full)
            ni += 1
            for _ in range(self.items[u]):
                st = g % NS
                if g >= NS:
                    yield ("wait", self.k_empty[st], g // NS - 1)
                self.load(self.k_full[st])
                if g >= NS:
                    yield ("wait", self.v_empty[st], g // NS - 1)
                for x in range(2):
                    if g >= NS and self.pv_done[x][1].completed < g - NS + 1:
                        raise ProtocolError("V of step %d refilled before map %d read it" % (g - NS, x))
                self.load(self.v_full[st])
                g += 1
        for j in range(max(0, g - NS), g):
            yield ("wait", self.k_full[j % NS], j // NS)
            yield ("wait", self.v_full[j % NS], j // NS)
        if ni > 0:
            yield ("wait", self.q_full, ni - 1)

    def fetch(self, kc):
        yield ("wait", self.item_full[kc & 1], kc >> 1)
        k, u = self.mailbox[kc & 1]
        if k != kc:
            raise ProtocolError("mailbox slot of item %d overwritten" % kc)
        self.item_empty[kc & 1].arrive()
        return u

    def s_issuer(self):
        g = ni = kc = 0
        while True:
            u = yield from self.fetch(kc)
            kc += 1
            if u < 0:
                return
            if self.items[u] == 0:
                continue
            yield ("wait", self.q_full, ni)
            for _ in range(self.items[u]):
                yield ("wait", self.k_full[g % NS], g // NS)
                for j in range(2):
                    for x in range(2):
                        h = 2 * g + j
                        if h > 0 and self.plant != "s_ungated":
                            yield ("wait", self.s_free[x], h - 1)
                        if self.s_free[x].completed < h:
                            raise ProtocolError("S_%d(%d) written over scores not yet read" % (x, h))
                        if g > 0 and self.plant != "p_ungated":
                            yield ("wait", self.pv_done[x][j], g - 1)
                        self.engine.later("S", self.s_full[x])
                self.engine.later("S", self.k_empty[g % NS])
                g += 1
            self.engine.later("S", self.q_empty)
            ni += 1

    def pv_issuer(self, x):
        g = kc = 0
        while True:
            u = yield from self.fetch(kc)
            kc += 1
            if u < 0:
                return
            for s in range(self.items[u]):
                yield ("wait", self.v_full[g % NS], g // NS)
                for j in range(2):
                    yield ("wait", self.p_full[x][j], g)
                    if any(self.reading):
                        raise ProtocolError("P V_%d(%d) issued while the last O is being read" % (x, g))
                    self.issued[x] += 1
                    self.engine.later("PV%d" % x, self.pv_done[x][j])
                self.engine.later("PV%d" % x, self.v_empty[g % NS])
                g += 1

    def softmax(self, x):
        g = kc = nm = 0
        rng = random.Random(self.seed + x)
        while True:
            u = yield from self.fetch(kc)
            kc += 1
            if u < 0:
                return
            for s in range(self.items[u]):
                for j in range(2):
                    yield ("wait", self.s_full[x], 2 * g + j)
                    self.s_free[x].arrive()
                    if self.pv_done[x][j].completed < g:
                        raise ProtocolError("P_%d%d(%d) written under the product that reads it" % (x, j, g))
                    if (s > 0 or j > 0) and rng.random() < 0.5:      # the reference maximum moved: O is rescaled
                        if self.plant != "rescale_ungated":
                            yield ("wait", self.pv_done[x][j ^ 1], g if j else g - 1)
                        if self.pv_done[x][0].completed + self.pv_done[x][1].completed < self.issued[x]:
                            raise ProtocolError("O_%d rescaled under a product" % x)
                    self.p_full[x][j].arrive()
                g += 1
            if self.items[u] == 0:
                continue
            # the last product of the group's own map; the other's may be
            # phases behind, so it is learned from the barrier of both groups
            y = 1 - x if self.plant == "waits_for_other_map" else x
            yield ("wait", self.pv_done[y][1], g - 1)
            self.meet.arrive()
            yield ("wait", self.meet, nm)
            nm += 1
            self.reading[x] = True
            yield ("wait", self.meet, nm - 1)          # some time passes while O is read
            self.reading[x] = False
            if self.plant != "no_second_meet":
                self.meet.arrive()
                yield ("wait", self.meet, nm)
                nm += 1

    def run(self):
        self.engine.run({"P": self.producer(), "S": self.s_issuer(), "V0": self.pv_issuer(0), "V1": self.pv_issuer(1),
                         "X0": self.softmax(0), "X1": self.softmax(1)})


def test_forward_protocol():
    rng = random.Random(20260)
    for _ in range(300):
        Forward([rng.choice([0, 1, 1, 2, 3, 5, 9]) for _ in range(rng.randrange(0, 8))], random.Random(rng.random())).run()


@pytest.mark.parametrize("plant", ["v_one_reader", "s_ungated", "waits_for_other_map", "no_second_meet",
                                   "p_ungated", "rescale_ungated"])
def test_forward_planted_mistakes_are_caught(plant):
    rng = random.Random(3)
    for _ in range(400):
        try:
            Forward([rng.choice([1, 2, 3, 4]) for _ in range(6)], random.Random(rng.random()), plant=plant).run()
        except ProtocolError:
            return
    pytest.fail("not caught")


NQ = 2       # Q / dO ring stages


class Backward:
    def __init__(self, items, rng, plant=None):
        self.items, self.plant = items, plant
        B = Bar
        self.item_full = [B("item_full%d" % i, 1) for i in range(2)]
        self.item_empty = [B("item_empty%d" % i, 4) for i in range(2)]
        self.q_full = [B("q_full%d" % i, 1) for i in range(NQ)]
        self.q_empty = [B("q_empty%d" % i, 1) for i in range(NQ)]
        self.k_full = [B("k_full%d" % i, 1) for i in range(2)]
        self.k_empty = [B("k_empty%d" % i, 1 if plant == "k_one_reader" else 2) for i in range(2)]   # S and dQ issuers
        self.v_full, self.v_empty = B("v_full", 1), B("v_empty", 1)
        self.k_read = {}
        for n in ("s_full", "p_full", "dp_full", "ds_full", "dq_full", "dq_free", "dkv_full", "pt_free"):
            setattr(self, n, B(n, 1))
        self.dsm_free = B("dsm_free", 2)
        self.mailbox = [None, None]
        self.engine = Engine(rng)
        self.nloads = 0

    def commit(self, who, bar):
        self.engine.later(who, bar)

    def load(self, bar):
        self.nloads += 1
        self.engine.later(("tma", self.nloads), bar)

    def producer(self):
        g = kf = nkv = 0
        for u in list(range(len(self.items))) + [-1]:
            slot = kf & 1
            yield ("wait", self.item_empty[slot], (kf >> 1) - 1)
            self.mailbox[slot] = u
            self.item_full[slot].arrive()
            kf += 1
            if u < 0 or self.items[u] == 0:
                continue
            yield ("wait", self.k_empty[nkv & 1], (nkv >> 1) - 1)
            if nkv >= 2 and self.k_read.get(nkv - 2, 0) != 2:
                raise ProtocolError("K of item %d refilled before both readers finished" % (nkv - 2))
            self.load(self.k_full[nkv & 1])
            for t in range(self.items[u]):
                yield ("wait", self.q_empty[g % NQ], g // NQ - 1)
                self.load(self.q_full[g % NQ])
                g += 1
                if t == 0:
                    if self.plant != "v_ungated":
                        yield ("wait", self.v_empty, nkv - 1)
                    if self.v_empty.completed < nkv:
                        raise ProtocolError("V refilled under the last item's products")
                    self.load(self.v_full)
            nkv += 1
        for t in range(max(0, g - NQ), g):
            yield ("wait", self.q_full[t % NQ], t // NQ)
        for t in range(max(0, nkv - 2), nkv):
            yield ("wait", self.k_full[t & 1], t >> 1)
        if nkv:
            yield ("wait", self.v_full, nkv - 1)

    def fetch(self, kc):
        slot = kc & 1
        yield ("wait", self.item_full[slot], kc >> 1)
        v = self.mailbox[slot]
        self.item_empty[slot].arrive()
        return v

    def s_issuer(self):
        kc = g = nkv = 0
        while True:
            u = yield from self.fetch(kc)
            kc += 1
            if u < 0:
                return
            if self.items[u] == 0:
                continue
            yield ("wait", self.k_full[nkv & 1], nkv >> 1)
            for t in range(self.items[u]):
                if g > 0:
                    yield ("wait", self.p_full, g - 1)
                yield ("wait", self.q_full[g % NQ], g // NQ)
                if g > 0 and self.plant != "s1_ungated":
                    yield ("wait", self.pt_free, g - 1)
                if self.pt_free.completed < g:
                    raise ProtocolError("S_1(%d) written over W that dV still reads" % g)
                self.commit("S", self.s_full)
                if t == self.items[u] - 1:
                    self.k_read[nkv] = self.k_read.get(nkv, 0) + 1
                    self.commit("S", self.k_empty[nkv & 1])
                if g > 0:
                    yield ("wait", self.ds_full, g - 1)
                if t == 0:
                    yield ("wait", self.v_full, nkv)
                self.commit("S", self.dp_full)
                g += 1
            self.commit("S", self.v_empty)
            nkv += 1

    def dvdk_issuer(self):
        kc = g = 0
        while True:
            u = yield from self.fetch(kc)
            kc += 1
            if u < 0:
                return
            if self.items[u] == 0:
                continue
            for _ in range(self.items[u]):
                yield ("wait", self.p_full, g)
                yield ("wait", self.q_full[g % NQ], g // NQ)
                self.commit("D", self.pt_free)
                yield ("wait", self.ds_full, g)
                self.commit("D", self.dsm_free)
                self.commit("D", self.q_empty[g % NQ])
                g += 1
            self.commit("D", self.dkv_full)

    def dq_issuer(self):
        kc = g = nkv = 0
        while True:
            u = yield from self.fetch(kc)
            kc += 1
            if u < 0:
                return
            if self.items[u] == 0:
                continue
            if self.items[u] % 2:                 # some items end inside a tile: K is cleaned first
                yield ("wait", self.k_full[nkv & 1], nkv >> 1)
            for _ in range(self.items[u]):
                yield ("wait", self.ds_full, g)
                if g > 0:
                    yield ("wait", self.dq_free, g - 1)
                self.commit("Q", self.dq_full)
                self.commit("Q", self.dsm_free)
                g += 1
            self.k_read[nkv] = self.k_read.get(nkv, 0) + 1
            self.commit("Q", self.k_empty[nkv & 1])
            nkv += 1

    def compute(self):
        t = nit = kc = 0

        def drain(r):
            yield ("wait", self.dq_full, r)
            self.dq_free.arrive()

        while True:
            u = yield from self.fetch(kc)
            kc += 1
            if u < 0:
                break
            if self.items[u] == 0:
                continue
            for _ in range(self.items[u]):
                yield ("wait", self.s_full, t)
                yield ("wait", self.q_full[t % NQ], t // NQ)
                yield ("wait", self.dp_full, t)
                self.p_full.arrive()
                if t >= 1:
                    yield ("wait", self.dsm_free, t - 1)
                self.ds_full.arrive()
                if t > 0:
                    yield from drain(t - 1)
                t += 1
            yield ("wait", self.dkv_full, nit)
            nit += 1
        if t > 0:
            yield from drain(t - 1)

    def run(self):
        self.engine.run({"P": self.producer(), "S": self.s_issuer(), "D": self.dvdk_issuer(), "Q": self.dq_issuer(),
                         "C": self.compute()})


def _items(rng):
    return [rng.choice([0, 1, 2, 2, 3, 4, 5, 8, 16]) for _ in range(rng.randrange(1, 14))]


def test_backward_protocol():
    rng = random.Random(20261)
    for trial in range(400):
        Backward(_items(rng), random.Random(rng.random())).run()
    for items in ([1], [0], [0, 0, 1], [1, 0, 1, 0], [8], [1] * 12, [2] * 9, [0] * 5 + [2]):
        for seed in range(20):
            Backward(items, random.Random(seed)).run()


@pytest.mark.parametrize("plant", ["s1_ungated", "k_one_reader", "v_ungated"])
def test_backward_planted_mistakes_are_caught(plant):
    rng = random.Random(8)
    for trial in range(300):
        try:
            Backward(_items(rng), random.Random(rng.random()), plant=plant).run()
        except ProtocolError:
            return
    pytest.fail("not caught")
