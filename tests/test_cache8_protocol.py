"""The barrier protocol of the attention over the 8-bit cache (csrc/cache8.cu), simulated on the CPU.

Warp 4 issues stages four at a time: all its lanes wait until the four places of the ring are free, then each lane
publishes the item that begins with its stage (a mailbox of eight slots) and starts its copies; nothing orders the
lanes.  The four compute warps form 1, 2 or 4 row groups and 4, 2 or 1 key groups; a stage belongs to one key group,
whose warps release it for all four.  They meet at a barrier of their own to join key groups and to hand over rows that
were cut.  tests/protocol_sim.py checks for deadlocks and for parity waits that pass early or alias; here also that a
stage is refilled, a mailbox slot rewritten and a join buffer overwritten only after their readers.  Planted mistakes
must fail.
"""
import random

import pytest

from tests.protocol_sim import Bar, Engine, ProtocolError

NS, SLOTS = 8, 8


class Cta:
    def __init__(self, items, rgs, rng, plant=None):
        self.items, self.rgs, self.kgs, self.rng, self.plant = items, rgs, 4 // rgs, rng, plant    # (stages, meets behind)
        self.slots = 2 if plant == "two_slots" else SLOTS
        self.engine = Engine(rng)
        self.full = [Bar("full%d" % i, 2) for i in range(NS)]                 # the copies with their bytes, the record
        self.empty = [Bar("empty%d" % i, 3 if plant == "three_readers" else 4) for i in range(NS)]
        self.item_full = [Bar("item_full%d" % i, 1) for i in range(self.slots)]
        self.item_empty = [Bar("item_empty%d" % i, 4) for i in range(self.slots)]
        self.join = Bar("join", 4)
        self.mailbox, self.buffer = {}, {}
        self.read, self.got, self.records = {}, {}, {}
        self.loads = 0

    def publish(self, kk, what):
        slot = kk % self.slots
        if kk >= self.slots and self.got.get(kk - self.slots, 0) != 4:
            raise ProtocolError("mailbox slot of item %d rewritten before every warp read it" % (kk - self.slots))
        self.mailbox[slot] = (kk, what)
        self.item_full[slot].arrive()

    def loader(self):
        stages = [(u, t) for u, (n, _) in enumerate(self.items) for t in range(n)]
        g0 = 0
        for i0 in range(0, len(stages), 4):
            batch = stages[i0:i0 + 4]
            for y in range(len(batch)):
                if g0 + y >= NS and self.plant != "ring_ungated":
                    yield ("wait", self.empty[(g0 + y) % NS], (g0 + y) // NS - 1)
            order = list(range(len(batch)))
            self.rng.shuffle(order)                      # lanes in any order, one held up holds up the others
            for y in order:
                (u, t), gi = batch[y], g0 + y
                if t == 0:
                    if u >= self.slots and self.plant != "mailbox_ungated":
                        yield ("wait", self.item_empty[u % self.slots], u // self.slots - 1)
                    self.publish(u, self.items[u])
                if gi >= NS and self.read.get(gi - NS, 0) != 4:
                    raise ProtocolError("stage %d refilled before every warp let it go" % (gi - NS))
                self.loads += 1
                self.engine.later(("tma", self.loads), self.full[gi % NS])
                self.records[gi] = True
                self.full[gi % NS].arrive()
            g0 += len(batch)
        u = len(self.items)
        if u >= self.slots:
            yield ("wait", self.item_empty[u % self.slots], u // self.slots - 1)
        self.publish(u, None)
        for j in range(max(0, g0 - NS), g0):
            yield ("wait", self.full[j % NS], j // NS)

    def warp(self, w):
        rg, kg = w % self.rgs, w // self.rgs
        g = nj = kc = 0
        while True:
            slot = kc % self.slots
            yield ("wait", self.item_full[slot], kc // self.slots)
            k, what = self.mailbox[slot]
            if k != kc:
                raise ProtocolError("mailbox slot of item %d overwritten" % kc)
            self.got[kc] = self.got.get(kc, 0) + 1
            self.item_empty[slot].arrive()
            if what is None:
                return
            nt, behind = what
            lk = (kg - g) % self.kgs
            lw, busy = lk * self.rgs + rg, lk < nt
            for _ in range(nt):
                st = g % NS
                if st % self.kgs == kg:
                    yield ("wait", self.full[st], g // NS)
                    assert self.records[g] and busy
                    for _ in range(self.kgs):
                        self.read[g] = self.read.get(g, 0) + 1
                        self.empty[st].arrive()
                g += 1
            half = 2
            while half >= self.rgs:
                groups = half // self.rgs
                if nt > groups:
                    if busy and half <= lw < 2 * half:
                        if self.buffer.get(lw - half) is not None:
                            raise ProtocolError("join buffer %d overwritten before it was read" % (lw - half))
                        self.buffer[lw - half] = (kc, half)
                    self.join.arrive()
                    yield ("wait", self.join, nj)
                    nj += 1
                    if busy and lw < half and lk + groups < nt:
                        if self.buffer.get(lw) != (kc, half):
                            raise ProtocolError("join of item %d reads buffer %d early" % (kc, lw))
                        self.buffer[lw] = None
                    if self.plant != "one_meeting":
                        self.join.arrive()
                        yield ("wait", self.join, nj)
                        nj += 1
                half //= 2
            for _ in range(behind):                      # rows that were cut: two meetings for each counter
                self.join.arrive()
                yield ("wait", self.join, nj)
                nj += 1
            kc += 1

    def run(self):
        roles = {"P": self.loader()}
        roles.update({"W%d" % w: self.warp(w) for w in range(4)})
        self.engine.run(roles)
        n = sum(n for n, _ in self.items)
        assert all(self.read[g] == 4 for g in range(n)) and all(v is None for v in self.buffer.values())


def _items(rng):
    n = rng.choice([1, 2, 5, 30])
    # the first and last items of a CTA may be cut: their rows are handed over
    return [(rng.choice([1, 1, 1, 2, 3, 4, 7, 9, 17, 40]), rng.choice([2, 4]) if u in (0, n - 1) else 0) for u in range(n)]


@pytest.mark.parametrize("rgs", [1, 2, 4])
def test_protocol(rgs):
    rng = random.Random(rgs)
    for _ in range(250):
        Cta(_items(rng), rgs, random.Random(rng.random())).run()
    for n in (1, 7, 8, 9, 40):                           # one stage an item: the mailbox at its fullest
        for _ in range(20):
            Cta([(1, 0)] * n, rgs, random.Random(rng.random())).run()


@pytest.mark.parametrize("plant", ["three_readers", "ring_ungated", "mailbox_ungated", "two_slots", "one_meeting"])
def test_planted_mistakes_are_caught(plant):
    rng = random.Random(7)
    for i in range(300):
        try:
            Cta(_items(rng) if i % 2 else [(1, 0)] * 40, rng.choice([1, 2]), random.Random(rng.random()), plant=plant).run()
        except ProtocolError:
            return
    pytest.fail("not caught")
