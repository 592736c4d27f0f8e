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
