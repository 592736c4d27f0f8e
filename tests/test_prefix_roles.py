"""What tests/test_prefix_protocol.py's simulations leave out.

Tensor-memory kernel (csrc/prefix_tc.cu): the softmax waits for a product only
where a row's reference maximum moves, which is at random here.  P(h) lies where
P(h - 2) did, and only the S issuer's wait for the product of half h - 2 keeps
them apart; O is rescaled only after the product of half h - 1.

Register-product kernel (csrc/prefix.cu): a work item's stages go to the key
groups by their place in the ring, which depends on the items before; the order
in which the groups' parts are joined must not.

Planted mistakes must fail.
"""
import random

import pytest

from tests.protocol_sim import ProtocolError
from tests.test_prefix_protocol import TensorMemory, _slots

RINGS = [(False, 2), (False, 4), (False, 5), (True, 2), (True, 4)]


class Checked(TensorMemory):
    """The same roles with the waits of the kernel's softmax, and with the data they protect."""

    def __init__(self, tiles, fold, NS, rng, plant=None):
        super().__init__(tiles, fold, NS, rng, plant)
        self.moves = [random.Random(rng.randrange(1 << 30)) for _ in range(2)]
        self.issued = [0, 0]                        # products
        self.s_read = [0, 0]                        # halves whose scores are in registers

    def s_issuer(self, x):
        for s in range(self.tiles[x]):
            g = self.place(s, x)
            yield ("wait", self.k_full[g % self.NS], g // self.NS)
            for j in range(2):
                if s + j > 0:
                    yield ("wait", self.s_free[x], 2 * s + j - 1)
                if self.s_read[x] < 2 * s + j:
                    raise ProtocolError("S_%d(%d) written over scores not yet read" % (x, 2 * s + j))
                if s > 0 and self.plant != "p_ungated":
                    yield ("wait", self.pv_done[x][j], s - 1)
                self.engine.later("S%d" % x, self.s_full[x])
            self.engine.later("S%d" % x, self.k_empty[g % self.NS])

    def pv_issuer(self, x):
        for s in range(self.tiles[x]):
            g = self.place(s, x)
            yield ("wait", self.v_full[g % self.NS], g // self.NS)
            for j in range(2):
                yield ("wait", self.p_full[x][j], s)
                self.issued[x] += 1
                self.engine.later("PV%d" % x, self.pv_done[x][j])
            self.engine.later("PV%d" % x, self.v_empty[g % self.NS])

    def softmax(self, x):
        for s in range(self.tiles[x]):
            for j in range(2):
                yield ("wait", self.s_full[x], 2 * s + j)
                self.s_read[x] += 1
                self.s_free[x].arrive()
                if self.pv_done[x][j].completed < s:
                    raise ProtocolError("P_%d%d(%d) written under the product that reads it" % (x, j, s))
                if s + j > 0 and self.moves[x].random() < 0.5:
                    if self.plant != "rescale_ungated":
                        yield ("wait", self.pv_done[x][j ^ 1], s if j else s - 1)
                    if self.pv_done[x][0].completed + self.pv_done[x][1].completed < self.issued[x]:
                        raise ProtocolError("O_%d rescaled under a product" % x)
                self.p_full[x][j].arrive()
        yield ("wait", self.pv_done[x][1], self.tiles[x] - 1)
        if self.pv_done[x][0].completed + self.pv_done[x][1].completed < 2 * self.tiles[x]:
            raise ProtocolError("O_%d read under a product" % x)


@pytest.mark.parametrize("fold,NS", RINGS)
def test_tensor_memory(fold, NS):
    rng = random.Random(NS)
    for _ in range(400):
        Checked(_slots(rng, fold), fold, NS, random.Random(rng.random())).run()


@pytest.mark.parametrize("plant", ["p_ungated", "rescale_ungated"])
@pytest.mark.parametrize("fold,NS", RINGS)
def test_planted_mistakes_in_tensor_memory(fold, NS, plant):
    rng = random.Random(7)
    for _ in range(400):
        try:
            Checked(_slots(rng, fold), fold, NS, random.Random(rng.random()), plant=plant).run()
        except ProtocolError:
            return
    pytest.fail("not caught")


# ---- register-product kernel: the order of the joins --------------------------------------------------------
def joined(g0, nt, rgs, by_ring=False):
    """How row group 0's parts of an item of nt stages join in a CTA whose ring has run g0 stages: nested pairs of
    the item's stages (a pair: the second is added to the first)."""
    NS, kgs = 4, 4 // rgs
    parts, lw = {}, {}
    for kg in range(kgs):
        parts[kg] = tuple(t for t in range(nt) if (g0 + t) % NS & (kgs - 1) == kg)
        lw[kg] = kg * rgs if by_ring else ((kg - g0) & (kgs - 1)) * rgs
    at = {lw[kg]: parts[kg] for kg in range(kgs)}
    assert sorted(at) == [k * rgs for k in range(kgs)]
    half = 2
    while half >= rgs:
        for w in [w for w in at if half <= w < 2 * half]:
            at[w - half] = (at[w - half], at.pop(w))
        half //= 2
    assert list(at) == [0]
    return at[0]


@pytest.mark.parametrize("rgs", [1, 2, 4])
def test_joins_follow_from_the_item(rgs):
    for nt in range(1, 12):
        assert len({joined(g0, nt, rgs) for g0 in range(16)}) == 1
        first = joined(0, nt, rgs)
        assert joined(0, nt, rgs, by_ring=True) == first


@pytest.mark.parametrize("rgs", [1, 2])
def test_joins_by_the_ring_are_caught(rgs):
    assert any(len({joined(g0, nt, rgs, by_ring=True) for g0 in range(4)}) > 1 for nt in range(1, 12))
