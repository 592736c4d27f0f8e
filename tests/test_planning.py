"""The kernels' planning arithmetic itself, compiled for the host (tests/plan_host.cu) and compared with the masks.

* windows with first keys: the plan of a call (sink_plan), the backward items, the forward tile lists of all three
  kernels, and the float32 lists cover each tile with a visible pair once;
* the 8-bit cache: units of keys, equal shares of their line, places of pieces, the keys' order.

CPU only; a mistake in the headers that the kernels include fails here.
"""
import ctypes
import random
import subprocess
from pathlib import Path

import numpy as np
import pytest

from exact_io_aware_tiled_gb300 import _build

HERE = Path(__file__).resolve().parent
CSRC, INCLUDE = _build.CSRC, _build.PKG.parent / "include"
ALL, WINDOW, SINKS, FEW = range(4)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    try:
        nvcc = _build._nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    so = tmp_path_factory.mktemp("plan") / "libplan.so"
    subprocess.run([nvcc, *_build.ARCH, "-std=c++17", "-O1", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-shared",
                    "-I", str(CSRC), "-I", str(INCLUDE), str(HERE / "plan_host.cu"), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    for n in ("plan_items",):
        getattr(lib, n).restype = ctypes.c_longlong
    lib.plan_share.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p]
    lib.plan_owners.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    return lib


@pytest.fixture(scope="module")
def const(lib):
    out = (ctypes.c_int * 6)()
    lib.plan_constants(out)
    return dict(zip(("item_units", "group", "c_max", "tile", "few", "sub"), out))


def ptr(a):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


class Lists:
    """Row and column lists of a block mask, as the library makes them."""

    def __init__(self, keep):
        nb = self.nb = len(keep)
        self.rl, self.cl = (np.full((nb, nb), -1, dtype=np.int16) for _ in range(2))
        self.rc, self.cc = (np.zeros(nb, dtype=np.int32) for _ in range(2))
        for i in range(nb):
            r, c = np.flatnonzero(keep[i]), np.flatnonzero(keep[:, i])
            self.rl[i, :len(r)], self.rc[i] = r, len(r)
            self.cl[i, :len(c)], self.cc[i] = c, len(c)


class NoLists:
    nb, rl, cl, rc, cc = 0, None, None, None, None


def visible_tiles(N, causal, w, s, Lk, keep, T):
    """{(query tile, key tile)} with at least one visible pair."""
    i, j = np.arange(N)[:, None], np.arange(N)[None]
    see = np.broadcast_to(j < Lk, (N, N))
    if causal:
        see = see & (j <= i)
    if w:
        see = see & ((j > i - w) | (j < s))
    out = set()
    for a in range(-(-N // T)):
        for b in range(-(-N // T)):
            if (keep is None or keep[a, b]) and see[a * T:a * T + T, b * T:b * T + T].any():
                out.add((a, b))
    return out


def sink_plan(lib, B, H, Hkv, N, d, dtype, w, s):
    out = (ctypes.c_int * 7)()
    lib.plan_sink(B, H, Hkv, N, d, dtype, w, s, out)
    return dict(zip(("window", "sinks", "tiles", "chunks", "steps", "few", "few_chunks"), out))


def items(lib, kind, B, H, Hkv, N, causal, plan, lens, m):
    room = 1 << 20
    out = (ctypes.c_int * room)()
    n = lib.plan_items(kind, B, H, Hkv, N, causal, plan["window"], 0 if plan["few"] else plan["sinks"], plan["tiles"],
                       plan["chunks"], plan["steps"], ptr(lens), m.nb, ptr(m.rl), ptr(m.rc), ptr(m.cl), ptr(m.cc), out,
                       ctypes.c_longlong(room))
    assert n >= 0
    at, got = 0, []
    while at < n:
        b, hk, jt, part, per, steps = out[at:at + 6]
        at += 6
        got.append((b, hk, jt, part, per, [(out[at + 2 * t], out[at + 2 * t + 1]) for t in range(steps)]))
        at += 2 * steps
    return got


def problems(seed, n):
    rng = random.Random(seed)
    for _ in range(n):
        N = rng.choice([2, 127, 128, 129, rng.randint(2, 1400)])
        w = rng.choice([0, 1, N - 1, N, rng.randint(1, N), 2 ** 31 - 1])
        s = rng.choice([0, 1, 4, 8, 9, 128, 129, rng.randint(0, N + 3)])
        Hkv, g, B = rng.choice([1, 2, 3]), rng.choice([1, 2, 4]), rng.choice([1, 2, 3])
        lens = None
        if rng.random() < 0.5:
            lens = np.array([rng.choice([0, 1, N, rng.randint(0, N)]) for _ in range(B)], dtype=np.int32)
        keep = None
        if rng.random() < 0.4:
            nb = -(-N // 128)
            keep = np.array([[rng.random() < 0.6 for _ in range(nb)] for _ in range(nb)])
        yield N, w, s, B, Hkv * g, Hkv, lens, keep, rng.choice([0, 1, 2]), rng


def test_window_of_a_call(lib):
    for N, w, s, B, H, Hkv, _, _, dtype, _ in problems(1, 300):
        p = sink_plan(lib, B, H, Hkv, N, 64, dtype, w, s)
        hides = 0 < w < N
        assert p["window"] == (w if hides and s < N else 0)
        assert p["sinks"] == (s if hides and s < N else 0)
        if p["sinks"] == 0:
            assert p["tiles"] == p["chunks"] == p["few"] == 0
        elif p["few"]:
            assert dtype != 0 and p["few"] == s <= 8 and p["tiles"] == 0 and p["few_chunks"] >= 1
        else:
            assert p["tiles"] == -(-s // 128) and p["chunks"] >= 1 and p["steps"] >= 1
            steps = -(-N // 128) * (H // Hkv)
            assert (p["chunks"] - 1) * p["steps"] < steps <= p["chunks"] * p["steps"]


def test_backward_items_cover_every_visible_tile_once(lib, const):
    T = const["tile"]
    cut = False
    for N, w, s, B, H, Hkv, lens, keep, dtype, rng in problems(2, 250):
        causal = 1 if w else rng.choice([0, 1])
        p = sink_plan(lib, B, H, Hkv, N, 64, dtype, w, s)
        if p["chunks"] > 0 and rng.random() < 0.5:             # other cuts than the plan's hold too
            total = -(-N // T) * (H // Hkv)
            p["steps"] = rng.randint(1, total)
            p["chunks"] = -(-total // p["steps"])
        cut |= p["chunks"] > 1
        kind = FEW if p["few"] else SINKS if p["sinks"] else WINDOW if p["window"] else ALL
        m = NoLists if keep is None else Lists(keep)
        got = items(lib, kind, B, H, Hkv, N, causal, p, lens, m)
        nq = -(-N // T)
        done, parts = {}, {}
        for b, hk, jt, part, per, steps in got:
            for qt, h in steps:
                assert h // (H // Hkv) == hk
                key = (b, h, qt, jt)
                done[key] = done.get(key, 0) + 1
            if part >= 0:
                assert part not in parts
                parts[part] = (b, hk, jt, per, steps)
        assert all(n == 1 for n in done.values())
        for b in range(B):
            Lk = N if lens is None else int(lens[b])
            want = visible_tiles(N, causal, p["window"], 0 if p["few"] else p["sinks"], Lk, keep, T)
            for h in range(H):
                mine = {(q, j) for (bb, hh, q, j) in done if (bb, hh) == (b, h)}
                assert want <= mine
                assert all(keep is None or keep[q, j] for q, j in mine)
        # every key tile of every K/V head is written by one item, or by the parts that its sum reads
        written = [(b, hk, jt) for b, hk, jt, part, _, _ in got if part < 0 or kind == FEW]
        if kind == SINKS and p["chunks"] > 1:
            for u, (b, hk, jt, per, steps) in parts.items():
                assert u == ((b * Hkv + hk) * p["tiles"] + jt) * p["chunks"] + u % p["chunks"]
                used = min(p["chunks"], -(-per * (H // Hkv) // p["steps"]))
                assert (len(steps) > 0) == (u % p["chunks"] < used)
            written += [(b, hk, jt) for b in range(B) for hk in range(Hkv) for jt in range(p["tiles"])]
        assert sorted(written) == [(b, hk, jt) for b in range(B) for hk in range(Hkv) for jt in range(nq)]
        if kind == FEW:
            assert sorted(parts) == list(range(B * Hkv)) and all(v[2] == 0 for v in parts.values())
    assert cut


@pytest.mark.parametrize("which", [0, 1, 2])
def test_forward_lists_cover_every_visible_tile_once(lib, const, which):
    T = const["tile"]
    for N, w, s, B, H, Hkv, lens, keep, dtype, rng in problems(3 + which, 200):
        causal = 1 if w else rng.choice([0, 1])
        p = sink_plan(lib, 1, 1, 1, N, 64, dtype, w, s)
        m = NoLists if keep is None else Lists(keep)
        Lk = N if lens is None else int(lens[0])
        want = visible_tiles(N, causal, p["window"], p["sinks"], Lk, keep, T)
        for qt in range(-(-N // T)):
            out = (ctypes.c_int * 64)()
            n = lib.plan_forward(which, N, causal, p["window"], p["sinks"], Lk, m.nb, ptr(m.rl), ptr(m.rc), qt, out)
            got = list(out[:n])
            assert got == sorted(set(got)) and {j for q, j in want if q == qt} <= set(got)
            assert all(keep is None or keep[qt, j] for j in got)


def test_float32_lists_and_sub_tiles(lib, const):
    T, sub = const["tile"], const["sub"]
    for N, w, s, B, H, Hkv, lens, keep, _, rng in problems(9, 120):
        causal = 1 if w else rng.choice([0, 1])
        p = sink_plan(lib, 1, 1, 1, N, 64, 0, w, s)
        w, s = p["window"], p["sinks"]
        m = NoLists if keep is None else Lists(keep)
        Lk = N if lens is None else int(lens[0])
        want = visible_tiles(N, causal, w, s, Lk, keep, T)
        for jt in range(-(-N // T)):
            out = (ctypes.c_int * 64)()
            n = lib.plan_f32_backward(N, causal, w, s, Lk, m.nb, ptr(m.cl), ptr(m.cc), jt, out)
            got = list(out[:n])
            assert got == sorted(set(got)) and {q for q, j in want if j == jt} <= set(got)
        for _ in range(40):                       # a sub-tile that is left out has no visible pair
            rows = rng.choice([32, T])
            i0, j0 = rng.randrange(0, N + T, rows), rng.randrange(0, N + T, sub)
            i, j = np.arange(i0, i0 + rows)[:, None], np.arange(j0, j0 + sub)[None]
            see = np.ones((rows, sub), dtype=bool)
            if causal:
                see &= j <= i
            if w:
                see &= (j > i - w) | (j < s)
            if lib.plan_hidden(causal, w, s, j0, i0, rows):
                assert not see.any()


@pytest.mark.parametrize("KS", [32, 64])
def test_cache_units_cover_the_visible_keys_once(lib, const, KS):
    rng = random.Random(KS)
    for _ in range(600):
        cap = rng.choice([64, 304, 640])
        n, T = rng.choice([0, cap, cap + rng.randint(0, 400), rng.randint(0, 700)]), rng.randint(1, 9)
        window, sinks = rng.choice([0, rng.randint(1, 800), 2 ** 31 - 1]), rng.choice([0, 4, rng.randint(0, 800), 2 ** 31 - 1])
        out = (ctypes.c_int * 4)()
        lib.plan_units(KS, n, T, window, sinks, cap, out)
        units, ns, skip, line = out
        assert line == (units + const["item_units"] if units else 0)
        got = [(i if i < ns else i + skip) * KS for i in range(units)]
        L = min(n, cap)
        assert got == sorted(set(got)) and all(0 <= k < L for k in got)
        seen = {j for t in range(T) for p in [n - T + t] for j in range(min(p + 1, L))
                if window == 0 or j > p - window or j < sinks}
        assert seen <= {j for k in got for j in range(k, k + KS)}
        if n >= T:
            assert all(seen & set(range(k, k + KS)) for k in got)
        if window:
            for t in range(T):
                first = lib.plan_first_seen(window, n - T + t)
                assert first == max(0, n - T + t - window + 1)
    # lengths and windows at the end of int32
    for n, window in ((2 ** 31 - 1, 1), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        lib.plan_units(KS, n, 2 ** 26, window, 4, 640, out)
        assert 0 <= out[0] <= 640 // KS


def test_cache_line_shares_and_pieces(lib, const):
    cost, rng = const["item_units"], random.Random(2)
    for _ in range(300):
        segs = [rng.choice([1, 2, rng.randint(1, 300)]) for _ in range(rng.randint(1, 20))]
        X = sum(n + cost for n in segs)
        C = rng.randint(1, min(const["c_max"], X))
        begin = (ctypes.c_longlong * (C + 1))()
        lib.plan_share(X, C, begin)
        assert begin[0] == 0 and begin[C] == X
        assert max(begin[c + 1] - begin[c] for c in range(C)) - min(begin[c + 1] - begin[c] for c in range(C)) <= 1
        own = (ctypes.c_int * X)()
        lib.plan_owners(X, C, X, (ctypes.c_longlong * X)(*range(X)), own)
        assert all(begin[own[x]] <= x < begin[own[x] + 1] for x in range(X))
        at, begun, slots = cost, [], []
        for n in segs:
            c0, c1 = own[at], own[at + n - 1]
            if c1 > c0:
                begun.append(c0)
                # the place as the CTA itself takes it: by whether the rows begin in it
                mine = [2 * c + (1 if at >= begin[c] else 0) for c in range(c0, c1 + 1)]
                assert mine == [lib.plan_piece_slot(c0, c - c0) for c in range(c0, c1 + 1)]
                slots += mine
            assert (c1 == c0) == (at >= begin[c0] and at + n <= begin[c0 + 1])
            at += n + cost
        assert len(set(begun)) == len(begun) and len(set(slots)) == len(slots) and max(slots, default=0) < 2 * const["c_max"]
    # lines past 32 bits
    for X in (2 ** 31 - 1, 2 ** 31, 2 ** 40 + 7):
        C = const["c_max"]
        begin = (ctypes.c_longlong * (C + 1))()
        lib.plan_share(X, C, begin)
        xs = [x for c in range(C) for x in (begin[c], begin[c + 1] - 1)]
        own = (ctypes.c_int * len(xs))()
        lib.plan_owners(X, C, len(xs), (ctypes.c_longlong * len(xs))(*xs), own)
        assert begin[C] == X and list(own) == [c for c in range(C) for _ in range(2)]
    assert const["c_max"] <= 32 * const["group"]


@pytest.mark.parametrize("D", [64, 128])
def test_cache_key_order_meets_different_banks(lib, D):
    key = lambda m, e: lib.plan_key(D, m, e)  # noqa: E731
    assert sorted(key(m, e) for m in range(4) for e in range(2)) == list(range(8))

    def swizzled(row, byte):                 # the copy's pattern: 16-byte pieces by address bits 7 and up
        at = row * D + byte
        return at ^ ((at >> 3) & (0x30 if D == 64 else 0x70))

    def conflict_free(addresses, width):
        banks = [(a // 4 + i) % 32 for a in addresses for i in range(width // 4)]
        return len(set(banks)) == len(banks) == 32

    for h in range(D // 64):
        for p in range(4):
            assert conflict_free([swizzled(key((x // 4) >> 1, (x // 4) & 1), 64 * h + 16 * (x % 4))
                                  for x in range(8 * p, 8 * p + 8)], 16)
    w = D // 8
    for e in range(2):
        for p in range(w // 4):
            lanes = range(p * 128 // w, (p + 1) * 128 // w)
            assert conflict_free([swizzled(key(x % 4, e), w * (x // 4)) for x in lanes], w)
