"""Paged cache in 8 bits (fa_cache8_append, fa_cache8_read, fa_cache8_fwd).

CPU: struct layout, refusals, the cut of the work into pieces, the keys' order in shared memory.  GPU: codes and scales
bit for bit against a plain form, attention against a 64-bit one.

Tolerances of the attention.  delta = 2^-19 (1 + tau sum |q k|) bounds a weight's relative error from its score: float32
products and sums of d terms, the scale's product and the exponent's rounding.  Weights are rounded to 11 bits (2^-11;
below 2^-14 of the largest by 2^-25 of it), O once more: |error| <= (2^-11 + 2 delta + 2^-20) sum P |v| + u |O| +
2^-25 sum |code| / sum exp2(s - t_max), t_max the largest s + log2(V scale; 2^-64 for a page of zeros).  lse: delta + 2^-20 (1 + |lse|).
"""
import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from exact_io_aware_tiled_gb300 import _cache8, _ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load()


# ---- CPU -------------------------------------------------------------------------------------------------------
def test_params_layout_matches_c(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    st = _cache8.fa_cache8_params
    prog = ['#include <stdio.h>', '#include <stddef.h>', '#include "fa.h"', 'int main(void){',
            'printf("%zu\\n", sizeof(fa_cache8_params));']
    prog += ['printf("%%zu\\n", offsetof(fa_cache8_params, %s));' % f for f, _ in st._fields_] + ['return 0;}']
    c = tmp_path / "l.c"
    c.write_text("\n".join(prog))
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(c), "-o", str(tmp_path / "l")], check=True)
    vals = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True).stdout.split()]
    assert vals == [ctypes.sizeof(st)] + [getattr(st, f).offset for f, _ in st._fields_]


def _params(**kw):
    p = _cache8.fa_cache8_params()
    p.B, p.H, p.H_kv, p.T, p.d, p.dtype, p.page, p.pages, p.width = 3, 4, 2, 2, 64, 2, 32, 20, 6
    p.table_stride, p.seqlens_k, p.table = 6, 1 << 22, 1 << 22
    for t, h in (("q", 4), ("o", 4), ("k", 2), ("v", 2)):
        for x, v in (("n", 64), ("h", 128), ("b", 128 * h)):
            setattr(p, "%s_stride_%s" % (t, x), v)
    for t in ("kc", "vc"):
        for x, v in (("n", 64), ("h", 2048), ("p", 4096)):
            setattr(p, "%s_stride_%s" % (t, x), v)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _rows(name, p, ptrs=None):
    f = _ops._fn(name, *([ctypes.c_void_p] * 8))
    x = [1 << 20] * 6
    for i, v in (ptrs or {}).items():
        x[i] = v
    return f(None if p is None else ctypes.addressof(p), *x, None)


def _fwd(p, ptrs=None, ws=1 << 40, ws_ptr=1 << 21):
    f = _ops._fn("fa_cache8_fwd", *([ctypes.c_void_p] * 9), ctypes.c_size_t, ctypes.c_void_p)
    x = [1 << 20] * 7
    for i, v in (ptrs or {}).items():
        x[i] = v
    return f(None if p is None else ctypes.addressof(p), *x, ws_ptr, ws, None)


ALL = [
    (dict(B=0), 1), (dict(H=0), 1), (dict(T=0), 1), (dict(d=0), 1), (dict(H_kv=-1), 1), (dict(H_kv=3), 1),
    (dict(pages=0), 1), (dict(width=0), 1), (dict(dtype=5), 1), (dict(dtype=0), 2), (dict(d=96), 2), (dict(page=48), 2),
    (dict(page=8), 2), (dict(page=256), 2), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(table_stride=5), 1),
    (dict(seqlens_k=0), 1), (dict(table=0), 1), (dict(table=(1 << 22) + 2), 3), (dict(seqlens_k=(1 << 22) + 1), 3),
    (dict(B=1 << 30), 2), (dict(width=1 << 24, table_stride=1 << 24), 2), (dict(pages=1 << 30), 2),
    (dict(kc_stride_n=48), 1), (dict(kc_stride_n=72), 3), (dict(vc_stride_h=2056), 3), (dict(vc_stride_p=0), 1),
]


@pytest.mark.parametrize("mut,code", ALL)
def test_refusals_before_launch(mut, code):
    assert _fwd(_params(**mut)) == code
    for name in ("fa_cache8_append", "fa_cache8_read"):
        assert _rows(name, _params(**mut)) == code


def test_limits_of_the_attention():
    for mut in (dict(B=1 << 23), dict(T=1 << 23), dict(B=300, width=1 << 23, table_stride=1 << 23),
                dict(H=1 << 13, H_kv=1 << 13, width=1 << 23, table_stride=1 << 23)):
        p = dict(mut)
        for t in "qo":
            p.update({t + "_stride_h": 64 * mut.get("T", 2), t + "_stride_b": 64 * mut.get("T", 2) * mut.get("H", 4)})
        assert _fwd(_params(**p)) == 2


def test_strides_pointers_and_workspace():
    for t in ("q", "o"):
        assert _fwd(_params(**{t + "_stride_n": 68})) == 3 and _fwd(_params(**{t + "_stride_n": 32})) == 1
    for name in ("fa_cache8_append", "fa_cache8_read"):
        for t in ("k", "v"):
            assert _rows(name, _params(**{t + "_stride_n": 68})) == 3
            assert _rows(name, _params(**{t + "_stride_b": 0})) == 1
        for i in range(6):
            assert _rows(name, _params(), {i: None}) == 1 and _rows(name, _params(), {i: (1 << 20) + 2}) == 3
        assert _rows(name, None) == 1
    assert _fwd(None) == 1
    for i in range(7):
        assert _fwd(_params(), {i: None}) == 1 and _fwd(_params(), {i: (1 << 20) + 2}) == 3
    size = _ops._fn("fa_cache8_workspace_size", ctypes.c_void_p, restype=ctypes.c_size_t)
    p = _params()
    need = size(ctypes.addressof(p))
    assert size(None) == 256 and need >= 256 + 2 * 456 * 8 * (64 * 4 + 8)
    assert _fwd(p, ws=need - 1) == 4 and _fwd(p, ws_ptr=None) == 4 and _fwd(p, ws_ptr=(1 << 21) + 8) == 4
    big = _params(B=1000)
    assert size(ctypes.addressof(big)) >= need + 4004


def test_binding_refuses():
    q = torch.zeros(1, 2, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache8_fwd(q, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache8_append(q, q, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache8_read(q, q, None, None, None, None)


def units(L, T, window, sinks, KS):
    """The kernel's units_of: the first keys of the units that a sequence's rows read."""
    if L <= 0:
        return []
    hi = -(-L // KS)
    lo = max(0, L - T - window + 1) // KS if window > 0 else 0
    ns = min(-(-min(sinks, L) // KS), lo)
    return [(i if i < ns else i + lo - ns) * KS for i in range(ns + hi - lo)]


@pytest.mark.parametrize("KS", [32, 64])
def test_units_cover_the_visible_keys_once(KS):
    rng = random.Random(KS)
    for _ in range(400):
        L, T = rng.randint(0, 700), rng.randint(1, 9)
        window, sinks = rng.choice([0, rng.randint(1, 800)]), rng.choice([0, 4, rng.randint(0, 800)])
        got = units(L, T, window, sinks, KS)
        assert got == sorted(set(got)) and all(0 <= k < L for k in got)
        seen = {j for t in range(T) for p in [L - T + t] for j in range(p + 1)
                if window == 0 or j > p - window or j < sinks}
        assert seen <= {j for k in got for j in range(k, k + KS)}
        # no unit that nobody sees, where each row exists
        if L >= T:
            assert all(seen & set(range(k, k + KS)) for k in got)


def test_pieces_of_the_line():
    # the kernel's cut of the line (kItemUnits in front of every row set): each unit has one owner, a row set's pieces
    # are neighbours, and a CTA begins one cut row set at most
    cost = 12
    rng = random.Random(2)
    for _ in range(300):
        segs = [rng.choice([1, 2, rng.randint(1, 300)]) for _ in range(rng.randint(1, 20))]
        X = sum(n + cost for n in segs)
        C = rng.randint(1, min(456, X))
        each, more = divmod(X, C)
        begin = [each * c + min(c, more) for c in range(C + 1)]
        wide = (each + 1) * more
        owner = lambda x: x // (each + 1) if x < wide else more + (x - wide) // each  # noqa: E731
        assert begin[C] == X
        for x in range(X):
            assert begin[owner(x)] <= x < begin[owner(x) + 1]
        at, cut, slots = cost, [], []
        for n in segs:
            c0, c1 = owner(at), owner(at + n - 1)
            if c1 > c0:
                cut.append(c0)
                slots += [2 * c + (1 if at >= begin[c] else 0) for c in range(c0, c1 + 1)]
                assert [2 * c + (1 if c == c0 else 0) for c in range(c0, c1 + 1)] == slots[-(c1 - c0 + 1):]
            # whole, as the one CTA that has the first unit sees it
            assert (c1 == c0) == (at >= begin[c0] and at + n <= begin[c0 + 1])
            at += n + cost
        assert len(set(cut)) == len(cut) and len(set(slots)) == len(slots)


@pytest.mark.parametrize("D", [64, 128])
def test_key_order_and_banks(D):
    def key(m, e):
        return ((m & 2) << 1 | e << 1 | ((m & 1) ^ e)) if D == 64 else (((m >> 1) ^ e) << 2 | (m & 1) << 1 | e)

    assert sorted(key(m, e) for m in range(4) for e in range(2)) == list(range(8))

    def swizzled(row, byte):                 # the copy's pattern: 16-byte pieces by address bits 7 and up
        at = row * D + byte
        return at ^ ((at >> 3) & (0x30 if D == 64 else 0x70))

    def conflict_free(addresses, width):     # one pass of 128 bytes
        banks = [(a // 4 + i) % 32 for a in addresses for i in range(width // 4)]
        return len(set(banks)) == len(banks) == 32

    for h in range(D // 64):                 # K: 16 bytes a lane, 8 lanes a pass
        for p in range(4):
            assert conflict_free([swizzled(key((l // 4) >> 1, (l // 4) & 1), 64 * h + 16 * (l % 4))
                                  for l in range(8 * p, 8 * p + 8)], 16)
    w = D // 8                               # V: 8 or 16 bytes a lane
    for e in range(2):
        for p in range(w // 4):
            lanes = range(p * 128 // w, (p + 1) * 128 // w)
            assert conflict_free([swizzled(key(l % 4, e), w * (l // 4)) for l in lanes], w)


# ---- a cache in plain form ----------------------------------------------------------------------------------------
def grid():
    v = torch.tensor([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127],
                     dtype=torch.float64)
    return v, (v[1:] + v[:-1]) / 2


def nearest(y):
    """The E4M3 value next to y (float64, |y| <= 448), ties to the even code."""
    v, mid = (t.to(y.device) for t in grid())
    a = y.abs()
    n = torch.searchsorted(mid, a.contiguous())
    tie = (n < 126) & (mid[n.clamp(max=125)] == a) & (n % 2 == 1)
    return torch.where(y.isnan(), y, v[(n + tie.long()).clamp(max=126)] * torch.sign(y))


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def exponent(m):
    e = -126
    if m > 0:
        e = math.ceil(math.log2(m / 448)) if m > 1e-300 else -126
        while e > -126 and 448 * 2.0 ** (e - 1) >= m:
            e -= 1
        while 448 * 2.0 ** e < m:
            e += 1
    return max(e, -126)


def plain_append(x, codes, scale, table, lens, page):
    """New rows x [B,Hkv,T,d] into values codes [P,Hkv,page,d] (float64) and scale, in place."""
    B, Hkv, T, _ = x.shape
    for b in range(B):
        L = max(0, min(lens[b], table.shape[1] * page))
        for w in range(table.shape[1]):
            id = int(table[b, w])
            n0, n1 = max(w * page, L - T, 0), min(w * page + page, L)
            if n0 >= n1 or not 0 <= id < codes.shape[0]:
                continue
            for h in range(Hkv):
                rows = x[b, h, n0 - (L - T):n1 - (L - T)].double()
                fin = rows[rows.isfinite()]
                m = float(fin.abs().max()) if fin.numel() else 0.0
                was = float(scale[id, h]) if n0 > w * page else 0.0
                now = max(was, 2.0 ** exponent(m) if m > 0 else 0.0)
                if was > 0 and now > was:
                    old = codes[id, h, :n0 - w * page]
                    codes[id, h, :n0 - w * page] = nearest(old * (was / now))
                y = rows / now if now > 0 else rows * 0
                codes[id, h, n0 - w * page:n1 - w * page] = nearest(y.clamp(-448, 448))
                scale[id, h] = now


def make_cache(B, Hkv, d, page, lens, width, seed=0, spread=1.0, spare=3, nan_behind=True):
    """Random pages in no order; codes as uint8 (rows behind a sequence hold NaN), scales, table (-1 behind)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-max(0, min(n, width * page)) // page) for n in lens]
    P = sum(need) + spare
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    kc, vc = (torch.full((P, Hkv, page, d), 0x7F, device="cuda", dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.full((P, Hkv), math.nan, device="cuda") for _ in range(2))
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
        for w in range(n):
            rows = min(page, max(0, lens[b]) - w * page) if nan_behind else page
            id = int(table[b, w])
            for c, s in ((kc, ks), (vc, vs)):
                x = torch.randn(Hkv, rows, d, generator=g, device="cuda")
                top = x.abs().amax((1, 2), keepdim=True)
                c[id, :, :rows] = (x / top * 400).to(torch.float8_e4m3fn).view(torch.uint8)
                e = torch.round(torch.randn(Hkv, generator=g, device="cuda") * spread)
                s[id] = torch.exp2(e - 7)
    return kc, vc, ks, vs, table.cuda()


def gathered(c, s, table, page, lens):
    """[B,Hkv,M,d] float64 values and codes, hidden rows as zeros, and which rows are there [B, M]."""
    B, W = table.shape
    P, Hkv, _, d = c.shape
    ok = (table >= 0) & (table < P)
    ids = torch.where(ok, table, torch.zeros_like(table)).long()
    v = values(c)[ids].transpose(1, 2).reshape(B, Hkv, W * page, d)
    sc = s.double()[ids].transpose(1, 2).repeat_interleave(page, 2)[..., None]
    j = torch.arange(W * page, device=c.device)
    there = ok.repeat_interleave(page, 1) & (j[None] < lens[:, None])
    hide = ~there[:, None, :, None]
    return (v * sc).masked_fill(hide, 0.0), v.masked_fill(hide, 0.0), sc.squeeze(-1), there


def plain_fwd(q, cache, lens, page, window=0, sinks=0, scale=None):
    kc, vc, ks, vs, table = cache
    B, H, T, d = q.shape
    Hkv = kc.shape[1]
    G = H // Hkv
    scale = d ** -0.5 if scale is None else scale
    lens = lens.to(q.device).long().clamp(0, table.shape[1] * page)
    k, _, _, there = gathered(kc, ks, table, page, lens)
    v, code, vsc, _ = gathered(vc, vs, table, page, lens)
    j, t = torch.arange(k.shape[2], device=q.device), torch.arange(T, device=q.device)
    p = (lens[:, None] - T + t)[:, :, None]
    see = (j <= p) & there[:, None]
    if window:
        see = see & ((j > p - window) | (j < sinks))
    see = see[:, None, None].expand(B, 1, G, T, -1).reshape(B, 1, G * T, -1)
    qq = q.double().reshape(B, Hkv, G * T, d)
    s = qq @ k.transpose(-1, -2) * scale
    smag = (qq.abs() @ k.abs().transpose(-1, -2) * abs(scale)).masked_fill(~see, 0).amax(-1, keepdim=True)
    s = s.masked_fill(~see, -math.inf)
    none = ~see.any(-1, keepdim=True)
    m = s.amax(-1, keepdim=True).masked_fill(none, 0.0)
    w = torch.exp(s - m)
    l = w.sum(-1, keepdim=True)
    w = w / l.masked_fill(none, 1.0)
    o, mag = w @ v, w @ v.abs()
    lse = (m + torch.log(l)).squeeze(-1)
    lv = torch.where(there[:, None] & (vsc > 0), torch.log(vsc.clamp(min=1e-300)), torch.full_like(vsc, -64 * math.log(2)))[:, :, None]
    tmax = (s + lv).masked_fill(~see, -math.inf).amax(-1, keepdim=True).masked_fill(none, 0.0)
    ell = torch.exp(s - tmax).sum(-1, keepdim=True).masked_fill(none, 1.0)
    small = 2.0 ** -25 * (see.double() @ code.abs()) / ell
    r = lambda x: x.reshape(B, H, T, -1)  # noqa: E731
    return r(o), lse.reshape(B, H, T), r(mag), r(smag), r(small)


def check(got, want, dtype):
    u = torch.finfo(DT[dtype]).eps / 2
    o, lse = got
    wo, wl, mag, smag, small = want
    delta = 2.0 ** -19 * (1 + smag)
    err = (o.double() - wo).abs()
    bound = (2.0 ** -11 + 2 * delta + 2.0 ** -20) * mag + u * wo.abs() + small + (2.0 ** -25 if dtype == "f16" else 0)
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())
    fin = torch.isfinite(wl)
    assert torch.equal(fin, torch.isfinite(lse)) and bool((lse[~fin] == -math.inf).all())
    ok = (lse.double() - wl).abs() <= delta.squeeze(-1) + 2.0 ** -20 * (1 + wl.abs())
    assert bool(ok[fin].all())


def run(B, H, Hkv, T, d, page, dtype, lens, width=None, window=0, sinks=0, seed=0, spread=1.0, scale=None):
    width = max(1, -(-max(lens) // page)) if width is None else width
    cache = make_cache(B, Hkv, d, page, lens, width, seed, spread)
    q = torch.randn(B, H, T, d, generator=torch.Generator(device="cuda").manual_seed(seed + 1), device="cuda").to(DT[dtype])
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = fa.cache8_fwd(q, *cache, ln, window=window, sinks=sinks, scale=scale)
    assert fa.check_status(fa.cache8_fwd.last_workspace) == 0
    check(got, plain_fwd(q, cache, ln, page, window, sinks, scale), dtype)
    return q, cache, ln, got


# ---- GPU: rows in and out -------------------------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 3, 16, 130])
def test_append_and_read(dtype, d, page, T):
    B, Hkv, width = 6, 2, -(-400 // page)
    lens = [0, T, max(T - 1, 0), T + page - 1, T + page, 400 - T % 7]
    old = [max(0, n - T) for n in lens]
    kc, vc, ks, vs, table = make_cache(B, Hkv, d, page, lens, width, seed=T, spread=2.0)
    for b, n in enumerate(old):          # what the new tokens will write holds NaN before
        for j in range(n, min(lens[b], width * page)):
            kc[table[b, j // page], :, j % page] = 0x7F
    x = [(torch.randn(B, Hkv, T, d, device="cuda") * torch.exp2(torch.randint(-3, 4, (B, Hkv, T, 1), device="cuda"))).to(DT[dtype])
         for _ in range(2)]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = []
    for xx, c, s in ((x[0], kc, ks), (x[1], vc, vs)):
        cv, sv = values(c).cpu(), s.double().cpu()
        plain_append(xx.cpu(), cv, sv, table.cpu(), lens, page)
        want.append((cv, sv))
    for again in range(2):               # the same tokens once more change nothing
        fa.cache8_append(*x, kc, vc, ks, vs, table, ln)
        for (cv, sv), c, s in zip(want, (kc, vc), (ks, vs)):
            assert torch.equal(values(c).cpu().nan_to_num(nan=9999.0), cv.nan_to_num(nan=9999.0))
            assert torch.equal(s.double().cpu().nan_to_num(nan=9999.0), sv.nan_to_num(nan=9999.0))
    for rows in (None, 1, min(77, width * page), width * page + 33):
        k, v = fa.cache8_read(kc, vc, ks, vs, table, ln, dtype=DT[dtype], rows=rows)
        for got, c, s in ((k, kc, ks), (v, vc, vs)):
            full = gathered(c, s, table, page, ln)[0].to(DT[dtype])
            n = got.shape[2]
            ref = torch.zeros(B, Hkv, n, d, device="cuda", dtype=DT[dtype])
            ref[:, :, :min(n, full.shape[2])] = full[:, :, :n]
            assert torch.equal(got, ref)


@gpu
def test_append_keeps_what_is_not_its_own():
    B, Hkv, d, page, lens = 3, 2, 64, 16, [5, 16, 33]
    kc, vc, ks, vs, table = make_cache(B, Hkv, d, page, lens, 3, seed=3, spare=4)
    keep = [t.clone() for t in (kc, vc, ks, vs)]
    x = torch.randn(B, Hkv, 1, d, device="cuda").bfloat16() * 50
    fa.cache8_append(x, x, kc, vc, ks, vs, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    touched = {int(table[0, 0]), int(table[1, 0]), int(table[2, 2])}
    for t, k in zip((kc, vc, ks, vs), keep):
        for id in range(t.shape[0]):
            if id not in touched:
                assert torch.equal(t[id].nan_to_num(), k[id].nan_to_num())
    for id, n in ((int(table[0, 0]), 5), (int(table[1, 0]), 16), (int(table[2, 2]), 1)):
        assert torch.equal(kc[id, :, n:], keep[0][id, :, n:])


@gpu
def test_append_absent_pages_and_bad_entries():
    Hkv, d, page = 2, 64, 16
    lens = [40, 40, 40]
    kc, vc, ks, vs, table = make_cache(3, Hkv, d, page, lens, 3, seed=4)
    table[0, 1], table[1, 2], table[2, 0] = -1, kc.shape[0], -2 ** 31
    want = [values(c).cpu() for c in (kc, vc)], [s.double().cpu() for s in (ks, vs)]
    x = torch.randn(3, Hkv, 40, d, device="cuda").half()
    for c, s in zip(*want):
        plain_append(x.cpu(), c, s, table.cpu(), lens, page)
    ln = torch.tensor(lens, device="cuda")
    fa.cache8_append(x, x, kc, vc, ks, vs, table, ln)
    for (c, s), cc, ss in zip(zip(*want), (kc, vc), (ks, vs)):
        assert torch.equal(values(cc).cpu().nan_to_num(nan=9999.0), c.nan_to_num(nan=9999.0))
        assert torch.equal(ss.double().cpu().nan_to_num(nan=9999.0), s.nan_to_num(nan=9999.0))
    k, _ = fa.cache8_read(kc, vc, ks, vs, table, ln)
    assert bool((k[0, :, 16:32] == 0).all() and (k[1, :, 32:] == 0).all() and (k[2, :, :16] == 0).all())
    assert bool((k[0, :, :16] != 0).any())
    # the same table in 64 bits, with numbers that int32 does not hold
    wide = table.long()
    wide[0, 1] = 2 ** 32
    assert torch.equal(fa.cache8_read(kc, vc, ks, vs, wide, ln)[0], k)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_special_values(dtype):
    page, d = 16, 64
    kc, vc = (torch.full((2, 1, page, d), 0x7F, device="cuda", dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.full((2, 1), math.nan, device="cuda") for _ in range(2))
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")

    def put(x, n):
        fa.cache8_append(x, x, kc, vc, ks, vs, table, torch.tensor([n], device="cuda"))
        return values(kc)[1, 0], float(ks[1, 0])

    zero = torch.zeros(1, 1, 4, d, device="cuda", dtype=DT[dtype])
    c, s = put(zero, 4)                          # zeros alone: scale 0
    assert s == 0.0 and bool((c[:4] == 0).all())
    x = zero[:, :, :2].clone()
    x[0, 0, 0, 3], x[0, 0, 1, 5] = -2.0 ** -14, 448 * 2.0 ** -18
    c, s = put(x, 6)                             # behind zeros: the new rows' own scale
    assert s == 2.0 ** -18 and bool((c[:4] == 0).all()) and float(c[4, 3]) == -16.0 and float(c[5, 5]) == 448.0
    x = zero[:, :, :1].clone()
    x[0, 0, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, 100.0])
    c, s = put(x, 7)                             # 100 <= 448 / 4; 400 lies between 384 and 416, ties to the even code
    assert s == 0.25 and bool(c[6, 0].isnan()) and c[6, 1:4].tolist() == [448.0, -448.0, 384.0]
    # rounded again, 2^16 times smaller: 448 becomes 3.5 steps of 2^-9, 16 an eighth of one
    assert float(c[5, 5]) == 4 * 2.0 ** -9 and float(c[4, 3]) == 0.0
    big = torch.full((1, 1, 1, d), torch.finfo(DT[dtype]).max, device="cuda", dtype=DT[dtype])
    c, s = put(big, 8)
    assert math.isfinite(s) and bool((c[7] * s >= 0.93 * float(big[0, 0, 0, 0])).all())
    assert all(float(t) == s for t in (ks[1, 0], vs[1, 0])) and bool(ks[0].isnan().all())


@gpu
def test_layouts_and_streams_of_rows():
    B, Hkv, d, page, T = 3, 4, 64, 32, 5
    lens = [5, 40, 90]
    kc, vc, ks, vs, table = make_cache(B, Hkv, d, page, lens, 3, seed=5)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = torch.randn(B, T, 2 * Hkv, d, device="cuda").bfloat16()          # a fused projection
    k, v = x[:, :, :Hkv].transpose(1, 2), x[:, :, Hkv:].transpose(1, 2)
    a = [t.clone() for t in (kc, vc, ks, vs)]
    fa.cache8_append(k.contiguous(), v.contiguous(), *a, table, ln)
    # [pages, page, Hkv, d] memory, K and V interleaved in one tensor, a table with longer rows
    P = kc.shape[0]
    both = torch.zeros(P, page, 2, Hkv, d, device="cuda", dtype=torch.uint8)
    kc2, vc2 = both[:, :, 0].permute(0, 2, 1, 3), both[:, :, 1].permute(0, 2, 1, 3)
    kc2.copy_(kc)
    vc2.copy_(vc)
    b = [kc2, vc2, ks.clone(), vs.clone()]
    t2 = torch.full((B, 9), 7, dtype=torch.int32, device="cuda")[:, :3]
    t2.copy_(table)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    fa.cache8_append(k, v, *b, t2, ln.long(), stream=s)
    r2 = fa.cache8_read(*b, t2, ln, stream=s)
    s.synchronize()
    for m, n in zip(a, b):
        assert torch.equal(m.float().nan_to_num(), n.float().nan_to_num())
    r1 = fa.cache8_read(*a, table, ln)
    assert all(torch.equal(m, n) for m, n in zip(r1, r2))
    out = [torch.empty(B, 96, Hkv, d, device="cuda", dtype=torch.bfloat16).transpose(1, 2) for _ in range(2)]
    fa.cache8_read(*a, table, ln, out=out)
    assert all(torch.equal(m, n) for m, n in zip(r1, out))
    # and the attention over both layouts
    q = torch.randn(B, 8, 1, d, device="cuda").bfloat16()
    f1, f2 = fa.cache8_fwd(q, *a, table, ln), fa.cache8_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), *b, t2, ln)
    assert all(torch.equal(m, n) for m, n in zip(f1, f2))
    f8 = fa.cache8_fwd(q, a[0].view(torch.float8_e4m3fn), a[1].view(torch.float8_e4m3fn), a[2], a[3], table, ln)
    assert all(torch.equal(m, n) for m, n in zip(f1, f8))


# ---- GPU: attention ------------------------------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_lengths(dtype, d, page):
    run(8, 4, 2, 1, d, page, dtype, [0, 1, 15, 16, 17, 63, 64, 65], seed=page)
    run(8, 2, 2, 1, d, page, dtype, [127, 128, 129, 200, 31, 33, 255, 511], seed=page)
    run(1, 2, 1, 1, d, page, dtype, [1], seed=page)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,T", [(1, 1, 1, 1), (1, 16, 16, 1), (2, 16, 2, 1), (17, 2, 1, 1), (5, 8, 1, 2),
                                       (3, 12, 12, 5), (2, 8, 2, 9), (1, 32, 1, 1), (4, 6, 2, 33), (1, 2, 1, 100),
                                       (2, 16, 1, 3)])
def test_rows_and_groups(dtype, d, B, H, Hkv, T):
    lens = [(137 * b + T) % 300 for b in range(B)]
    run(B, H, Hkv, T, d, 32, dtype, lens, seed=B * T)
    run(B, H, Hkv, T, d, 16, dtype, lens, window=40, sinks=3, seed=B * T)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (63, 64), (65, 65), (100, 0), (500, 4), (2, 499), (3, 600),
                                          (10000, 5), (2 ** 31 - 1, 2 ** 31 - 1), (0, 4)])
def test_window_and_sinks(d, window, sinks):
    lens = [0, 1, 64, 65, 130, 500, 333]
    run(7, 4, 2, 1, d, 64, "f16", lens, window=window, sinks=sinks, seed=1)
    run(7, 4, 4, 4, d, 16, "bf16", lens, window=window, sinks=sinks, seed=2)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_long_rows_are_cut_and_joined(d):
    # one sequence over every CTA, several over a few each, many over less than one
    for B, H, Hkv, T, lens in ((1, 1, 1, 1, [30000]), (1, 8, 1, 1, [65000]), (3, 8, 2, 2, [20000, 1, 7777]),
                               (1, 40, 1, 1, [9000]), (40, 4, 4, 1, [137 * b % 3000 for b in range(40)])):
        x = run(B, H, Hkv, T, d, 128, "bf16", lens, seed=B)
        q, cache, ln, got = x
        again = fa.cache8_fwd(q, *cache, ln)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


@gpu
@pytest.mark.parametrize("B", [191, 192, 193, 385, 1500])
def test_many_sequences(B):
    rng = random.Random(B)
    lens = [rng.choice([0, 0, 1, rng.randint(0, 150)]) for _ in range(B)]
    run(B, 2, 1, 1, 64, 32, "bf16", lens, width=5, seed=B)
    run(B, 2, 1, 2, 128, 16, "f16", lens, width=10, window=30, sinks=2, seed=B)


@gpu
def test_a_batch_without_keys():
    q, cache, ln, (o, lse) = run(3, 4, 2, 2, 64, 16, "bf16", [0, 0, 0], width=2)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    run(2, 4, 2, 6, 64, 16, "bf16", [3, 0], width=2)          # fewer rows than tokens
    o, lse = fa.cache8_fwd(q, *cache, torch.tensor([-5, -2 ** 31, 0], device="cuda"))
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


@gpu
def test_lengths_past_the_table():
    q, cache, _, _ = run(2, 4, 2, 1, 64, 16, "bf16", [48, 48])
    full = fa.cache8_fwd(q, *cache, torch.tensor([48, 48], device="cuda"))
    for n in (49, 2 ** 31 - 1, 2 ** 40):
        got = fa.cache8_fwd(q, *cache, torch.tensor([48, n], device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(full, got))


@gpu
@pytest.mark.parametrize("d,page", [(64, 16), (64, 32), (64, 128), (128, 16), (128, 64)])
def test_absent_pages(d, page):
    lens = [300, 300, 300, 300]
    cache = make_cache(4, 2, d, page, lens, -(-300 // page), seed=6)
    table, P = cache[4], cache[0].shape[0]
    table[0, 0], table[1, 1], table[2, -1], table[3, :] = -1, P, 2 ** 31 - 1, -7
    q = torch.randn(4, 4, 2, d, device="cuda").bfloat16()
    ln = torch.tensor(lens, device="cuda")
    for w, s in ((0, 0), (150, 20)):
        got = fa.cache8_fwd(q, *cache, ln, window=w, sinks=s)
        assert fa.check_status(fa.cache8_fwd.last_workspace) == 0
        check(got, plain_fwd(q, cache, ln, page, w, s), "bf16")
    assert bool((got[0][3] == 0).all()) and bool((got[1][3] == -math.inf).all())


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_scales_and_ranges(d):
    # scales that differ by 2^24 between pages, zero pages, tiny and huge q, scores far from zero
    run(3, 4, 2, 1, d, 16, "f16", [200, 100, 37], spread=6.0, seed=7)
    for f in (2.0 ** -60, 2.0 ** 20):
        cache = make_cache(2, 2, d, 16, [100, 50], 7, seed=8)
        q = (torch.randn(2, 4, 1, d, device="cuda") * f).bfloat16()
        cache[2].mul_(2.0 ** -20 if f > 1 else 2.0 ** 30)
        cache[3].mul_(2.0 ** 40 if f > 1 else 2.0 ** -70)
        ln = torch.tensor([100, 50], device="cuda")
        check(fa.cache8_fwd(q, *cache, ln), plain_fwd(q, cache, ln, 16), "bf16")
    cache = make_cache(1, 1, d, 16, [64], 4, seed=9)
    for i, c in ((2, 0), (3, 1)):
        id = int(cache[4][0, c])
        cache[i][id] = 0.0
        cache[i - 2][id] = 0
    q = torch.randn(1, 2, 1, d, device="cuda").half()
    ln = torch.tensor([64], device="cuda")
    check(fa.cache8_fwd(q, *cache, ln), plain_fwd(q, cache, ln, 16), "f16")
    q.zero_()
    check(fa.cache8_fwd(q, *cache, ln), plain_fwd(q, cache, ln, 16), "f16")


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("vs", [2.0 ** -126, 2.0 ** -20, 2.0 ** 90])
def test_zero_pages_and_the_ends_of_the_value_scales(d, vs):
    # 40 rows of 300 keys, in one CTA and cut: a page of zeros in V whose keys score highest, the others' values small
    # enough to overflow a plain sum of weights over scales (2^-126) or large
    for B, Hkv in ((1, 1), (20, 2)):
        lens = [300] * B
        cache = make_cache(B, Hkv, d, 16, lens, 19, seed=11)
        kc, vc, ks, v_scale, table = cache
        v_scale.fill_(vs)
        ks.fill_(2.0 ** -8)
        if vs < 1:
            zero = table[:, 7].long()
            vc[zero] = 0
            v_scale[zero] = 0.0
            ks[zero] = 2.0 ** -6
        q = torch.randn(B, 2 * Hkv, 1, d, generator=torch.Generator(device="cuda").manual_seed(12), device="cuda").bfloat16()
        ln = torch.tensor(lens, device="cuda")
        got = fa.cache8_fwd(q, *cache, ln)
        check(got, plain_fwd(q, cache, ln, 16), "bf16")


@gpu
def test_a_row_of_nan_stays_alone():
    q, cache, ln, want = run(2, 8, 2, 2, 64, 16, "bf16", [70, 200], seed=10)
    bad = q.clone()
    bad[1, 3, 0, 5] = math.nan
    o, lse = fa.cache8_fwd(bad, *cache, ln)
    assert bool(o[1, 3, 0].isnan().all()) and bool(lse[1, 3, 0].isnan())
    o[1, 3, 0], lse[1, 3, 0] = want[0][1, 3, 0], want[1][1, 3, 0]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@gpu
def test_pages_shared_by_sequences():
    # the same pages under two sequences, and twice in one
    cache = make_cache(2, 2, 64, 32, [96, 0], 4, seed=11)
    table = cache[4]
    table[1] = table[0]
    table[1, 3] = table[0, 1]
    ln = torch.tensor([96, 128], device="cuda")
    q = torch.randn(2, 4, 1, 64, device="cuda").bfloat16()
    check(fa.cache8_fwd(q, *cache, ln), plain_fwd(q, cache, ln, 32), "bf16")


@gpu
def test_graphs_streams_and_two_at_once():
    lens = [700, 33, 0, 1500]
    cache = make_cache(4, 2, 64, 32, [1600] * 4, 50, seed=12, nan_behind=False)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(4, 8, 1, 64, device="cuda").bfloat16()
    kw = dict(window=300, sinks=4)
    fa.cache8_fwd(q, *cache, ln, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fa.cache8_fwd(q, *cache, ln, **kw)
    for n in ([700, 33, 0, 1500], [1, 1600, 64, 0], [0, 0, 0, 0]):
        ln.copy_(torch.tensor(n))
        q.copy_(torch.randn(4, 8, 1, 64, device="cuda"))
        g.replay()
        check(out, plain_fwd(q, cache, ln, 32, **kw), "bf16")
    ln.copy_(torch.tensor(lens))
    want = fa.cache8_fwd(q, *cache, ln, **kw)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [fa.cache8_fwd(q, *cache, ln, **kw, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


@gpu
def test_a_cache_past_32_bits():
    # page ids whose codes lie past 2^32 bytes
    P, Hkv, page, d = 2 ** 32 // (128 * 128) + 64, 1, 128, 128
    kc, vc = (torch.empty((P, Hkv, page, d), device="cuda", dtype=torch.uint8) for _ in range(2))
    small = make_cache(1, 1, d, page, [300], 3, seed=13)
    ks, vs = (torch.empty((P, Hkv), device="cuda") for _ in range(2))
    ids = [P - 1, 5, P - 30]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    for i, id in enumerate(ids):
        src = int(small[4][0, i])
        kc[id], vc[id], ks[id], vs[id] = (t[src] for t in small[:4])
    q = torch.randn(1, 4, 1, d, device="cuda").bfloat16()
    ln = torch.tensor([300], device="cuda")
    got, want = fa.cache8_fwd(q, kc, vc, ks, vs, table, ln), fa.cache8_fwd(q, *small, ln)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = torch.randn(1, 1, 45, d, device="cuda").half()
    fa.cache8_append(x, x, kc, vc, ks, vs, table, ln)
    fa.cache8_append(x, x, *small, ln)
    a, b = fa.cache8_read(kc, vc, ks, vs, table, ln, rows=300), fa.cache8_read(*small, ln, rows=300)
    assert all(torch.equal(m, n) for m, n in zip(a, b))


@gpu
def test_refusals_of_the_binding():
    kc, vc, ks, vs, table = make_cache(2, 2, 64, 16, [20, 20], 2)
    ln = torch.tensor([20, 20], device="cuda")
    q = torch.randn(2, 4, 1, 64, device="cuda").bfloat16()
    k = torch.randn(2, 2, 1, 64, device="cuda").bfloat16()
    good = [kc, vc, ks, vs, table, ln]
    for i, bad in ((0, kc.float()), (0, kc[:, :1]), (1, vc.cpu()), (2, ks.double()), (2, ks[:1]), (3, vs.t()), (4, table[:1]),
                   (4, table.float()), (5, ln[:1]), (5, ln.float()), (5, None), (0, kc.transpose(2, 3))):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            fa.cache8_fwd(q, *args)
        with pytest.raises(ValueError):
            fa.cache8_append(k, k, *args)
        with pytest.raises(ValueError):
            fa.cache8_read(*args)
    for bad in (q[:, :3], q[..., :32].contiguous()):
        with pytest.raises(ValueError):
            fa.cache8_fwd(bad, *good)
    with pytest.raises(ValueError):
        fa.cache8_append(q, q, *good)
    with pytest.raises(ValueError):
        fa.cache8_read(*good, dtype=torch.float32)
    with pytest.raises(ValueError):
        fa.cache8_read(*good, rows=0)
    for kw in (dict(window=-1), dict(sinks=-1)):
        with pytest.raises(fa.FAError):
            fa.cache8_fwd(q, *good, **kw)
    with pytest.raises(fa.FAError):
        fa.cache8_fwd(q.float(), *good)


@gpu
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("T", [1, 5, 100])
def test_new_tokens_past_the_table_are_dropped(d, page, T):
    # as if the table went on with absent pages; the rows that are there keep their places and their codes
    width, cap = 4, 4 * page
    lens = [cap + 1, cap + T, cap + 3 * T, cap, 2 ** 31 - 1, cap - 1 + T // 2]
    B = len(lens)
    kc, vc, ks, vs, table = make_cache(B, 2, d, page, [cap] * B, width, seed=T)
    more = torch.cat([table, torch.full((B, -(-3 * T // page) + 1), -1, dtype=torch.int32, device="cuda")], 1)
    x = torch.randn(B, 2, T, d, device="cuda").bfloat16() * 50
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    keep = [t.clone() for t in (kc, vc, ks, vs)]
    cv, sv = values(kc).cpu(), ks.double().cpu()
    for b, n in enumerate(lens):             # what fits, at its own place
        if cap > n - T:
            fits = x[b:b + 1, :, :cap - (n - T)] if n > cap else x[b:b + 1]
            plain_append(fits.cpu(), cv, sv, table[b:b + 1].cpu(), [min(n, cap)], page)
    for tab in (more, table):
        a = [t.clone() for t in keep]
        fa.cache8_append(x, x, *a, tab, ln)
        assert torch.equal(values(a[0]).cpu().nan_to_num(nan=9999.0), cv.nan_to_num(nan=9999.0))
        assert torch.equal(a[2].double().cpu().nan_to_num(nan=9999.0), sv.nan_to_num(nan=9999.0))
    for b in (2, 4):                         # nothing of theirs fits, and nothing is written
        ids = table[b].long()
        assert all(torch.equal(m[ids], n[ids]) for m, n in zip(a, keep))
    k, _ = fa.cache8_read(*a, table, ln, rows=cap + 7)
    assert bool((k[:, :, cap:] == 0).all()) and bool((k[0, :, :cap] != 0).any())


@gpu
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("T", [1, 5, 70])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (40, 3), (300, 20), (1, 0), (2 ** 31 - 1, 5)])
def test_queries_past_the_table_keep_their_positions(d, page, T, window, sinks):
    # as if the table went on with absent pages
    width, cap = 4, 4 * page
    lens = [cap + 1, cap + 39, cap + 40, cap + 300, cap, 30]
    B = len(lens)
    *cache, table = make_cache(B, 2, d, page, [cap] * B, width, seed=T)
    more = torch.cat([table, torch.full((B, -(-300 // page)), -1, dtype=torch.int32, device="cuda")], 1)
    q = torch.randn(B, 4, T, d, device="cuda").half()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks)
    want = plain_fwd(q, (*cache, more), ln, page, window, sinks)
    for tab in (more, table):
        check(fa.cache8_fwd(q, *cache, tab, ln, **kw), want, "f16")
        assert fa.check_status(fa.cache8_fwd.last_workspace) == 0
    # the last length of int32: everything there is without a window, the first keys alone with one
    ln = torch.full((B,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    here = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    got = fa.cache8_fwd(q, *cache, table, ln, **kw)
    if window in (0, 2 ** 31 - 1):
        check([t[:, :, T - 1:] for t in got], plain_fwd(q[:, :, T - 1:], (*cache, table), here, page), "f16")
    elif sinks == 0:
        assert bool((got[0] == 0).all()) and bool((got[1] == -math.inf).all())
    else:
        one = torch.full((B,), sinks, dtype=torch.int32, device="cuda")
        check([t[:, :, :1] for t in got], plain_fwd(q[:, :, :1], (*cache, table), one, page), "f16")


@pytest.mark.parametrize("T", [2 ** 30 + 1, 2 ** 31 - 127, 2 ** 31 - 1])
def test_rows_near_the_end_of_int32_are_refused(T):
    # the pages that T rows touch are counted in 32 bits
    for name in ("fa_cache8_append", "fa_cache8_read"):
        assert _rows(name, _params(B=1, H=1, H_kv=1, T=T)) == 2


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("vs", [1.0, 2.0 ** 30, 2.0 ** 70, 2.0 ** -40, 2.0 ** -60])
def test_logsumexp_near_zero(d, vs):
    # 100,000 rows of one to three keys with scores near zero: the logsumexp, a sum of numbers of the size of log2(V scale)
    # that cancel, keeps its absolute precision
    B, H, T = 200, 64, 8
    lens = [1 + b % 3 for b in range(B)]
    cache = make_cache(B, 1, d, 16, lens, 1, seed=51, spread=3.0)
    cache[2].fill_(2.0 ** -13)
    cache[3].mul_(vs)
    q = torch.randn(B, H, T, d, generator=torch.Generator(device="cuda").manual_seed(52), device="cuda").bfloat16()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    check(fa.cache8_fwd(q, *cache, ln), plain_fwd(q, cache, ln, 16), "bf16")
