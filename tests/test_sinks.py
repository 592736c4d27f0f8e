"""Attention with a sliding window and first keys that stay visible (fa_fwd_sinks, fa_bwd_sinks).

CPU: refusals, workspace, the tile schedules' coverage.  GPU: every dtype and head dimension against a 64-bit form.

Tolerances, u = eps / 2 of the dtype.  16 bit: weights rounded once and normalised by their rounded sum (2u), one
rounding of O: |error| <= 2u sum P |v| + u |O| + 2^-20; with dropout the weights' rounding no longer cancels against
the sum (3u).  lse 2^-18 (1 + |lse|).  Gradients, relative in the 2-norm: P and dS are rounded once each, O (in D) and
the result once: 4u.  float32: 1e-5 throughout, the bound of the library's float32 path (a few hundred additions of
2^-24, in the row sums and over the keys).
"""
import ctypes
import math
import random

import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from tests.test_abi import _params

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
gpu = pytest.mark.gpu
T = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load()


# ---- CPU -------------------------------------------------------------------------------------------------------
FAKE, WS = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)


def _both(p, sinks, ws=1 << 40):
    lib = fa.load()
    r = ctypes.byref(p)
    return (lib.fa_fwd_sinks(r, sinks, FAKE, FAKE, FAKE, FAKE, FAKE, WS, ws, None),
            lib.fa_bwd_sinks(r, sinks, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, WS, ws, None))


@pytest.mark.parametrize("mut,sinks,code", [
    (dict(causal=1, window=50), -1, 1), (dict(window=50), 4, 2), (dict(window=-1, causal=1), 4, 1), (dict(N=0), 4, 1),
    (dict(d=96, causal=1, window=50), 4, 2), (dict(causal=1, window=50, stride_n=68), 4, 3),
    (dict(causal=1, window=50, dropout_p=1.0), 4, 1), (dict(causal=1, window=50, H_kv=2), 4, 1),
])
def test_refusals_before_launch(mut, sinks, code):
    assert _both(_params(**mut), sinks) == (code, code)


def test_workspaces():
    lib = fa.load()
    size = lambda p, s: lib.fa_bwd_sinks_workspace_size(ctypes.byref(p), s)  # noqa: E731
    n = 5000
    p = _params(causal=1, window=300, N=n, stride_h=n * 64, stride_b=3 * n * 64)
    plain = lib.fa_bwd_workspace_size(ctypes.byref(p))
    assert size(p, 0) == plain and size(p, -3) == plain and size(p, n) == plain
    # 40 query tiles of a first key tile: items of 16 of them for each of the 6 heads; few first keys: their rows
    assert size(p, 9) >= plain + 6 * 3 * T * 2 * 64 * 4
    assert plain + 6 * 2 * 8 * 2 * 64 * 4 <= size(p, 4) <= plain + (6 + 456) * 8 * 2 * 64 * 4 + 512
    assert _both(p, 4, ws=plain)[1] == 4
    assert size(_params(causal=1, window=0), 4) == lib.fa_bwd_workspace_size(ctypes.byref(_params()))
    # however many the first keys and heads, the pieces stay within about 1,216
    big = _params(causal=1, window=1000, N=65536, stride_h=65536 * 64, stride_b=3 * 65536 * 64)
    base = lib.fa_bwd_workspace_size(ctypes.byref(big))
    for s in (1, 129, 5000, 60000):
        assert size(big, s) <= base + (2 * 608 + 6) * T * 2 * 64 * 4


def forward_tiles(qt, N, Lk, w, s, rows=None):
    """The kernels' schedule of one query tile: first keys' tiles, then the window's."""
    lim = min(-(-Lk // T), qt + 1)
    lo = max(0, qt * T - w + 1) // T
    head = min(-(-s // T), min(lo, lim))
    if rows is None:
        return list(range(head)) + list(range(lo, max(lo, lim)))
    return [t for t in rows if t < head] + [t for t in rows if lo <= t < lim]


def test_schedules_cover_the_visible_pairs_once():
    rng = random.Random(5)
    for _ in range(300):
        N = rng.randint(2, 1500)
        w, s = rng.randint(1, N - 1), rng.randint(1, N - 1)
        Lk = rng.choice([N, rng.randint(0, N)])
        nq, group = -(-N // T), rng.choice([1, 2, 5])
        tiles = -(-s // T)
        steps = nq * group
        chunks = min(-(-steps // rng.choice([2, 16, 40])), max(1, 608 // (rng.choice([1, 3, 100]) * tiles)))
        per = -(-steps // chunks)
        chunks = -(-steps // per)
        pairs = {}
        for jt in range(nq):                    # the backward pass's items
            first = jt < tiles
            qlast = nq - 1 if first else min(nq - 1, (jt * T + T - 1 + w - 1) // T)
            n = max(0, qlast - jt + 1) if jt * T < Lk else 0
            for c in range(chunks if first else 1):
                t0 = c * per if first else 0
                for t in range(t0, min(n * group, t0 + per) if first else n * group):
                    key = (jt, jt + t % n, t // n)
                    pairs[key] = pairs.get(key, 0) + 1
        assert all(v == 1 for v in pairs.values())
        for qt in range(nq):
            got = forward_tiles(qt, N, Lk, w, s)
            assert len(set(got)) == len(got) and got == sorted(got)
            rows = range(qt * T, min(N, qt * T + T))
            seen = set()
            for i in (rows[0], rows[-1], rng.choice(rows)):
                for j in range(min(i + 1, Lk)):
                    if j > i - w or j < s:
                        seen.add(j // T)
            assert seen <= set(got)
            for jt in seen:
                assert all((jt, qt, g) in pairs for g in range(group))


# ---- the 64-bit form -------------------------------------------------------------------------------------------
def plain(q, k, v, do, w, s, lens=None, keep=None, p_drop=0.0, blocks=None, scale=None):
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    scale = d ** -0.5 if scale is None else scale
    i = torch.arange(N, device=q.device)
    see = i[None] <= i[:, None]
    if w:
        see = see & ((i[None] > i[:, None] - w) | (i[None] < s))
    if blocks is not None:
        see = see & blocks.bool().repeat_interleave(T, 0).repeat_interleave(T, 1)[:N, :N]
    see = see[None, None, None]
    if lens is not None:
        see = see & (i < lens.to(q.device)[:, None])[:, None, None, None, :]
    qq, dd = (t.double().view(B, Hkv, G, N, d) for t in (q, do))
    kk, vv = (t.double().view(B, Hkv, 1, N, d) for t in (k, v))
    x = (qq @ kk.transpose(-1, -2) * scale)
    none = ~see.any(-1, keepdim=True)
    x = x.masked_fill(~(see | none), -math.inf)
    P = torch.softmax(x, -1) * ~none
    lse = torch.logsumexp(x, -1).masked_fill(none.squeeze(-1).expand(x.shape[:-1]), -math.inf)
    Z = 1.0 if keep is None else keep.view(B, Hkv, G, N, N).double() / (1 - p_drop)
    Pt = P * Z
    o, mag = Pt @ vv, Pt @ vv.abs()
    dP = (dd @ vv.transpose(-1, -2)) * Z
    dS = P * (dP - (P * dP).sum(-1, keepdim=True)) * scale
    r = lambda t: t.reshape(B, H, N, -1)  # noqa: E731
    return (r(o), lse.reshape(B, H, N), r(mag), r(dS @ kk), (dS.transpose(-1, -2) @ qq).sum(2),
            (Pt.transpose(-1, -2) @ dd).sum(2))


def test_the_form_against_differences():
    # central differences of sum O dO with steps of 1e-6: rounding 2^-53 x 100 / 1e-6, the step's square below it
    g = torch.Generator().manual_seed(1)
    r = lambda h: torch.randn(2, h, 9, 8, generator=g, dtype=torch.float64)  # noqa: E731
    q, do = r(4), r(4)
    k, v = r(2), r(2)
    lens = torch.tensor([9, 6])
    keep = torch.rand(2, 4, 9, 9, generator=g) > 0.3
    for kw in (dict(lens=lens), dict(keep=keep, p_drop=0.3), dict(scale=0.7)):
        grads = plain(q, k, v, do, 3, 2, **kw)[3:]
        for n, t in enumerate((q, k, v)):
            u = torch.randn(t.shape, generator=g, dtype=torch.float64)
            o = []
            for e in (1e-6, -1e-6):
                x = [q, k, v]
                x[n] = t + e * u
                o.append((plain(*x, do, 3, 2, **kw)[0] * do).sum())
            assert abs(float((o[0] - o[1]) / 2e-6 - (grads[n] * u).sum())) < 1e-7


def rel(a, b):
    n = float(b.norm())
    return float((a.double() - b).norm()) / n if n else float(a.double().norm())


def check(got, want, dtype, drop=False):
    o, lse, dq, dk, dv = got
    wo, wl, mag, *wg = want
    u = torch.finfo(DT[dtype]).eps / 2
    err = (o.double() - wo).abs()
    bound = 1e-5 * (1 + mag) if dtype == "f32" else (3 if drop else 2) * u * mag + u * wo.abs() + 2.0 ** -20
    assert bool((err <= bound).all()), float((err / bound).max())
    fin = torch.isfinite(wl)
    assert torch.equal(fin, torch.isfinite(lse)) and bool((lse[~fin] == -math.inf).all())
    assert bool(((lse.double() - wl)[fin].abs() <= 2.0 ** -18 * (1 + wl[fin].abs())).all())
    for g, x, n in zip((dq, dk, dv), wg, ("dq", "dk", "dv")):
        assert rel(g, x) <= (1e-5 if dtype == "f32" else 4 * u), (n, rel(g, x))
        if n != "dq":
            assert bool((g[(wg[2] == 0).all(-1)] == 0).all())   # keys that nobody sees


def make(B, H, Hkv, N, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(B, h, N, d, generator=g, device="cuda").to(DT[dtype]) for h in (H, Hkv, Hkv, H)]


def run(x, w, s, lens=None, **kw):
    q, k, v, do = x
    mask = dict(causal=True, window=w, sinks=s, seqlens_k=lens, **kw)
    o, lse = fa.fwd(q, k, v, **mask)
    assert fa.check_status(fa.fwd.last_workspace) == 0
    size = fa.bwd(q, k, v, o, do, lse, **mask)[0].numel() and fa.bwd.last_workspace.numel()
    ws = torch.full((size,), 255, device="cuda", dtype=torch.uint8)      # a workspace full of NaN
    grads = fa.bwd(q, k, v, o, do, lse, workspace=ws, **mask)
    assert fa.check_status(ws) == 0
    return (o, lse) + tuple(grads)


KINDS = [("bf16", 64), ("f16", 64), ("f32", 64), ("bf16", 128), ("f16", 128)]


@gpu
@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("N,w,s", [(2, 1, 1), (100, 10, 3), (128, 64, 4), (129, 128, 1), (300, 1, 1), (300, 64, 4),
                                   (300, 200, 130), (513, 129, 128), (700, 100, 129), (700, 2, 300), (640, 128, 256),
                                   (1000, 999, 1), (1000, 300, 999), (1500, 17, 1),
                                   (1500, 40, 8), (1500, 40, 9), (2050, 129, 2), (135, 130, 4)])
def test_lengths_windows_and_first_keys(dtype, d, N, w, s):
    x = make(2, 3, 3, N, d, dtype, N + w + s)
    check(run(x, w, s), plain(*x, w, s), dtype)


@gpu
@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("H,Hkv", [(4, 1), (6, 2), (8, 8)])
def test_grouped_heads_and_padding(dtype, d, H, Hkv):
    x = make(4, H, Hkv, 777, d, dtype, H)
    for w, s in ((150, 4), (90, 200)):
        for lens in ([777, 0, 1, 300], [5, 130, 776, 128]):
            ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
            check(run(x, w, s, ln), plain(*x, w, s, ln), dtype)


@gpu
@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("B,H,Hkv,N", [(1, 4, 2, 5000), (8, 16, 16, 1100)])
def test_long_rows_are_cut(dtype, d, B, H, Hkv, N):
    # 40 query tiles and more at the first key tile: several items, in float32 parts; and many heads, an item each
    x = make(B, H, Hkv, N, d, dtype, 7)
    lib = fa.load()
    p = fa.make_params(x[0], k=x[1], causal=True, window=200)
    parts = lib.fa_bwd_sinks_workspace_size(ctypes.byref(p), 9) > lib.fa_bwd_workspace_size(ctypes.byref(p))
    assert parts == (B == 1)
    for w, s in ((200, 4), (513, 140), (300, 8), (300, 9)):
        got = run(x, w, s)
        check(got, plain(*x, w, s), dtype)
        again = run(x, w, s)
        for i in (0, 1, 3, 4):                  # dQ is added up in the order in which key tiles finish
            assert torch.equal(got[i], again[i])


@gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128), ("f32", 64)])
def test_dropout(dtype, d):
    B, H, N, p = 1, 2, 400, 0.2
    x = make(B, H, 1, N, d, dtype, 9)
    keep = torch.stack([fa.dropout_mask(B, H, N, 0, h, 0, N, dropout_p=p, seed=11, offset=3) for h in range(H)])
    p16 = round(p * 65536) / 65536              # the mask's own threshold; the scale is 1 / (1 - p)
    assert abs(p16 - p) < 1e-5
    kw = dict(dropout_p=p, seed=11, offset=3)
    for w, s in ((100, 5), (30, 150)):
        check(run(x, w, s, **kw), plain(*x, w, s, keep=keep[None], p_drop=p), dtype, drop=True)
    # long enough for several items of the first key tile, and for several CTAs of few first keys
    N = 2500
    x = make(1, 1, 1, N, d, dtype, 10)
    keep = fa.dropout_mask(1, 1, N, 0, 0, 0, N, dropout_p=p, seed=11, offset=3)
    for s in (5, 20):
        check(run(x, 100, s, **kw), plain(*x, 100, s, keep=keep[None, None], p_drop=p), dtype, drop=True)


@gpu
@pytest.mark.parametrize("dtype,d", KINDS)
def test_block_masks(dtype, d):
    N = 1100
    nb = -(-N // T)
    g = torch.Generator().manual_seed(3)
    x = make(1, 2, 2, N, d, dtype, 11)
    for keep_first in (True, False):
        blocks = (torch.rand(nb, nb, generator=g) < 0.5) | torch.eye(nb, dtype=torch.bool)
        blocks[:, 0] = keep_first
        blocks[0, 0] = True
        b = blocks.to(torch.uint8).cuda()
        for w, s in ((300, 4), (140, 300)):
            check(run(x, w, s, block_mask=b), plain(*x, w, s, blocks=b), dtype)


@gpu
@pytest.mark.parametrize("dtype,d", KINDS)
def test_the_same_call_in_other_words(dtype, d):
    x = make(2, 2, 2, 333, d, dtype, 12)
    q, k, v, do = x

    def call(**kw):
        o, lse = fa.fwd(q, k, v, causal=True, **kw)
        return (o, lse) + tuple(fa.bwd(q, k, v, o, do, lse, causal=True, **kw))

    same = lambda a, b: all(torch.equal(m, n) for i, (m, n) in enumerate(zip(a, b)) if i != 2)  # noqa: E731
    causal = call()
    assert same(causal, call(window=333, sinks=4)) and same(causal, call(window=5, sinks=333))
    assert same(causal, call(window=0, sinks=7)) and same(causal, call(window=2 ** 31 - 1, sinks=2 ** 31 - 1))
    assert same(call(window=50), call(window=50, sinks=0))
    # first keys that the window reaches anyway
    a, b = call(window=332, sinks=1), plain(*x, 0, 0)
    check(a, b, dtype)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("place", [0, 3])
def test_dq_in_the_place_of_q_or_do(dtype, place):
    x = make(1, 3, 3, 1000, 64, dtype, 15)
    for s in (0, 3, 20):
        q, k, v, do = (t.clone() for t in x)
        kw = dict(causal=True, window=150, sinks=s)
        o, lse = fa.fwd(q, k, v, **kw)
        want = fa.bwd(q, k, v, o, do, lse, **kw)
        got = fa.bwd(q, k, v, o, do, lse, out=((q, do)[place == 3], torch.empty_like(k), torch.empty_like(v)), **kw)
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        assert rel(got[0], want[0].double()) <= (1e-6 if dtype == "f32" else torch.finfo(torch.bfloat16).eps / 2)


@gpu
def test_both_forward_kernels_agree():
    x = make(1, 3, 3, 1300, 64, "bf16", 13)
    for w, s in ((200, 4), (100, 300)):
        a, b = (fa.fwd(*x[:3], causal=True, window=w, sinks=s, fwd_kernel=n, return_o_f32=True) for n in (1, 2))
        assert all(torch.equal(m, n) for m, n in zip(a, b))


@gpu
@pytest.mark.parametrize("dtype,d", KINDS)
def test_layouts(dtype, d):
    x = make(2, 4, 2, 260, d, dtype, 14)
    t = lambda y: y.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    a, b = run(x, 70, 5), run([t(y) for y in x], 70, 5)
    for i, (m, n) in enumerate(zip(a, b)):
        assert i == 2 or torch.equal(m, n)


@gpu
def test_hidden_rows_and_empty_rows():
    # a sequence without keys, and rows whose window lies behind the padding but whose first keys do not
    x = make(3, 2, 2, 500, 64, "bf16", 15)
    ln = torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda")
    got = run(x, 20, 2, ln)
    check(got, plain(*x, 20, 2, ln), "bf16")
    o, lse = got[:2]
    assert bool((o[0] == 0).all()) and bool((lse[0] == -math.inf).all()) and bool(torch.isfinite(lse[1:]).all())


@gpu
def test_streams_and_graphs():
    x = make(1, 4, 2, 3500, 64, "bf16", 16)
    q, k, v, do = x
    kw = dict(causal=True, window=130, sinks=4)

    def step(stream=None):
        o, lse = fa.fwd(q, k, v, stream=stream, **kw)
        return (o, lse) + tuple(fa.bwd(q, k, v, o, do, lse, stream=stream, **kw))

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for y in x:
        y.copy_(torch.randn_like(y))
    g.replay()
    torch.cuda.synchronize()
    want = step()
    check(out, plain(*x, 130, 4), "bf16")
    for i in (0, 1, 3, 4):
        assert torch.equal(out[i], want[i])


@gpu
def test_refusals_of_the_binding():
    q, k, v, do = make(1, 2, 2, 64, 64, "bf16")
    with pytest.raises(fa.FAError):
        fa.fwd(q, k, v, causal=True, window=10, sinks=-1)
    with pytest.raises(fa.FAError):
        fa.fwd(q, k, v, window=10, sinks=1)
    o, lse = fa.fwd(q, k, v, causal=True, window=10, sinks=1)
    with pytest.raises(fa.FAError):
        fa.bwd(q, k, v, o, do, lse, causal=True, window=10, sinks=-1)


@gpu
@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_of_a_sequence_without_keys_may_hold_anything(dtype, d, bad):
    # padding: nobody sees these rows, whatever they hold, with no, few and many first keys
    x = make(2, 4, 2, 400, d, dtype, 17)
    ln = torch.tensor([0, 400], dtype=torch.int32, device="cuda")
    want = {s: run(x, 64, s, ln) for s in (0, 4, 8, 9)}
    for t in x:
        t[0] = bad
    for s in want:
        got = run(x, 64, s, ln)
        o, lse, *grads = got
        assert bool((o[0] == 0).all()) and bool((lse[0] == -math.inf).all())
        for g, n in zip(grads, ("dq", "dk", "dv")):
            assert bool((g[0] == 0).all()), (s, n)
        for i, (a, b) in enumerate(zip(got, want[s])):
            assert i == 2 or torch.equal(a[1], b[1])


@gpu
@pytest.mark.parametrize("dtype,d", KINDS)
def test_a_window_longer_than_the_sequence_hides_nothing(dtype, d):
    N = 333
    x = make(2, 4, 2, N, d, dtype, 18)
    q, k, v, do = x
    want = run(x, 0, 0)
    for w in (N, N + 1, 2 ** 30, 2 ** 31 - 130, 2 ** 31 - 1, 2 ** 32 + 5, 2 ** 40):
        got = run(x, w, 0)
        for i, (a, b) in enumerate(zip(got, want)):
            if i == 2:
                assert rel(a, b.double()) <= (1e-6 if dtype == "f32" else torch.finfo(DT[dtype]).eps / 2), w
            else:
                assert torch.equal(a, b), (w, i)
        kw = dict(causal=True, window=w)
        assert torch.equal(fa.bwd_noalloc(q, k, v, *got[:1], do, got[1], **kw)[1], want[3]), w
        if dtype != "f32":
            assert torch.equal(fa.fwd_fp8(q, k, v, **kw)[0], fa.fwd_fp8(q, k, v, causal=True)[0]), w


@gpu
@pytest.mark.parametrize("dtype,d", KINDS)
def test_slices_of_a_fused_projection(dtype, d):
    # q, k and v as they lie in one projection, and rows and columns of larger tensors: outputs share their strides
    B, H, Hkv, N = 2, 4, 2, 300
    x = make(B, H, Hkv, N, d, dtype, 19)
    fused = torch.full((B, N, 2 * H + 2 * Hkv, d), math.nan, device="cuda", dtype=DT[dtype])
    at = (0, H, H + Hkv, H + 2 * Hkv)
    sliced = [fused[:, :, a:a + t.shape[1]].transpose(1, 2) for a, t in zip(at, x)]
    wide = [torch.full((B, t.shape[1], N + 5, d + 16), math.nan, device="cuda", dtype=DT[dtype])[:, :, :N, :d] for t in x]
    for w, s in ((0, 0), (70, 5), (70, 40)):
        want = run(x, w, s)
        for y in (sliced, wide):
            for a, b in zip(y, x):
                a.copy_(b)
            got = run(y, w, s)
            assert got[0].stride() == y[0].stride() and got[2].stride() == y[0].stride() and got[3].stride() == y[1].stride()
            for i, (m, n) in enumerate(zip(got, want)):
                assert i == 2 or torch.equal(m, n)
            assert rel(got[2], want[2].double()) <= (1e-6 if dtype == "f32" else torch.finfo(DT[dtype]).eps / 2)
            if s == 0:
                q, k, v, do = y
                assert torch.equal(fa.bwd_noalloc(q, k, v, got[0], do, got[1], causal=True, window=w)[1], want[3])
                if dtype != "f32":
                    assert torch.equal(fa.fwd_fp8(q, k, v, causal=True)[0], fa.fwd_fp8(*x[:3], causal=True)[0])
    keep = fused[:, :, at[-1] + H:]
    assert keep.numel() == 0 or bool(keep.isnan().all())
