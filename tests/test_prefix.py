"""Attention over a shared prefix (fa_prefix_fwd).

CPU: struct layout, refusals, the split rules' coverage.  GPU: both dtypes and
head dimensions over prefix and cache lengths around the 64-key tiles and the
split sizes, grouped heads, one and several tokens, empty parts, layouts,
rows that hold NaN, against a 64-bit plain form.

Tolerance, u = eps / 2 of the dtype: weights rounded once and normalised by
their rounded sum (2u), one rounding of O (u): |error| <= 2u sum P |v| + u |O|
(+ 2^-20 for the float32 sums); lse 2^-18 (1 + |lse|).
"""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from exact_io_aware_tiled_gb300 import _ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load()


# ---- CPU ----------------------------------------------------------------------------------------------------
def test_params_layout_matches_c(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    st = _ops.fa_prefix_params
    prog = ['#include <stdio.h>', '#include <stddef.h>', '#include "fa.h"', 'int main(void){',
            'printf("%zu\\n", sizeof(fa_prefix_params));']
    prog += ['printf("%%zu\\n", offsetof(fa_prefix_params, %s));' % f for f, _ in st._fields_] + ['return 0;}']
    c = tmp_path / "l.c"
    c.write_text("\n".join(prog))
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(c), "-o", str(tmp_path / "l")], check=True)
    vals = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True).stdout.split()]
    assert vals == [ctypes.sizeof(st)] + [getattr(st, f).offset for f, _ in st._fields_]


def _params(**kw):
    p = _ops.fa_prefix_params()
    p.B, p.H, p.H_kv, p.T, p.P, p.M, p.d, p.dtype = 3, 4, 2, 2, 500, 100, 64, 2
    for t, h, n in (("q", 4, 2), ("o", 4, 2), ("k", 2, 100), ("v", 2, 100), ("kp", 2, 500), ("vp", 2, 500)):
        setattr(p, t + "_stride_n", 64)
        setattr(p, t + "_stride_h", 64 * n)
        if t not in ("kp", "vp"):
            setattr(p, t + "_stride_b", 64 * n * h)
    p.seqlens_k = 1 << 22
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _call(p, ptrs=None, ws=1 << 40, ws_ptr=1 << 21):
    f = _ops._fn("fa_prefix_fwd", *([ctypes.c_void_p] * 9), ctypes.c_size_t, ctypes.c_void_p)
    return f(None if p is None else ctypes.addressof(p), *(ptrs or [1 << 20] * 7), ws_ptr, ws, None)


def _size(p):
    return _ops._fn("fa_prefix_workspace_size", ctypes.c_void_p, restype=ctypes.c_size_t)(ctypes.addressof(p))


@pytest.mark.parametrize("mut,code", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(T=0), 1), (dict(P=-1), 1), (dict(M=-1), 1), (dict(d=0), 1),
    (dict(dtype=4), 1), (dict(dtype=0), 2), (dict(d=96), 2), (dict(H_kv=3), 1), (dict(H_kv=-2), 1),
    (dict(P=(1 << 28) + 1), 2), (dict(M=(1 << 28) + 1), 2), (dict(B=1 << 22, T=64), 2),
    (dict(seqlens_k=0), 1), (dict(seqlens_k=(1 << 22) + 2), 3),
    (dict(q_stride_n=68), 3), (dict(k_stride_n=32), 1), (dict(kp_stride_h=4), 3), (dict(vp_stride_n=66), 3),
    (dict(v_stride_b=0), 1), (dict(lam=(1 << 22) + 2), 3), (dict(lam=1 << 22), 1), (dict(lam=1 << 22, d=128), 2),
])
def test_refusals_before_launch(mut, code):
    assert _call(_params(**mut)) == code


def test_null_misaligned_and_small_workspaces():
    assert _call(None) == 1
    for i in range(7):
        ptrs = [1 << 20] * 7
        ptrs[i] = None
        assert _call(_params(), ptrs) == 1
        ptrs[i] = (1 << 20) + 2
        assert _call(_params(), ptrs) == 3
    need = _size(_params())
    assert need > 256
    assert _call(_params(), ws=need - 1) == 4 and _call(_params(), ws_ptr=None) == 4
    assert _call(_params(), ws_ptr=(1 << 21) + 8) == 4


def test_workspace_holds_every_split():
    # 1,024 rows of a head against a long prefix, and ragged caches: never less than one partial row per query row
    for kw in (dict(), dict(P=0), dict(M=0), dict(B=128, H=16, P=32769, M=2048, d=128), dict(T=64, P=10),
               dict(B=1, H=2, T=1, P=100000, M=1)):
        p = _params(**kw)
        for t in ("q", "o", "k", "v", "kp", "vp"):
            setattr(p, t + "_stride_n", p.d)
        rows = p.B * p.H * p.T * ((p.P > 0) + (p.M > 0))
        assert _size(p) >= 256 + rows * (p.d * 4 + 16)


def test_binding_refuses():
    q = torch.zeros(1, 2, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.prefix_fwd(q, None, None, None, None, None)


# ---- GPU ----------------------------------------------------------------------------------------------------
def inputs(B, H, Hkv, T, P, M, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    return r(B, H, T, d), r(Hkv, P, d), r(Hkv, P, d), r(B, Hkv, M, d), r(B, Hkv, M, d)


def plain(q, kp, vp, k, v, lens, scale=None):
    """Float64: o, lse, sum P |v|."""
    B, H, T, d = q.shape
    Hkv, P = kp.shape[:2]
    M, G, dv = k.shape[2], H // Hkv, v.shape[3]
    scale = d ** -0.5 if scale is None else scale
    kk = torch.cat((kp[None].expand(B, Hkv, P, d), k), 2).double()
    vv = torch.cat((vp[None].expand(B, Hkv, P, dv), v), 2).double()
    j = torch.arange(M, device=q.device)
    t = torch.arange(T, device=q.device)
    lens = lens.clamp(0, M)
    own = j[None, None] <= lens.to(q.device)[:, None, None] - T + t[None, :, None]
    see = torch.cat((torch.ones(B, T, P, dtype=torch.bool, device=q.device), own), -1)
    see = see[:, None].expand(B, G, T, P + M).reshape(B, 1, G * T, P + M)
    hidden = ~torch.cat((torch.ones(B, P, dtype=torch.bool, device=q.device),
                         j[None] < lens.to(q.device)[:, None]), 1)[:, None, :, None]
    kk, vv = kk.masked_fill(hidden, 0.0), vv.masked_fill(hidden, 0.0)
    s = q.double().reshape(B, Hkv, G * T, d) @ kk.transpose(-1, -2) * scale
    none = ~see.any(-1, keepdim=True)
    s = s.masked_fill(~(see | none), -math.inf)
    p = torch.softmax(s, -1) * ~none
    o, mag = p @ vv, p @ vv.abs()
    lse = torch.logsumexp(s, -1).masked_fill(none.squeeze(-1), -math.inf)
    return o.reshape(B, H, T, dv), lse.reshape(B, H, T), mag.reshape(B, H, T, dv)


def check(got, want, dtype):
    u = torch.finfo(DT[dtype]).eps / 2
    o, lse = got
    wo, wl, mag = want
    err = (o.double() - wo).abs()
    bound = 2 * u * mag + u * wo.abs() + 2.0 ** -20
    assert bool((err <= bound).all()), float((err / bound).max())
    fin = torch.isfinite(wl)
    assert torch.equal(fin, torch.isfinite(lse)) and bool((lse[~fin] == -math.inf).all())
    assert bool(((lse.double() - wl)[fin].abs() <= 2.0 ** -18 * (1 + wl[fin].abs())).all())


def run(B, H, Hkv, T, P, M, d, dtype, lens, seed=0, scale=None):
    x = inputs(B, H, Hkv, T, P, M, d, dtype, seed)
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = fa.prefix_fwd(*x, lens, scale=scale)
    assert fa.check_status(fa.prefix_fwd.last_workspace) == 0
    check(got, plain(*x, lens, scale=scale), dtype)
    return x, lens, got


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [0, 1, 63, 64, 65, 257, 1500])
def test_prefix_lengths(dtype, d, P):
    run(3, 4, 2, 1, P, 70, d, dtype, [0, 1, 70], seed=P)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("M,lens", [(1, [0, 1, 1, 0]), (64, [0, 15, 16, 64]), (65, [63, 64, 65, 17]),
                                    (700, [0, 255, 256, 257]), (700, [699, 700, 3, 320]), (256, [300, -4, 5, 256])])
def test_cache_lengths(d, M, lens):
    run(4, 6, 3, 1, 100, M, d, "bf16", lens, seed=M)
    run(4, 6, 3, 1, 0, M, d, "f16", lens, seed=M)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,H,Hkv,T", [(1, 1, 1, 1), (1, 16, 16, 1), (2, 16, 2, 1), (17, 2, 1, 1), (5, 8, 1, 2),
                                       (3, 12, 12, 5), (2, 8, 2, 9), (70, 8, 1, 1), (1, 2, 1, 100), (4, 6, 2, 33)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_and_groups(dtype, B, H, Hkv, T, d):
    lens = [(37 * b + T) % 200 for b in range(B)]
    run(B, H, Hkv, T, 330, 200, d, dtype, lens, seed=B * T)


@pytest.mark.gpu
def test_fewer_rows_filled_than_tokens():
    # the first T - L_b tokens see only the prefix; without one they see nothing
    for P in (0, 5):
        x, lens, (o, lse) = run(4, 4, 2, 6, P, 40, 64, "bf16", [0, 1, 5, 6])
        if P == 0:
            assert bool((o[0] == 0).all()) and bool((lse[1, :, :5] == -math.inf).all())


@pytest.mark.gpu
def test_empty_parts_and_none():
    q, kp, vp, k, v = inputs(2, 4, 4, 1, 90, 50, 64, "bf16", 2)
    lens = torch.tensor([50, 20], dtype=torch.int32, device="cuda")
    a = fa.prefix_fwd(q, None, None, k, v, lens)
    b = fa.prefix_fwd(q, kp[:, :0], vp[:, :0], k, v, lens)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = fa.prefix_fwd(q, kp, vp, None, None, lens)
    check(c, plain(q, kp, vp, k[:, :, :0], v[:, :, :0], lens), "bf16")
    z = fa.prefix_fwd(q, kp[:, :0], vp[:, :0], k, v, torch.zeros_like(lens))
    assert bool((z[0] == 0).all()) and bool((z[1] == -math.inf).all())
    with pytest.raises(ValueError):
        fa.prefix_fwd(q, None, None, None, None, lens)
    with pytest.raises(ValueError):
        fa.prefix_fwd(q, kp, None, k, v, lens)
    with pytest.raises(ValueError):
        fa.prefix_fwd(q, kp, vp, k, v, None)
    with pytest.raises(ValueError):
        fa.prefix_fwd(q, kp, vp, k, v, lens.float())
    with pytest.raises(ValueError):
        fa.prefix_fwd(q, kp[:3], vp[:3], k, v, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 4), (5, 16)])
def test_rows_behind_the_caches_may_hold_nan_and_stay(T, H):
    q, kp, vp, k, v = inputs(4, H, 2, T, 300, 400, 128, "bf16", 3)
    lens = torch.tensor([0, 77, 256, 399], dtype=torch.int32, device="cuda")
    want = fa.prefix_fwd(q, kp, vp, k, v, lens)
    k2, v2 = k.clone(), v.clone()
    for b, n in enumerate(lens.tolist()):
        k2[b, :, n:] = float("nan")
        v2[b, :, n:] = float("nan")
        v2[b, :, n] = float("inf")
    kc, vc = k2.clone(), v2.clone()
    got = fa.prefix_fwd(q, kp, vp, k2, v2, lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(k2.view(torch.int16), kc.view(torch.int16)) and torch.equal(v2.view(torch.int16), vc.view(torch.int16))


@pytest.mark.gpu
def test_large_scores_and_a_long_prefix():
    # scores of several hundred: the maxima of the splits differ by far more than float32's exponent step
    x = list(inputs(5, 8, 2, 1, 9000, 300, 64, "f16", 5))
    x[0] = x[0] * 20
    lens = torch.tensor([0, 300, 1, 64, 299], dtype=torch.int32, device="cuda")
    got = fa.prefix_fwd(*x, lens)
    check(got, plain(*x, lens), "f16")


@pytest.mark.gpu
def test_layouts_buffers_and_repeats():
    B, H, Hkv, T, P, M, d = 3, 8, 4, 2, 200, 130, 64
    q, kp, vp, k, v = inputs(B, H, Hkv, T, P, M, d, "bf16", 6)
    lens = torch.tensor([130, 60, 2], dtype=torch.int32, device="cuda")
    want = fa.prefix_fwd(q, kp, vp, k, v, lens)
    sw = lambda t: t.transpose(-3, -2).contiguous().transpose(-3, -2)  # noqa: E731
    wide = torch.zeros(B, Hkv, M, 3 * d, device="cuda", dtype=torch.bfloat16)
    wide[..., d:2 * d] = v
    o = torch.empty(B, T, H, d, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
    lse = torch.empty(B, H, T, device="cuda")
    ws = torch.empty(1 << 24, device="cuda", dtype=torch.uint8).fill_(255)
    for _ in range(3):
        got = fa.prefix_fwd(sw(q), sw(kp), sw(vp), sw(k), wide[..., d:2 * d], lens.long(), out=(o, lse), workspace=ws)
        assert got[0] is o and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # float64 lens are refused, other whole types converted
    assert torch.equal(fa.prefix_fwd(q, kp, vp, k, v, lens.to(torch.int16))[0], want[0])


@pytest.mark.gpu
def test_agrees_with_the_square_forward():
    # the last query of a causal forward over prefix + cache is one decoding step
    B, H, d, P, n = 2, 4, 64, 130, 71
    q, kp, vp, k, v = inputs(B, H, H, 1, P, n, d, "bf16", 7)
    full_q = torch.zeros(B, H, P + n, d, device="cuda", dtype=torch.bfloat16)
    full_q[:, :, -1:] = q
    kk = torch.cat((kp[None].expand(B, H, P, d), k), 2).contiguous()
    vv = torch.cat((vp[None].expand(B, H, P, d), v), 2).contiguous()
    o, lse = fa.fwd(full_q, kk, vv, causal=True)
    got = fa.prefix_fwd(q, kp, vp, k, v, torch.full((B,), n, device="cuda", dtype=torch.int32))
    # both round their weights once: 2u apart from the exact value each, plus one rounding each
    assert bool(((got[0] - o[:, :, -1:]).float().abs() <= 6 * 2.0 ** -8 * vv.float().abs().amax()).all())
    assert torch.allclose(got[1], lse[:, :, -1:], atol=2e-5)


@pytest.mark.gpu
def test_graph_replay_grows_with_the_caches_and_other_stream():
    B, H, Hkv, T, P, M, d = 4, 8, 2, 1, 500, 300, 128
    q, kp, vp, k, v = inputs(B, H, Hkv, T, P, M, d, "bf16", 8)
    lens = torch.tensor([1, 0, 64, 200], dtype=torch.int32, device="cuda")
    fa.prefix_fwd(q, kp, vp, k, v, lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = fa.prefix_fwd(q, kp, vp, k, v, lens)
    for step in range(3):
        g.replay()
        check((o, lse), plain(q, kp, vp, k, v, lens), "bf16")
        lens += 33
        q.copy_(torch.randn_like(q.float()).bfloat16())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = fa.prefix_fwd(q, kp, vp, k, v, lens, stream=s)
    s.synchronize()
    b = fa.prefix_fwd(q, kp, vp, k, v, lens)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,T,P", [(33, 8, 2, 1, 256), (65, 4, 1, 1, 700), (129, 2, 2, 1, 385), (16, 8, 1, 3, 4097),
                                         (300, 2, 2, 1, 1000), (7, 6, 1, 40, 2049)])
def test_many_rows_against_the_prefix(dtype, d, B, H, Hkv, T, P):
    # row tiles of 64 that the last rows fill in part
    lens = [(11 * b) % 31 for b in range(B)]
    run(B, H, Hkv, T, P, 31, d, dtype, lens, seed=B + P)


@pytest.mark.gpu
def test_many_rows_layouts_and_large_scores():
    B, H, Hkv, T, P, M, d = 50, 8, 2, 1, 900, 20, 128
    q, kp, vp, k, v = inputs(B, H, Hkv, T, P, M, d, "f16", 9)
    lens = torch.arange(B, device="cuda", dtype=torch.int32) % 21
    qs = (q * 15).transpose(0, 1).contiguous().transpose(0, 1)
    kps = kp.transpose(0, 1).contiguous().transpose(0, 1)
    check(fa.prefix_fwd(qs, kps, vp, k, v, lens), plain(qs, kp, vp, k, v, lens), "f16")


# ---- differential form --------------------------------------------------------------------------------------
def diff_inputs(B, H, Hkv, T, P, M, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    lam = torch.rand(H, generator=g, device="cuda") * 0.9 + 0.05
    return (r(B, 2 * H, T, 64), r(2 * Hkv, P, 64), r(Hkv, P, 128), r(B, 2 * Hkv, M, 64), r(B, Hkv, M, 128)), lam


def diff_plain(q, kp, vp, k, v, lens, lam, scale=None):
    a, b = (plain(q[:, x::2], kp[x::2], vp, k[:, x::2], v, lens, scale) for x in range(2))
    w = lam.double()[None, :, None, None]
    return a[0] - w * b[0], torch.stack((a[1], b[1]), 2).flatten(1, 2), a[2] + w.abs() * b[2]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,H,Hkv,T,P,M", [(1, 1, 1, 1, 0, 5), (2, 4, 4, 1, 130, 40), (5, 6, 2, 1, 700, 300),
                                          (3, 4, 1, 5, 65, 64), (33, 8, 2, 1, 300, 20), (70, 8, 1, 2, 1025, 9),
                                          (9, 2, 2, 3, 0, 600), (2, 16, 4, 1, 20000, 50)])
def test_differential_steps(dtype, B, H, Hkv, T, P, M):
    x, lam = diff_inputs(B, H, Hkv, T, P, M, dtype, seed=B + P)
    lens = (torch.arange(B, device="cuda", dtype=torch.int32) * 7 + T) % (M + 1)
    got = fa.prefix_fwd(*x, lens, lam=lam)
    assert fa.check_status(fa.prefix_fwd.last_workspace) == 0
    check(got, diff_plain(*x, lens, lam), dtype)


@pytest.mark.gpu
def test_differential_step_is_the_forward_pass_last_row():
    from tests import test_diff
    B, H, Hkv, N = 2, 4, 2, 211
    q, k, v, lam, _ = test_diff.inputs(B, H, Hkv, N, "bf16", 3)
    o, lse, _ = fa.diff_fwd(q, k, v, lam, causal=True)
    lens = torch.full((B,), N, device="cuda", dtype=torch.int32)
    got = fa.prefix_fwd(q[:, :, -3:], None, None, k, v, lens, lam=lam)       # the last three tokens
    # each side rounds its weights once (2u of sum P |v|) and O once
    u = 2.0 ** -8
    bound = 2 * (2 * u * 2 * v.float().abs().amax() + u * o.float().abs().amax())
    assert float((got[0] - o[:, :, -3:]).float().abs().max()) <= bound
    assert torch.allclose(got[1], lse[:, :, -3:], atol=2e-5)


@pytest.mark.gpu
def test_differential_form_masks_nan_and_refuses():
    x, lam = diff_inputs(3, 4, 2, 2, 100, 60, "bf16", 4)
    lens = torch.tensor([0, 60, 17], device="cuda", dtype=torch.int32)
    want = fa.prefix_fwd(*x, lens, lam=lam)
    k, v = x[3].clone(), x[4].clone()
    for b, n in enumerate(lens.tolist()):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("nan")
    got = fa.prefix_fwd(*x[:3], k, v, lens, lam=lam)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    none = fa.prefix_fwd(x[0], None, None, x[3], x[4], torch.zeros_like(lens), lam=lam)
    assert bool((none[0] == 0).all()) and bool((none[1] == -math.inf).all())
    for bad in (dict(lam=lam[:3]), dict(lam=lam.double()), dict()):
        with pytest.raises(ValueError):
            fa.prefix_fwd(*x, lens, **bad)


# ---- the tensor-memory kernel: more than 32 rows and a long prefix ------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,H,Hkv,T,P,d", [
    (1, 16, 4, 10, 65637, 64), (2, 8, 8, 33, 33001, 64), (1, 128, 4, 4, 70000, 64),    # two splits a CTA: 40, 66, 128 rows
    (2, 32, 4, 10, 30001, 64), (1, 16, 2, 129, 8000, 64), (16, 8, 1, 3, 60001, 64),    # 256-row tiles: 160, 1,032, 384 rows
    (1, 16, 4, 10, 33000, 128), (2, 32, 4, 10, 11001, 128), (1, 16, 2, 129, 3900, 128)])
def test_long_prefix(dtype, B, H, Hkv, T, P, d):
    lens = [(11 * b) % 31 for b in range(B)]
    run(B, H, Hkv, T, P, 31, d, dtype, lens, seed=B + P)


@pytest.mark.gpu
@pytest.mark.parametrize("d,P", [(64, 65600), (128, 33000)])
def test_long_prefix_layouts_and_large_scores(d, P):
    B, H, Hkv, T, M = 3, 8, 4, 10, 20
    q, kp, vp, k, v = inputs(B, H, Hkv, T, P, M, d, "f16", 9)
    lens = torch.tensor([0, 20, 13], device="cuda", dtype=torch.int32)
    qs = (q * 15).transpose(0, 1).contiguous().transpose(0, 1)
    kps = kp.transpose(0, 1).contiguous().transpose(0, 1)
    want = plain(qs, kp, vp, k, v, lens)
    check(fa.prefix_fwd(qs, kps, vp, k, v, lens), want, "f16")
    # without caches of their own
    got = fa.prefix_fwd(qs, kps, vp, None, None, torch.zeros_like(lens))
    check(got, plain(qs, kp, vp, k[:, :, :0], v[:, :, :0], torch.zeros_like(lens)), "f16")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,H,Hkv,T,P", [(1, 8, 4, 20, 40000), (3, 4, 2, 50, 14001)])
def test_long_prefix_differential(dtype, B, H, Hkv, T, P):
    x, lam = diff_inputs(B, H, Hkv, T, P, 60, dtype, seed=P)
    lens = (torch.arange(B, device="cuda", dtype=torch.int32) * 7 + T) % 61
    got = fa.prefix_fwd(*x, lens, lam=lam)
    assert fa.check_status(fa.prefix_fwd.last_workspace) == 0
    check(got, diff_plain(*x, lens, lam), dtype)


@pytest.mark.gpu
def test_no_keys_at_all():
    q, kp, vp, k, v = inputs(5, 4, 2, 3, 0, 0, 64, "bf16")
    lens = torch.tensor([0, 7, 0, 2, 1], device="cuda", dtype=torch.int32)
    for x in ((kp, vp, k, v), (kp, vp, None, None), (None, None, k, v)):
        o, lse = fa.prefix_fwd(q, *x, lens)
        assert fa.check_status(fa.prefix_fwd.last_workspace) == 0
        assert bool((o == 0).all()) and bool((lse == -math.inf).all())
