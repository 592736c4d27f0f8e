"""Differential attention (fa_diff_fwd, fa_diff_bwd).

CPU: struct layout, workspace sizes, refusals.  GPU: both dtypes over ragged
lengths, grouped heads, padding, windows and layouts against a 64-bit plain
form whose gradients come from autograd.

Tolerances, for a dtype whose rounding is off by at most u = torch.finfo.eps / 2
relative to the value (bf16 2^-8, fp16 2^-11):
* O: a convex combination of V rows with weights rounded once (u each) and
  normalised by the sum of the rounded weights, twice, then one rounding of O:
  |error| <= 2u (O_1bar + |lambda| O_2bar) + u |O| with O_mbar = sum P_m |V|.
* lse: float32; scores of 64 products and one exponential, 2^-18 absolute here
  (inputs of unit size).
* gradients, relative Frobenius: P (fp32) and dP are exact to 2^-20; W and dS
  are rounded once (u), D_m carries the rounding of O and O_2, the result is
  rounded once: 4u in all.
* dlambda: float32 sums of float32 products: 2^-16 of the sum of magnitudes'
  root-mean-square bound ||P_2 o dP||_F sqrt(n) is far above it; the check is
  1e-5 relative to sqrt(sum of D_2^2) summed over rows.
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
    st = _ops.fa_diff_params
    prog = ['#include <stdio.h>', '#include <stddef.h>', '#include "fa.h"', 'int main(void){',
            'printf("%zu\\n", sizeof(fa_diff_params));']
    prog += ['printf("%%zu\\n", offsetof(fa_diff_params, %s));' % f for f, _ in st._fields_] + ['return 0;}']
    c = tmp_path / "l.c"
    c.write_text("\n".join(prog))
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(c), "-o", str(tmp_path / "l")], check=True)
    vals = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True).stdout.split()]
    assert vals == [ctypes.sizeof(st)] + [getattr(st, f).offset for f, _ in st._fields_]


def _params(**kw):
    p = _ops.fa_diff_params()
    p.B, p.H, p.H_kv, p.N, p.d, p.dtype = 2, 4, 2, 200, 64, 2
    for t, h, c in (("q", 8, 64), ("k", 4, 64), ("v", 2, 128), ("o", 4, 128), ("do", 4, 128)):
        setattr(p, t + "_stride_n", c)
        setattr(p, t + "_stride_h", 200 * c)
        setattr(p, t + "_stride_b", 200 * c * h)
    p.lam = 1 << 22
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _fwd(p, ptrs=None, ws=1 << 30, ws_ptr=1 << 21):
    f = _ops._fn("fa_diff_fwd", *([ctypes.c_void_p] * 8), ctypes.c_size_t, ctypes.c_void_p)
    return f(p if p is None else ctypes.addressof(p), *(ptrs or [1 << 20] * 6), ws_ptr, ws, None)


def _bwd(p, ptrs=None, ws=1 << 30, ws_ptr=1 << 21):
    f = _ops._fn("fa_diff_bwd", *([ctypes.c_void_p] * 13), ctypes.c_size_t, ctypes.c_void_p)
    return f(p if p is None else ctypes.addressof(p), *(ptrs or [1 << 20] * 11), ws_ptr, ws, None)


@pytest.mark.parametrize("mut,code", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(N=0), 1), (dict(d=0), 1), (dict(dtype=9), 1), (dict(H_kv=-1), 1),
    (dict(d=128), 2), (dict(d=32), 2), (dict(dtype=0), 2), (dict(H_kv=3), 1), (dict(window=-1, causal=1), 1),
    (dict(window=4), 2), (dict(lam=0), 1), (dict(lam=(1 << 22) + 2), 3), (dict(seqlens_k=(1 << 22) + 1), 3),
    (dict(q_stride_n=68), 3), (dict(k_stride_h=12804), 3), (dict(v_stride_n=64), 1), (dict(o_stride_h=0), 1),
    (dict(B=1 << 12, N=1 << 18), 2),
])
def test_refusals_before_launch(mut, code):
    assert _fwd(_params(**mut)) == code
    assert _bwd(_params(**mut)) == code


def test_null_misaligned_and_small_workspaces():
    assert _fwd(None) == 1 and _bwd(None) == 1
    for i in range(6):
        ptrs = [1 << 20] * 6
        ptrs[i] = None
        if i != 4:                              # o2 may be left out
            assert _fwd(_params(), ptrs) == 1
        ptrs[i] = (1 << 20) + 8
        assert _fwd(_params(), ptrs) == 3
    for i in range(11):
        ptrs = [1 << 20] * 11
        ptrs[i] = None
        assert _bwd(_params(), ptrs) == 1
        ptrs[i] = (1 << 20) + 2
        assert _bwd(_params(), ptrs) == 3
    assert _bwd(_params(do_stride_n=130)) == 3
    p = _params()
    lib = fa.load()
    lib.fa_diff_bwd_workspace_size.restype = ctypes.c_size_t
    need = _ops._fn("fa_diff_bwd_workspace_size", ctypes.c_void_p, restype=ctypes.c_size_t)(ctypes.addressof(p))
    assert need >= 2 * 8 * 200 * 64 * 4 + 2 * 4 * 256 * 16
    assert _bwd(p, ws=need - 1) == 4 and _bwd(p, ws_ptr=None) == 4 and _bwd(p, ws_ptr=(1 << 21) + 4) == 4
    assert _fwd(p, ws=16) == 4


def test_binding_refuses():
    q, k, v, lam = torch.zeros(1, 4, 8, 64), torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 128), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.diff_fwd(q, k, v, lam)
    with pytest.raises(ValueError):
        fa.diff_fwd(q[0], k, v, lam)


# ---- GPU ----------------------------------------------------------------------------------------------------
def inputs(B, H, Hkv, N, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(DT[dtype]).cuda()  # noqa: E731
    return (r(B, 2 * H, N, 64), r(B, 2 * Hkv, N, 64), r(B, Hkv, N, 128),
            (torch.rand(H, generator=g) * 0.9 + 0.05).cuda(), r(B, H, N, 128))


def plain(q, k, v, lam, do, causal=False, lens=None, window=0, scale=0.125):
    """Float64 on the GPU: o, lse, o2, error scale of o, (dq, dk, dv, dlam), sqrt(sum D_2^2) per head."""
    B, H2, N, _ = q.shape
    H, Hkv = H2 // 2, v.shape[1]
    q, k, v, lam = (t.double().requires_grad_(True) for t in (q, k, v, lam))
    i = torch.arange(N, device=q.device)
    see = torch.ones(B, 1, N, N, dtype=torch.bool, device=q.device)
    if causal:
        see = see & (i[None, :] <= i[:, None])
    if window:
        see = see & (i[None, :] > i[:, None] - window)
    if lens is not None:
        see = see & (i[None, None, None, :] < lens.to(q.device)[:, None, None, None])
    none = ~see.any(-1, keepdim=True)
    rep = H // Hkv
    kk = k.view(B, Hkv, 1, 2, N, 64).expand(B, Hkv, rep, 2, N, 64).reshape(B, H, 2, N, 64)
    vv = v[:, :, None].expand(B, Hkv, rep, N, 128).reshape(B, H, N, 128)
    s = torch.einsum("bhmid,bhmjd->bhmij", q.view(B, H, 2, N, 64), kk) * scale
    s = s.masked_fill(~(see | none)[:, :, None], -math.inf)
    p = torch.softmax(s, -1) * (~none)[:, :, None]
    o1, o2 = p[:, :, 0] @ vv, p[:, :, 1] @ vv
    o = o1 - lam[None, :, None, None] * o2
    grads = torch.autograd.grad(o, (q, k, v, lam), do.double())
    lse = torch.logsumexp(s.detach(), -1).masked_fill(none.squeeze(-1)[:, :, None], -math.inf).reshape(B, H2, N)
    with torch.no_grad():
        av = vv.abs()
        mag = p[:, :, 0] @ av + lam.abs()[None, :, None, None] * (p[:, :, 1] @ av)
        d2 = (do.double() * o2).sum(-1)
    return o.detach(), lse, o2.detach(), mag, grads, d2.square().sum((0, 2)).sqrt()


def rel(x, y):
    n = float(y.norm())
    return float((x.double() - y).norm()) / n if n else float(x.double().norm())


def check_fwd(got, want, dtype):
    o, lse, o2 = got
    u = torch.finfo(DT[dtype]).eps / 2
    wo, wl, w2, mag = want[:4]
    assert bool(((o.double() - wo).abs() <= 2 * u * mag + u * wo.abs() + 1e-6).all())
    if o2 is not None:
        assert bool(((o2.double() - w2).abs() <= 2 * u * mag / 0.05 + u * w2.abs() + 1e-6).all())
        assert rel(o2, w2) <= 2 * u
    fin = torch.isfinite(wl)
    assert torch.equal(fin, torch.isfinite(lse)) and bool((lse[~fin] == -math.inf).all())
    assert bool(((lse.double() - wl)[fin].abs() <= 2.0 ** -18 * (1 + wl[fin].abs())).all())


def check_grads(got, want, dtype, floor=False):
    u = torch.finfo(DT[dtype]).eps / 2
    for x, y, n in zip(got[:3], want[4][:3], ("dq", "dk", "dv")):
        assert rel(x, y) <= 4 * u, (n, rel(x, y))
    err = (got[3].double() - want[4][3]).abs()
    assert bool((err <= 1e-5 * want[5] + 1e-6).all()), float((err / want[5]).max())


def run(B, H, Hkv, N, dtype, seed=0, **mask):
    q, k, v, lam, do = inputs(B, H, Hkv, N, dtype, seed)
    m = dict(mask)
    lens = m.pop("lens", None)
    if lens is not None:
        lens = torch.tensor(lens, dtype=torch.int32)
        m["seqlens_k"] = lens.cuda()
    o, lse, o2 = fa.diff_fwd(q, k, v, lam, **m)
    assert fa.check_status(fa.diff_fwd.last_workspace) == 0
    g = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, **m)
    assert fa.check_status(fa.diff_bwd.last_workspace) == 0
    m.pop("seqlens_k", None)
    want = plain(q, k, v, lam, do, lens=lens, **m)
    return (o, lse, o2), g, want


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("N", [2, 63, 64, 65, 127, 128, 129, 300, 513])
def test_lengths(dtype, causal, N):
    got, g, want = run(2, 3, 3, N, dtype, seed=N, causal=causal)
    check_fwd(got, want, dtype)
    check_grads(g, want, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_token(dtype):
    # one key: P = 1 on both maps, dQ = dK = 0 up to the rounding of O and O_2 in D
    got, g, want = run(3, 2, 1, 1, dtype)
    check_fwd(got, want, dtype)
    u = torch.finfo(DT[dtype]).eps / 2
    assert rel(g[2], want[4][2]) <= 4 * u
    # |dP - D| <= u sum |dO| (|O| + 2 |O_2|) over 128 columns of unit size, times tau and a column of size <= 5
    assert float(g[0].abs().max()) <= u * 128 * 4 * 3 * 5 * 0.125 and float(g[1].abs().max()) <= u * 128 * 4 * 6 * 5 * 0.125


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hkv", [(4, 1), (6, 2), (1, 1)])
@pytest.mark.parametrize("mask", [dict(causal=True), dict(causal=True, window=1), dict(causal=True, window=100),
                                  dict(causal=True, window=2 ** 31 - 1), dict(lens=[0, 1, 200, 257]),
                                  dict(causal=True, lens=[0, 129, 128, 300]),
                                  dict(causal=True, window=130, lens=[5, 0, 256, 257]), dict(scale=0.3)])
def test_masks_and_groups(dtype, H, Hkv, mask):
    got, g, want = run(4, H, Hkv, 257, dtype, seed=H, **mask)
    check_fwd(got, want, dtype)
    if mask.get("window") == 1:      # one key a row: no gradient through the maps but rounding residues
        assert rel(g[2], want[4][2]) <= 4 * torch.finfo(DT[dtype]).eps / 2
        return
    check_grads(g, want, dtype)


@pytest.mark.gpu
def test_long_row_with_window_and_many_heads():
    got, g, want = run(1, 2, 2, 2500, "bf16", seed=5, causal=True, window=700)
    check_fwd(got, want, "bf16")
    check_grads(g, want, "bf16")


@pytest.mark.gpu
def test_rows_behind_the_sequences_may_hold_nan():
    B, H, Hkv, N = 3, 2, 1, 300
    q, k, v, lam, do = inputs(B, H, Hkv, N, "bf16", 3)
    lens = torch.tensor([0, 77, 256], dtype=torch.int32).cuda()
    ref = fa.diff_fwd(q, k, v, lam, seqlens_k=lens)
    gref = fa.diff_bwd(q, k, v, lam, ref[0], ref[2], do, ref[1], seqlens_k=lens)
    k2, v2 = k.clone(), v.clone()
    for b, n in enumerate(lens.tolist()):
        k2[b, :, n:] = float("nan")
        v2[b, :, n:] = float("inf")
        v2[b, :, n + 1:] = float("nan")
    got = fa.diff_fwd(q, k2, v2, lam, seqlens_k=lens)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    g = fa.diff_bwd(q, k2, v2, lam, got[0], got[2], do, got[1], seqlens_k=lens)
    for i, (a, b) in enumerate(zip(g, gref)):
        if i == 0:        # dQ is accumulated in arrival order
            assert rel(a, b.double()) <= 2.0 ** -8
        else:
            assert torch.equal(a, b)
    assert bool((g[1][0] == 0).all()) and bool((g[2][1, :, 77:] == 0).all())


@pytest.mark.gpu
def test_lambda_zero_is_plain_attention_and_negative_adds():
    q, k, v, lam, do = inputs(2, 2, 2, 200, "bf16", 4)
    zero = torch.zeros_like(lam)
    o, lse, o2 = fa.diff_fwd(q, k, v, zero, causal=True)
    for half in (0, 1):
        po, pl = fa.fwd(q[:, 0::2].contiguous(), k[:, 0::2].contiguous(), v[..., 64 * half:64 * half + 64].contiguous(),
                        causal=True)
        assert rel(o[..., 64 * half:64 * half + 64], po.double()) <= 2.0 ** -8
        assert torch.allclose(pl, lse[:, 0::2], atol=1e-5)
    g = fa.diff_bwd(q, k, v, zero, o, o2, do, lse, causal=True)
    assert bool((g[0][:, 1::2] == 0).all()) and bool((g[1][:, 1::2] == 0).all())
    want = plain(q, k, v, zero, do, causal=True)
    assert rel(g[0], want[4][0]) <= 2.0 ** -7 and rel(g[3], want[4][3]) <= 1e-4
    got = fa.diff_fwd(q, k, v, -2 * lam, causal=True)
    check_fwd(got, plain(q, k, v, -2 * lam, do, causal=True), "bf16")


@pytest.mark.gpu
def test_strided_inputs_and_caller_buffers():
    B, H, Hkv, N = 2, 4, 2, 190
    base = inputs(B, H, Hkv, N, "bf16", 6)
    ref = fa.diff_fwd(*base[:4], causal=True)
    gref = fa.diff_bwd(*base[:4], ref[0], ref[2], base[4], ref[1], causal=True)
    bnhd = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    q, k, v, do = (bnhd(t) for t in (base[0], base[1], base[2], base[4]))
    empty = lambda: torch.full((B, N, H, 128), 7.0, device="cuda", dtype=torch.bfloat16).transpose(1, 2)  # noqa: E731
    o, o2, lse = empty(), empty(), torch.empty((B, 2 * H, N), device="cuda")
    ws = torch.empty(1 << 24, device="cuda", dtype=torch.uint8)
    got = fa.diff_fwd(q, k, v, base[3], causal=True, out=(o, lse, o2), workspace=ws)
    assert got[0] is o and got[2] is o2
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    g = fa.diff_bwd(q, k, v, base[3], o, o2, do, lse, causal=True, workspace=ws)
    assert g[0].stride() == q.stride() and g[2].stride() == v.stride()
    for a, b in zip(g[1:], gref[1:]):
        assert torch.equal(a, b)
    assert rel(g[0], gref[0].double()) <= 2.0 ** -8
    # 16-byte (not 32-byte) aligned dk, dv
    pad = lambda t: torch.empty(t.numel() + 8, device="cuda", dtype=t.dtype)[8:].view(t.shape)  # noqa: E731
    outs = (torch.empty_like(base[0]), pad(base[1]), pad(base[2]), torch.empty(H, device="cuda"))
    fa.diff_bwd(*base[:4], ref[0], ref[2], base[4], ref[1], causal=True, out=outs)
    assert torch.equal(outs[1], gref[1]) and torch.equal(outs[2], gref[2]) and torch.equal(outs[3], gref[3])
    no2 = fa.diff_fwd(*base[:4], causal=True, need_o2=False)
    assert no2[2] is None and torch.equal(no2[0], ref[0])
    with pytest.raises(ValueError):
        fa.diff_bwd(*base[:4], ref[0], o2, base[4], ref[1])      # o and o2 with other strides
    with pytest.raises(ValueError):
        fa.diff_fwd(*base[:3], base[3].double())
    with pytest.raises(fa.FAError):
        fa.diff_fwd(*base[:4], window=5)


@pytest.mark.gpu
def test_gradients_against_differences():
    # float64 differences of the plain form's loss: the kernel's gradient along random directions
    q, k, v, lam, do = inputs(1, 2, 1, 150, "f16", 7)
    o, lse, o2 = fa.diff_fwd(q, k, v, lam, causal=True)
    g = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True)

    def loss(*x):
        return float((plain(*x, do, causal=True)[0] * do.double()).sum())
    gen = torch.Generator().manual_seed(1)
    base = [t.double() for t in (q, k, v, lam)]
    for i in range(4):
        dx = torch.randn(base[i].shape, generator=gen).cuda().double()
        h = 1e-4
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + h * dx, base[i] - h * dx
        quot = (loss(*up) - loss(*dn)) / (2 * h)
        got = float((g[i].double() * dx).sum())
        # the gradient's error is 4u of its norm, in a random direction: |dx| times that, plus the h^2 term
        assert abs(got - quot) <= 4 * 2.0 ** -11 * float(g[i].double().norm()) * 4 + 1e-3 * abs(quot)


@pytest.mark.gpu
def test_graph_replay_and_other_stream():
    q, k, v, lam, do = inputs(2, 2, 2, 260, "bf16", 8)
    ref = fa.diff_fwd(q, k, v, lam, causal=True)
    gref = fa.diff_bwd(q, k, v, lam, ref[0], ref[2], do, ref[1], causal=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.diff_fwd(q, k, v, lam, causal=True, stream=s)
    g = fa.diff_bwd(q, k, v, lam, got[0], got[2], do, got[1], causal=True, stream=s)
    s.synchronize()
    for a, b in zip(list(got) + list(g[1:]), list(ref) + list(gref[1:])):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = fa.diff_fwd(q, k, v, lam, causal=True)
        cg = fa.diff_bwd(q, k, v, lam, c[0], c[2], do, c[1], causal=True)
    for _ in range(2):
        for t in list(c) + list(cg):
            t.zero_()
        graph.replay()
        for a, b in zip(list(c) + list(cg[1:]), list(ref) + list(gref[1:])):
            assert torch.equal(a, b)
    # repeats bit for bit (dQ apart)
    for _ in range(3):
        g2 = fa.diff_bwd(q, k, v, lam, ref[0], ref[2], do, ref[1], causal=True)
        for a, b in zip(g2[1:], gref[1:]):
            assert torch.equal(a, b)
