"""Norms of q and k with the rotation (fa_norm_rope, fa_norm_rope_bwd).

CPU: struct layout, refusals, the 64-bit form's gradient against differences.  GPU: every dtype over head dimensions,
rotated parts, pair layouts, lengths and strides against that form.

Tolerances, u = eps / 2 of the dtype.  z = w x r is off by 2^-20 relative in float32: 21 additions of squares and
rsqrtf's 2 steps halve to 12 steps of 2^-24, three products follow; sin and cos by 2^-22 each.  So an output is off by
u |y| + 2^-19 m (|z0| + |z1|) over the pair it is turned from (2^-20 + 2^-22 + products), dx by
u |dx| + 2^-17 r (|g| + |h| mean(|g| |h|)) with |g| such a pair sum (the mean's sum has 21 additions again), dw by
2^-16 of the sum of its terms' magnitudes: up to 100 additions in a row of 2^-24 (a thread's rows, a CTA's groups, the
CTAs) and 2^-18 of the terms.  Float16 results below its normal range are off by half of 2^-24 besides.
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
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load()


# ---- the 64-bit form -------------------------------------------------------------------------------------------
def turned(z, pos, inv, m, inter, back=False):
    """z rotated by pos [B or 1, 1, N], in float64; the pair sums |z0| + |z1| that bound its rounding."""
    rot = 0 if inv is None else 2 * len(inv)
    if rot == 0:
        return z, z.abs()
    a = pos.double()[..., None] * inv.double()
    c, s = torch.cos(a) * m, torch.sin(a) * m * (-1 if back else 1)
    y, mag = z.clone(), z.abs()
    i0 = slice(0, rot, 2) if inter else slice(0, rot // 2)
    i1 = slice(1, rot, 2) if inter else slice(rot // 2, rot)
    z0, z1 = z[..., i0], z[..., i1]
    y[..., i0], y[..., i1] = z0 * c - z1 * s, z1 * c + z0 * s
    mag[..., i0] = mag[..., i1] = (z0.abs() + z1.abs()) * abs(m)
    return y, mag


def plain(x, w, dy, eps, pos, inv, m=1.0, inter=False):
    """Float64: (y, mag) or, with dy, (dx, mag, dw, mag)."""
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    h = x * r
    if dy is None:
        return turned(w * h, pos, inv, m, inter)
    dz, mag = turned(dy.double(), pos, inv, m, inter, True)
    g, gm = w * dz, w.abs() * mag
    dx = r * (g - h * (g * h).mean(-1, keepdim=True))
    dxm = r * (gm + h.abs() * (gm * h.abs()).mean(-1, keepdim=True))
    return dx, dxm, (dz * h).sum((0, 1, 2)), (mag * h.abs()).sum((0, 1, 2))


def near(got, want, mag, dtype, steps):
    u = torch.finfo(DT[dtype]).eps / 2
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    err, bound = (got.double() - want).abs(), u * want.abs() + 2.0 ** steps * mag + tiny
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())


def test_the_form_against_differences():
    g = torch.Generator().manual_seed(1)
    x, dy, ux = (torch.randn(2, 3, 5, 16, generator=g, dtype=torch.float64) for _ in range(3))
    w, uw = (torch.randn(16, generator=g, dtype=torch.float64) for _ in range(2))
    inv, pos = torch.rand(6, generator=g, dtype=torch.float64), torch.arange(5)[None, None]
    for inter in (False, True):
        dx, _, dw, _ = plain(x, w, dy, 1e-3, pos, inv, 1.3, inter)
        for got, mx, mw in (((dx * ux).sum(), ux, 0 * uw), ((dw * uw).sum(), 0 * ux, uw)):
            e = 1e-6
            up, dn = (plain(x + s * e * mx, w + s * e * mw, None, 1e-3, pos, inv, 1.3, inter)[0] for s in (1, -1))
            assert abs(float(((up - dn) * dy).sum()) / (2 * e) - float(got)) < 1e-7


# ---- CPU -------------------------------------------------------------------------------------------------------
def test_params_layout_matches_c(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    st = _ops.fa_norm_rope_params
    prog = ['#include <stdio.h>', '#include <stddef.h>', '#include "fa.h"', 'int main(void){',
            'printf("%zu\\n", sizeof(fa_norm_rope_params));']
    prog += ['printf("%%zu\\n", offsetof(fa_norm_rope_params, %s));' % f for f, _ in st._fields_] + ['return 0;}']
    c = tmp_path / "l.c"
    c.write_text("\n".join(prog))
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(c), "-o", str(tmp_path / "l")], check=True)
    vals = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True).stdout.split()]
    assert vals == [ctypes.sizeof(st)] + [getattr(st, f).offset for f, _ in st._fields_]


def _params(**kw):
    p = _ops.fa_norm_rope_params()
    p.B, p.H, p.H_kv, p.N, p.d, p.rot, p.dtype = 2, 4, 2, 100, 64, 32, 2
    for t, h in (("q", 4), ("q_out", 4), ("dq", 4), ("k", 2), ("k_out", 2), ("dk", 2)):
        for x, v in (("n", 64), ("h", 6400), ("b", 6400 * h)):
            setattr(p, "%s_stride_%s" % (t, x), v)
    p.inv_freq, p.mscale, p.eps = 1 << 22, 1.0, 1e-6
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _fwd(p, ptrs=None):
    f = _ops._fn("fa_norm_rope", *([ctypes.c_void_p] * 8))
    x = [1 << 20, 1 << 21, 1 << 23, 1 << 23, 1 << 24, 1 << 25]
    for i, v in (ptrs or {}).items():
        x[i] = v
    return f(None if p is None else ctypes.addressof(p), *x, None)


def _bwd(p, ptrs=None, ws=1 << 40, ws_ptr=1 << 27):
    f = _ops._fn("fa_norm_rope_bwd", *([ctypes.c_void_p] * 12), ctypes.c_size_t, ctypes.c_void_p)
    x = [1 << 20, 1 << 21, 1 << 22, 3 << 21, 1 << 23, 1 << 23, 1 << 24, 1 << 25, 1 << 26, 1 << 26]
    for i, v in (ptrs or {}).items():
        x[i] = v
    return f(None if p is None else ctypes.addressof(p), *x, ws_ptr, ws, None)


@pytest.mark.parametrize("mut,code", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(H_kv=-1), 1), (dict(N=0), 1), (dict(d=0), 1), (dict(dtype=3), 1),
    (dict(rot=-2), 1), (dict(rot=66), 1), (dict(rot=31), 1), (dict(d=60, rot=32), 2), (dict(d=264), 2),
    (dict(mscale=math.inf), 1), (dict(eps=0.0), 1), (dict(eps=math.nan), 1), (dict(inv_freq=0), 1),
    (dict(inv_freq=(1 << 22) + 4), 3), (dict(positions=(1 << 22) + 2), 3),
    (dict(positions=(1 << 22) + 4, positions_i64=1), 3), (dict(q_stride_n=68), 3), (dict(k_out_stride_n=32), 1),
    (dict(q_out_stride_b=0), 1), (dict(k_stride_h=-64), 1), (dict(B=1 << 20, N=1 << 10), 2),
])
def test_refusals_before_launch(mut, code):
    assert _fwd(_params(**mut)) == code
    assert _bwd(_params(**mut)) == code


def test_pointers_and_workspace():
    assert _fwd(None) == 1 and _bwd(None) == 1
    for i in (0, 1, 4, 5):
        assert _fwd(_params(), {i: None}) == 1
        assert _fwd(_params(), {i: (1 << 20) + 8}) == 3
    for i in (2, 3):
        assert _fwd(_params(), {i: (1 << 20) + 2}) == 3
    for i in (0, 1, 2, 3, 6, 7):
        assert _bwd(_params(), {i: None}) == 1
        assert _bwd(_params(), {i: (1 << 20) + 8}) == 3
    for i in (4, 5, 8, 9):
        assert _bwd(_params(), {i: (1 << 20) + 2}) == 3
    # an output in its input's place, with other strides
    assert _fwd(_params(q_out_stride_n=128, q_out_stride_h=12800, q_out_stride_b=51200), {4: 1 << 20}) == 1
    assert _bwd(_params(dk_stride_n=128, dk_stride_h=12800, dk_stride_b=25600), {7: 3 << 21}) == 1
    size = _ops._fn("fa_norm_rope_bwd_workspace_size", ctypes.c_void_p, restype=ctypes.c_size_t)
    p = _params()
    need = size(ctypes.addressof(p))
    assert need > 256 and size(None) == 256
    assert _bwd(p, ws=need - 1) == 4 and _bwd(p, ws_ptr=None) == 4 and _bwd(p, ws_ptr=(1 << 27) + 8) == 4


def test_binding_refuses():
    q = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.norm_rope(q)
    with pytest.raises(ValueError, match="4 dimensions"):
        fa.norm_rope(q[0])


# ---- GPU -------------------------------------------------------------------------------------------------------
def make(B, H, Hkv, N, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k, dq, dk = (r(B, h, N, d).to(DT[dtype]) for h in (H, Hkv, H, Hkv))
    return q, k, dq, dk, 1 + 0.3 * r(d), 1 + 0.3 * r(d)


def freqs(rot):
    return None if rot == 0 else fa.rope_frequencies(rot)[0]


def check_both(x, dtype, inv, pos=None, start=0, m=1.0, inter=False, eps=1e-6, weights=True):
    q, k, dq, dk, wq, wk = x
    if not weights:
        wq = wk = None
    B, _, N, _ = q.shape
    p = torch.arange(N, device="cuda") + start if pos is None else pos
    p = (p[None] if p.dim() == 1 else p)[:, None]
    kw = dict(q_weight=wq, k_weight=wk, eps=eps, inv_freq=inv, positions=pos, start=start, mscale=m, interleaved=inter)
    keep = [t.clone() for t in (q, k, dq, dk)]
    yq, yk = fa.norm_rope(q, k, **kw)
    gq, gk, gwq, gwk = fa.norm_rope_bwd(q, k, dq, dk, **kw)
    assert all(torch.equal(a, b) for a, b in zip(keep, (q, k, dq, dk)))
    for t, w, dy, y, gx, gw in ((q, wq, dq, yq, gq, gwq), (k, wk, dk, yk, gk, gwk)):
        near(y, *plain(t, w, None, eps, p, inv, m, inter), dtype, -19)
        dx, dxm, dw, dwm = plain(t, w, dy, eps, p, inv, m, inter)
        near(gx, dx, dxm, dtype, -17)
        assert (gw is None) == (w is None)
        if w is not None:
            assert bool(((gw.double() - dw).abs() <= 2.0 ** -16 * dwm).all())
    return yq, yk, gq, gk, gwq, gwk


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 32), (64, 48), (64, 2), (64, 0), (64, 30), (128, 128), (128, 96),
                                   (128, 46), (256, 256), (256, 254), (8, 8), (8, 2), (40, 16), (200, 64), (96, 96)])
def test_head_dimensions_and_rotated_parts(dtype, inter, d, rot):
    check_both(make(2, 3, 2, 37, d, dtype, d + rot), dtype, freqs(rot), start=5, inter=inter)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hkv,N", [(1, 1, 1, 1), (64, 16, 4, 1), (1, 16, 1, 2), (3, 5, 5, 7), (2, 9, 3, 129),
                                       (1, 32, 8, 515), (5, 2, 1, 1023), (1, 1, 1, 20001)])
def test_lengths_and_heads(dtype, B, H, Hkv, N):
    check_both(make(B, H, Hkv, N, 64, dtype, N), dtype, freqs(64))
    check_both(make(B, H, Hkv, N, 128, dtype, N), dtype, freqs(64), inter=True)


@gpu
@pytest.mark.parametrize("wide", [False, True])
def test_positions(wide):
    x = make(3, 4, 2, 50, 64, "f32", 3)
    inv, m = fa.rope_frequencies(64, scaling="yarn", factor=8.0, original_len=64)
    t = torch.int64 if wide else torch.int32
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, 50), device="cuda", dtype=torch.int64).to(t)
    # the exact fraction of a turn against float64's own 2^-53 of 2^31: 2^-22 radians
    check_both(x, "f32", inv, pos=pos // 16, m=m)
    check_both(x, "f32", inv, pos=pos[0] // 16, m=m)
    check_both(x, "f32", inv, pos=pos[:1] // 16, m=m)
    check_both(x, "f32", inv, start=-1000000, m=m)
    wide_pos = (torch.arange(100, device="cuda", dtype=t) * 3)[::2]
    check_both(x, "f32", inv, pos=wide_pos, m=m)


@gpu
def test_without_weights_and_without_k():
    x = make(2, 4, 2, 33, 64, "bf16", 4)
    inv = freqs(64)
    check_both(x, "bf16", inv, weights=False)
    q, k, dq, dk, wq, wk = x
    yq, yk = fa.norm_rope(q, k, q_weight=wq, inv_freq=inv)
    assert torch.equal(fa.norm_rope(q, q_weight=wq, inv_freq=inv), yq)
    a = fa.norm_rope_bwd(q, k, dq, dk, q_weight=wq, inv_freq=inv)
    b = fa.norm_rope_bwd(q, None, dq, q_weight=wq, inv_freq=inv)
    assert a[3] is None and b[1] is None and b[3] is None
    assert torch.equal(a[0], b[0])
    near(b[2], *plain(q, wq, dq, 1e-6, torch.arange(33, device="cuda")[None, None], inv)[2:], "f32", -16)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layouts(dtype):
    # [B, N, H, d] memory, slices of a fused projection, broadcast inputs and gradients, in place
    q, k, dq, dk, wq, wk = make(2, 4, 2, 41, 64, dtype, 6)
    inv = freqs(48)
    kw = dict(q_weight=wq, k_weight=wk, inv_freq=inv)
    want, grads = fa.norm_rope(q, k, **kw), fa.norm_rope_bwd(q, k, dq, dk, **kw)
    t = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    got = fa.norm_rope(t(q), t(k), **kw)
    assert got[0].stride() == t(q).stride()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(grads, fa.norm_rope_bwd(t(q), k, dq, t(dk), **kw)))
    fused = torch.randn(2, 41, 8, 64, device="cuda").to(DT[dtype])
    fq, fk = fused[:, :, :4].transpose(1, 2), fused[:, :, 4:6].transpose(1, 2)
    keep = fused.clone()
    want_f = fa.norm_rope(fq.contiguous(), fk.contiguous(), **kw)
    fa.norm_rope(fq, fk, out=(fq, fk), **kw)
    assert torch.equal(fq, want_f[0]) and torch.equal(fk, want_f[1]) and torch.equal(fused[:, :, 6:], keep[:, :, 6:])
    one, g1 = q[:, :1].expand(2, 4, 41, 64), dq[:, :, :1].expand(2, 4, 41, 64)
    assert all(torch.equal(a, b) for a, b in zip(
        fa.norm_rope_bwd(one, k, g1, dk, out=(torch.empty_like(q), torch.empty_like(k)), **kw),
        fa.norm_rope_bwd(one.contiguous(), k, g1.contiguous(), dk, **kw)))
    assert torch.equal(fa.norm_rope(one, out=torch.empty_like(q), inv_freq=inv), fa.norm_rope(one.contiguous(), inv_freq=inv))
    # the gradients' own memory, and x's
    for out in ((dq.clone(), dk.clone()), (q.clone(), k.clone())):
        if torch.equal(out[0], dq):
            got = fa.norm_rope_bwd(q, k, out[0], out[1], out=out, **kw)
        else:
            got = fa.norm_rope_bwd(out[0], out[1], dq, dk, out=out, **kw)
        assert all(torch.equal(a, b) for a, b in zip(grads, got))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_zero_small_and_nonfinite_rows(dtype):
    q, k, dq, dk, wq, wk = make(1, 2, 1, 9, 64, dtype, 7)
    q[0, 0, 0] = 0
    q[0, 0, 1] = 0
    q[0, 0, 1, 5] = 2.0 ** -14
    check_both((q, k, dq, dk, wq, wk), dtype, freqs(64))
    want = fa.norm_rope(q, k, q_weight=wq, inv_freq=freqs(64))[0]
    bad = q.clone()
    bad[0, 1, 3, 7] = math.nan
    got = fa.norm_rope(bad, k, q_weight=wq, inv_freq=freqs(64))[0]
    assert bool(got[0, 1, 3].isnan().all())
    got[0, 1, 3] = want[0, 1, 3]
    assert torch.equal(got, want)
    gx, _, dw, dwk = fa.norm_rope_bwd(bad, k, dq, dk, q_weight=wq, k_weight=wk, inv_freq=freqs(64))
    assert bool(gx[0, 1, 3].isnan().all()) and int(gx.isnan().sum()) == 64
    assert bool(dw.isnan().all()) and not bool(dwk.isnan().any())


@gpu
def test_repeats_streams_and_graphs():
    x = make(4, 8, 2, 700, 64, "bf16", 8)
    q, k, dq, dk, wq, wk = x
    inv = freqs(64)
    kw = dict(q_weight=wq, k_weight=wk, inv_freq=inv)

    def both(**more):
        y = fa.norm_rope(q, k, **kw, **more)
        return list(y) + list(fa.norm_rope_bwd(q, k, dq, dk, **kw, **more))

    want = both()
    assert all(torch.equal(a, b) for a, b in zip(want, both()))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    side = both(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, side))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for t, c in ((q, 1), (dk, 2)):
        t.mul_(0.5 * c)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, both()))
    # two calls in flight at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [both(stream=st) for st in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(out, o))


@gpu
def test_offsets_past_32_bits():
    # two heads 2^32 elements apart in a buffer of float16
    base = torch.empty(2 ** 32 + 4096, device="cuda", dtype=torch.float16)
    q = base.as_strided((1, 2, 16, 64), (2 ** 32 + 2048, 2 ** 32, 64, 1))
    x = make(1, 2, 1, 16, 64, "f16", 9)
    q.copy_(x[0])
    kw = dict(q_weight=x[4], inv_freq=freqs(64))
    want = fa.norm_rope(x[0], **kw)
    assert torch.equal(fa.norm_rope(q, out=torch.empty_like(x[0]), **kw), want)
    grads = fa.norm_rope_bwd(x[0], None, x[2], **kw)
    got = fa.norm_rope_bwd(q, None, x[2], out=q, **kw)
    assert torch.equal(got[0], grads[0]) and torch.equal(got[2], grads[2])


@gpu
def test_refusals_of_the_binding():
    q, k, dq, dk, wq, wk = make(1, 4, 2, 8, 64, "bf16")
    inv = freqs(64)
    for bad in (dict(q_weight=wq.half()), dict(q_weight=wq[:32]), dict(q_weight=wq.cpu()), dict(inv_freq=inv.float()),
                dict(positions=torch.arange(7, device="cuda")), dict(positions=torch.arange(8.0, device="cuda")),
                dict(out=(q, q)), dict(out=(q.float(), k))):
        with pytest.raises(ValueError):
            fa.norm_rope(q, k, **bad)
    with pytest.raises(ValueError):
        fa.norm_rope(q, k_weight=wk)
    with pytest.raises(ValueError):
        fa.norm_rope_bwd(q, k, dq)
    with pytest.raises(ValueError):
        fa.norm_rope_bwd(q, k, dq, dq)
    for bad in (dict(eps=0.0), dict(mscale=math.inf), dict(inv_freq=fa.rope_frequencies(66)[0])):
        with pytest.raises(fa.FAError):
            fa.norm_rope(q, k, **bad)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_zeros_and_the_smallest_eps(dtype):
    # 1 / sqrt(eps) = 2^70, whose square passes float32: a row of zeros has the gradient 2^70 w R^T dy, not NaN
    x = make(2, 3, 1, 9, 64, dtype, 21)
    for t in x[:2]:
        t[:, :, ::2] = 0
    check_both(x, dtype, freqs(64), eps=2.0 ** -140)


@gpu
@pytest.mark.parametrize("dtype,d,rot,inter,rows", [("bf16", 256, 0, False, 3000), ("f16", 128, 64, True, 3000),
                                                    ("bf16", 64, 46, False, 3000), ("f32", 128, 128, False, 1500),
                                                    ("bf16", 64, 64, False, 100), ("f16", 8, 8, False, 700)])
def test_weight_gradients_of_many_rows(dtype, d, rot, inter, rows):
    # `rows` equal rows a thread, so that all terms of a column have one sign and every addition errs the same way
    lanes = (d + 8) // 16 if inter else (d - rot // 2) // 8 if rot % 16 == 0 else d // 8
    per = 128 >> (lanes - 1).bit_length()
    N = -(-rows * 456 * per // 16)
    g = torch.Generator(device="cuda").manual_seed(31)
    x, dy = (torch.randn(1, 1, 1, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    w = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    pos = torch.full((1,), 77, device="cuda", dtype=torch.int32).expand(N)
    many = lambda t: t.expand(1, 16, N, d)  # noqa: E731
    out = torch.empty(1, 16, N, d, device="cuda", dtype=DT[dtype])
    got = fa.norm_rope_bwd(many(x), None, many(dy), q_weight=w, inv_freq=freqs(rot), positions=pos, interleaved=inter, out=out)
    p = torch.full((1, 1, 1), 77, device="cuda")
    dx, dxm, dw, dwm = plain(x, w, dy, 1e-6, p, freqs(rot), 1.0, inter)
    near(got[0][:, :, ::N - 1], dx, dxm, dtype, -17)
    M = 16 * N
    assert bool(((got[2].double() - M * dw).abs() <= 2.0 ** -16 * M * dwm).all()), \
        float(((got[2].double() - M * dw).abs() / (M * dwm)).max() * 2 ** 16)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (46, False), (0, False)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_an_infinity_in_a_row(dtype, rot, inter, bad):
    # r = 0: the infinity and its partner in the rotation become NaN, the row's others 0; backward the whole row and the
    # infinity's column of the weights' gradient are NaN; no other row changes
    q, k, dq, dk, wq, wk = make(1, 3, 1, 9, 64, dtype, 41)
    kw = dict(q_weight=wq, inv_freq=freqs(rot), interleaved=inter)
    want, (gwant, _, dwant, _) = fa.norm_rope(q, **kw), fa.norm_rope_bwd(q, None, dq, **kw)
    for c in (0, 5, 22, 23, 45, 46, 63):
        x = q.clone()
        x[0, 1, 4, c] = bad
        pair = [c]
        if c < rot:
            pair.append(c ^ 1 if inter else (c + rot // 2) % rot)
        y = fa.norm_rope(x, **kw)
        assert sorted(y[0, 1, 4].isnan().nonzero().flatten().tolist()) == sorted(pair)
        assert int((y[0, 1, 4] == 0).sum()) == 64 - len(pair)
        dx, _, dw, _ = fa.norm_rope_bwd(x, None, dq, **kw)
        assert bool(dx[0, 1, 4].isnan().all())
        assert dw.isnan().nonzero().flatten().tolist() == [c]
        for got, ref in ((y, want), (dx, gwant)):
            got[0, 1, 4] = ref[0, 1, 4]
            assert torch.equal(got, ref)
