"""Rotary positions (fa_rope, fa_rope_frequencies).

CPU: the frequency rules against their formulas, struct layout, refusals
before any launch.  GPU: every dtype, both pair layouts, partial rotations,
strides, positions, in-place and transposed use against a 64-bit plain form.

Tolerance.  With exact cos and sin the kernel's error per output is one
rounding to the dtype (eps / 2 relative to the value) on top of float32 work:
cos and sin carry at most 2^-24 each from the fraction of a turn (absolute,
times pi) and a few units of sincospif, 2^-22 in all, and two products and one
sum add 2^-23.  So |error| <= eps(T)/2 |y| + 2^-21 m (|x0| + |x1|), plus half
the dtype's smallest step for float16 outputs near zero.
"""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from exact_io_aware_tiled_gb300 import _ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load()


def plain(x, pos, inv_freq, mscale, interleaved, backward):
    """Float64 CPU rotation of x [B,H,N,d]; pos [B,N]; inv_freq numpy [rot/2]. Also the error scale |x0| + |x1|."""
    x = x.detach().cpu().double()
    rot = 2 * len(inv_freq)
    a = pos.double()[:, None, :, None] * torch.from_numpy(np.asarray(inv_freq))
    c, s = torch.cos(a) * mscale, torch.sin(a) * mscale * (-1.0 if backward else 1.0)
    i0 = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    i1 = i0 + (1 if interleaved else rot // 2)
    y, mag = x.clone(), torch.zeros_like(x)
    x0, x1 = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = x0 * c - x1 * s, x1 * c + x0 * s
    mag[..., i0] = mag[..., i1] = abs(mscale) * (x0.abs() + x1.abs())
    return y, mag


def check(got, want, mag):
    eps = torch.finfo(got.dtype).eps
    tiny = torch.finfo(got.dtype).smallest_normal * eps / 2
    bound = eps / 2 * want.abs() * (1 + 2 ** -10) + 2.0 ** -21 * mag + tiny
    err = (got.cpu().double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp_min(1e-300)).max())


# ---- CPU ----------------------------------------------------------------------------------------------------
def test_frequencies_follow_their_formulas():
    rot = 64
    i = np.arange(rot // 2)
    plainf = 10000.0 ** (-2.0 * i / rot)
    f, m = fa.rope_frequencies(rot, device="cpu")
    assert m == 1.0 and np.allclose(f.numpy(), plainf, rtol=1e-14)
    f, m = fa.rope_frequencies(rot, scaling="linear", factor=4.0, device="cpu")
    assert m == 1.0 and np.allclose(f.numpy(), plainf / 4, rtol=1e-14)
    f, m = fa.rope_frequencies(rot, scaling="ntk", factor=4.0, device="cpu")
    assert m == 1.0 and f[0] == 1.0 and math.isclose(float(f[-1]), plainf[-1] / 4, rel_tol=1e-12)
    f, m = fa.rope_frequencies(rot, scaling="yarn", factor=8.0, original_len=4096, device="cpu")
    assert math.isclose(m, 0.1 * math.log(8.0) + 1.0, rel_tol=1e-6)
    turns = 4096 * plainf / (2 * math.pi)
    r = f.numpy() / plainf
    assert np.allclose(r[turns > 33], 1.0, rtol=1e-13) and np.allclose(r[turns < 0.7], 1 / 8, rtol=1e-12)
    assert np.all(np.diff(r) <= 1e-13) and r.min() >= 1 / 8 - 1e-13


@pytest.mark.parametrize("kw", [dict(rot=7), dict(rot=0), dict(rot=8, scaling="cubic"), dict(rot=8, base=1.0),
                                dict(rot=8, scaling="linear", factor=0.5), dict(rot=8, scaling="yarn", factor=2.0),
                                dict(rot=8, scaling="ntk", factor=float("nan")),
                                dict(rot=8, scaling="yarn", factor=2.0, original_len=64, beta_fast=1.0, beta_slow=2.0)])
def test_frequencies_refuse(kw):
    with pytest.raises((ValueError, fa.FAError)):
        fa.rope_frequencies(kw.pop("rot"), device="cpu", **kw)


def test_params_layout_matches_c(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    st = _ops.fa_rope_params
    prog = ['#include <stdio.h>', '#include <stddef.h>', '#include "fa.h"', 'int main(void){',
            'printf("%zu\\n", sizeof(fa_rope_params));']
    prog += ['printf("%%zu\\n", offsetof(fa_rope_params, %s));' % f for f, _ in st._fields_] + ['return 0;}']
    c = tmp_path / "l.c"
    c.write_text("\n".join(prog))
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(c), "-o", str(tmp_path / "l")], check=True)
    vals = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True).stdout.split()]
    assert vals == [ctypes.sizeof(st)] + [getattr(st, f).offset for f, _ in st._fields_]


def _params(**kw):
    p = _ops.fa_rope_params()
    p.B, p.H, p.H_kv, p.N, p.d, p.rot, p.dtype = 2, 3, 1, 10, 64, 64, 2
    for t, h in (("q", 3), ("k", 1), ("q_out", 3), ("k_out", 1)):
        setattr(p, t + "_stride_n", 64)
        setattr(p, t + "_stride_h", 640)
        setattr(p, t + "_stride_b", 640 * h)
    p.inv_freq, p.mscale = 1 << 22, 1.0
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("mut,code", [
    (dict(B=0), 1), (dict(N=0), 1), (dict(H_kv=-1), 1), (dict(dtype=5), 1),
    (dict(rot=63), 1), (dict(rot=0), 1), (dict(rot=66), 1),
    (dict(d=60, rot=60), 2), (dict(d=264), 2),
    (dict(mscale=float("inf")), 1), (dict(inv_freq=0), 1), (dict(inv_freq=(1 << 22) + 4), 3),
    (dict(positions=(1 << 22) + 2), 3), (dict(positions=(1 << 22) + 4, positions_i64=1), 3),
    (dict(q_stride_n=68), 3), (dict(k_out_stride_h=644), 1), (dict(q_out_stride_n=0), 1), (dict(q_out_stride_h=0), 1),
    (dict(B=1 << 20, N=1 << 12), 2),
])
def test_refusals_before_launch(mut, code):
    if mut == dict(k_out_stride_h=644):     # one head: its stride is not looked at; a second one's is
        mut = dict(H_kv=2, k_stride_h=640, k_out_stride_h=0)
    p = _params(**mut)
    f = _ops._fn("fa_rope", *([ctypes.c_void_p] * 6))
    a = 1 << 20
    assert f(ctypes.addressof(p), a, a + (1 << 16), a + (2 << 16), a + (3 << 16), None) == code


def test_null_misaligned_and_overlapping_pointers():
    f = _ops._fn("fa_rope", *([ctypes.c_void_p] * 6))
    a, b, c, d = (1 << 20), (2 << 20), (3 << 20), (4 << 20)
    p = _params()
    assert f(None, a, b, c, d, None) == 1
    assert f(ctypes.addressof(p), None, b, c, d, None) == 1
    assert f(ctypes.addressof(p), a, None, c, d, None) == 1
    assert f(ctypes.addressof(p), a + 8, b, c, d, None) == 3
    assert f(ctypes.addressof(p), a, b, c, d + 2, None) == 3
    q = _params(q_out_stride_n=128, q_out_stride_h=1280, q_out_stride_b=3840)
    assert f(ctypes.addressof(q), a, b, a, d, None) == 1       # same base, other strides


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    q = torch.zeros((1, 2, 3, 64))
    with pytest.raises(ValueError, match="CUDA"):
        fa.rope(q, inv_freq=torch.ones(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="4 dimensions"):
        fa.rope(q[0], inv_freq=torch.ones(32, dtype=torch.float64))


# ---- GPU ----------------------------------------------------------------------------------------------------
def _case(B, H, Hkv, N, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, H, N, d), generator=g).to(DT[dtype]).cuda()
    k = torch.randn((B, Hkv, N, d), generator=g).to(DT[dtype]).cuda()
    return q, k


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (64, 32), (128, 48), (64, 42), (64, 20), (64, 2), (96, 60),
                                   (8, 8), (256, 254)])
def test_layouts_and_partial_rotations(dtype, interleaved, d, rot):
    B, H, Hkv, N = 2, 5, 2, 37
    q, k = _case(B, H, Hkv, N, d, dtype, seed=d + rot)
    inv, m = fa.rope_frequencies(rot, scaling="yarn", factor=4.0, original_len=128)
    pos = torch.randint(0, 1000, (B, N))
    for back in (False, True):
        qo, ko = fa.rope(q, k, inv_freq=inv, positions=pos.cuda(), mscale=m, interleaved=interleaved, backward=back)
        for x, y in ((q, qo), (k, ko)):
            check(y, *plain(x, pos, inv.cpu().numpy(), m, interleaved, back))


@pytest.mark.gpu
@pytest.mark.parametrize("where", [0, 1, 131071, 2 ** 20 + 1, 2 ** 31 - 60, 2 ** 40 + 12345, -7])
def test_far_positions_keep_their_accuracy(where):
    # inverse frequencies with few bits, so that float64's own product on the CPU side is exact
    inv = torch.tensor([1.0, 0.40625, 0.03125, 1.0 / 1024], dtype=torch.float64, device="cuda")
    q, _ = _case(1, 2, 1, 50, 8, "f32", seed=3)
    pos = torch.arange(50)[None] + where
    got = fa.rope(q, inv_freq=inv, positions=pos.cuda())
    # p f mod 2 pi in exact integer / extended arithmetic
    from fractions import Fraction
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    x = q.cpu().double()
    want, mag = x.clone(), torch.zeros_like(x)
    for n in range(50):
        for i, f in enumerate(inv.cpu().tolist()):
            a = float((Fraction(int(pos[0, n])) * Fraction(f)) % two_pi)
            x0, x1 = x[0, :, n, i], x[0, :, n, i + 4]
            want[0, :, n, i] = x0 * math.cos(a) - x1 * math.sin(a)
            want[0, :, n, i + 4] = x1 * math.cos(a) + x0 * math.sin(a)
            mag[0, :, n, i] = mag[0, :, n, i + 4] = x0.abs() + x1.abs()
    # the float64 product f / 2 pi is off by 2^-52 relative: p f 2^-52 radians
    check(got, want, mag * (1 + 2.0 ** 21 * abs(where) * 2.0 ** -52))


@pytest.mark.gpu
def test_default_positions_start_and_shapes():
    q, k = _case(3, 4, 4, 21, 64, "bf16")
    inv, m = fa.rope_frequencies(64)
    pos = torch.arange(21) + 900
    a = fa.rope(q, k, inv_freq=inv, start=900)
    for variant in (pos.cuda(), pos.int().cuda(), pos[None].cuda(), pos[None].expand(3, 21).contiguous().cuda(),
                    pos[None].expand(3, 21).cuda(), torch.stack([pos, pos], 1).cuda()[:, 0]):
        b = fa.rope(q, k, inv_freq=inv, positions=variant)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(fa.rope(q, inv_freq=inv, start=900), a[0])
    check(a[0], *plain(q, pos[None].expand(3, 21), inv.cpu().numpy(), m, False, False))


@pytest.mark.gpu
@pytest.mark.parametrize("B,N", [(1, 1), (64, 1), (300, 1), (2, 3), (1, 5000)])
def test_single_tokens_and_long_rows(B, N):
    q, k = _case(B, 8, 2, N, 128, "bf16", seed=B)
    inv, m = fa.rope_frequencies(128, base=500000.0)
    pos = torch.randint(0, 200000, (B, N))
    qo, ko = fa.rope(q, k, inv_freq=inv, positions=pos.cuda())
    for x, y in ((q, qo), (k, ko)):
        check(y, *plain(x, pos, inv.cpu().numpy(), m, False, False))


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 42, 12])
def test_in_place_and_strided(interleaved, rot):
    B, H, N, d = 2, 6, 33, 64
    inv, _ = fa.rope_frequencies(rot)
    x = torch.randn((B, N, 3, H, d), device="cuda").bfloat16()       # a fused projection: [B, N, 3, H, d]
    q, k = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
    want = fa.rope(q.contiguous(), k.contiguous(), inv_freq=inv, interleaved=interleaved)
    got = fa.rope(q, k, inv_freq=inv, interleaved=interleaved)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    v = x[:, :, 2].clone()
    fa.rope(q, k, inv_freq=inv, interleaved=interleaved, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, :, 2], v)
    # a broadcast input (one head shown H times)
    one = torch.randn((B, 1, N, d), device="cuda").bfloat16()
    a = fa.rope(one.expand(B, H, N, d), inv_freq=inv, interleaved=interleaved,
                out=torch.empty((B, H, N, d), device="cuda", dtype=torch.bfloat16))
    b = fa.rope(one, inv_freq=inv, interleaved=interleaved)
    assert torch.equal(a, b.expand(B, H, N, d))


@pytest.mark.gpu
def test_transposed_rotation_is_the_gradient():
    q, _ = _case(2, 3, 1, 19, 64, "f32", seed=9)
    inv, m = fa.rope_frequencies(48, scaling="yarn", factor=2.0, original_len=64)
    dy = torch.randn_like(q)
    # <R x, dy> = <x, R^T dy> for the linear map R; float32 sums of n terms of size 1: n^0.5 2^-23 of the norm product
    lhs = (fa.rope(q, inv_freq=inv, mscale=m).double() * dy.double()).sum()
    rhs = (q.double() * fa.rope(dy, inv_freq=inv, mscale=m, backward=True).double()).sum()
    assert abs(float(lhs - rhs)) <= 2.0 ** -20 * float(q.double().norm() * dy.double().norm())
    # a difference quotient along one direction
    h = 2.0 ** -6
    dx = torch.randn_like(q)
    up, dn = (fa.rope(q + s * h * dx, inv_freq=inv, mscale=m).double() for s in (1, -1))
    quot = (((up - dn) / (2 * h)) * dy.double()).sum()
    grad = (dx.double() * fa.rope(dy, inv_freq=inv, mscale=m, backward=True).double()).sum()
    assert abs(float(quot - grad)) <= 2.0 ** -20 / h * float((q.double().norm() + dx.double().norm()) * dy.double().norm())


@pytest.mark.gpu
def test_masked_rows_keep_nan_to_themselves():
    q, _ = _case(1, 2, 1, 8, 64, "bf16")
    inv, _ = fa.rope_frequencies(32)
    want = fa.rope(q, inv_freq=inv)
    q2 = q.clone()
    q2[0, 1, 3, 40] = float("nan")     # a copied column
    q2[0, 0, 5, 2] = float("inf")      # one pair: columns 2 and 18
    got = fa.rope(q2, inv_freq=inv)
    bad = torch.zeros_like(q, dtype=torch.bool)
    bad[0, 1, 3, 40] = bad[0, 0, 5, 2] = bad[0, 0, 5, 18] = True
    assert torch.equal(got[~bad], want[~bad]) and bool(got[0, 1, 3, 40].isnan())


@pytest.mark.gpu
def test_other_stream_and_graph_replay():
    q, k = _case(4, 4, 2, 64, 64, "bf16")
    inv, _ = fa.rope_frequencies(64)
    want = fa.rope(q, k, inv_freq=inv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.rope(q, k, inv_freq=inv, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qs, pos = q.clone(), torch.arange(64, device="cuda")
    out = torch.empty_like(q)
    fa.rope(qs, inv_freq=inv, positions=pos, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.rope(qs, inv_freq=inv, positions=pos, out=out)
    for shift in (0, 1000):
        pos.copy_(torch.arange(64, device="cuda") + shift)
        qs.copy_(torch.randn_like(q.float()).bfloat16())
        g.replay()
        assert torch.equal(out, fa.rope(qs, inv_freq=inv, start=shift))
    with pytest.raises(ValueError):
        fa.rope(q, k, inv_freq=inv.float())
    with pytest.raises(ValueError):
        fa.rope(q, k[:, :, :5], inv_freq=inv)
    with pytest.raises(ValueError):
        fa.rope(q, inv_freq=inv, positions=pos[:5])
