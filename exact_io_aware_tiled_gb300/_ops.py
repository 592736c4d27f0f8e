"""ctypes binding of the operators around the attention passes (include/fa.h,
ABI 1.4): rotary positions, differential attention, attention over a shared
prefix.

As in ``_lib``: argument checks, output and workspace allocation with torch,
raw pointers and the stream; the computation runs in ``libfa_gb300.so``.
A call runs on the device of its tensors, on ``stream`` or that device's
current stream.  With ``stream`` given, outputs and workspace are allocated
on that stream, and small conversions of index arguments run on it too.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from ._lib import DTYPE_CODE, FA_OK, FAError, load

ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class fa_rope_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "H", "H_kv", "N", "d", "rot", "dtype", "interleaved", "backward",
                                     "positions_i64")] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("q", "k", "q_out", "k_out") for x in "bhn"] +
                [("positions", _vp), ("pos_stride_b", _i64), ("pos_stride_n", _i64), ("start", _i64),
                 ("inv_freq", _vp), ("mscale", _f32)])


_typed = {}


def _fn(name, *argtypes, restype=ctypes.c_int):
    """The library's function `name` with its argument types set (once)."""
    f = _typed.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes, f.restype = list(argtypes), restype
        _typed[name] = f
    return f


@contextlib.contextmanager
def _entered(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


class _Plain:
    """_entered for the usual case (the tensors' device is current, no stream given), without its cost."""

    def __init__(self, device):
        self.device = device

    def __enter__(self):
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        return False


def _on(device, stream):
    """Context that makes the tensors' device (and the given stream) current; yields the raw stream."""
    if stream is not None:
        if stream.device != device:
            raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
        return _entered(device, stream)
    if torch.cuda.current_device() != device.index:
        return _entered(device, None)
    return _Plain(device)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _check4(t, name, device=None, dtype=None):
    if t.dim() != 4:
        raise ValueError("%s must have 4 dimensions, got shape %s" % (name, tuple(t.shape)))
    _check_place(t, name, device, dtype)
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError("%s: the last dimension must be contiguous (stride 1), got strides %s" % (name, t.stride()))


def _check_place(t, name, device=None, dtype=None):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if dtype is None:
        if t.dtype not in DTYPE_CODE:
            raise ValueError("unsupported dtype %s of %s" % (t.dtype, name))
    elif t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))


def _check_out(t, like, name):
    if t.shape != like.shape:
        raise ValueError("out %s must have shape %s, got %s" % (name, tuple(like.shape), tuple(t.shape)))
    _check4(t, "out " + name, like.device, like.dtype)


def rope_frequencies(rot, *, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0,
                     device="cuda"):
    """(inv_freq, mscale) of a rotation of ``rot`` columns, for :func:`rope`.

    inv_freq is a float64 tensor [rot/2] on ``device``; mscale the factor on
    cos and sin.  ``scaling``: "none", "linear" (positions interpolated by
    ``factor``), "ntk" (base stretched so that the slowest pair is slowed by
    ``factor``) or "yarn" (per pair, by how often it turns within
    ``original_len`` positions)."""
    if scaling not in ROPE_SCALING:
        raise ValueError("scaling must be one of %s, got %r" % (sorted(ROPE_SCALING), scaling))
    rot = int(rot)
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2, got %d" % rot)
    buf = (ctypes.c_double * (rot // 2))()
    m = _f32()
    dbl = ctypes.c_double
    f = _fn("fa_rope_frequencies", _i32, dbl, _i32, dbl, _i64, dbl, dbl, _vp, _vp)
    st = f(rot, float(base), ROPE_SCALING[scaling], float(factor), int(original_len), float(beta_fast), float(beta_slow),
           ctypes.addressof(buf), ctypes.addressof(m))
    if st != FA_OK:
        raise FAError(st, "fa_rope_frequencies")
    return torch.tensor(list(buf), dtype=torch.float64).to(device), float(m.value)


def rope(q, k=None, *, inv_freq, positions=None, start=0, mscale=1.0, interleaved=False, backward=False, out=None,
         stream=None):
    """q and k rotated by their positions (fa_rope), as (q_out, k_out); q_out alone without k.

    q [B,H,N,d], k [B,H_kv,N,d].  ``inv_freq`` (float64 [rot/2], see
    :func:`rope_frequencies`) sets how many leading columns turn; the others
    are copied.  ``positions``: int32 / int64 tensor [N], [1,N] or [B,N];
    None means start + n.  ``backward`` applies the transposed rotation: give
    it dQ and dK to get the gradients of the unrotated q and k.  ``out`` =
    (q_out, k_out), or q_out without k, may be the inputs themselves."""
    _check4(q, "q")
    B, H, N, d = q.shape
    if k is not None:
        _check4(k, "k", q.device, q.dtype)
        if (k.shape[0], k.shape[2], k.shape[3]) != (B, N, d):
            raise ValueError("k must be [B, H_kv, N, d] with the B, N, d of q")
    if inv_freq.dim() != 1 or inv_freq.dtype != torch.float64 or inv_freq.device != q.device or \
            not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 tensor [rot/2] on q's device")
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64) or positions.device != q.device:
            raise ValueError("positions must be an int32 or int64 tensor on q's device")
        if positions.dim() == 1:
            positions = positions[None]
        if positions.dim() != 2 or positions.shape[1] != N or positions.shape[0] not in (1, B):
            raise ValueError("positions must have shape [N], [1, N] or [B, N]")
    p = fa_rope_params()
    p.B, p.H, p.N, p.d, p.rot = B, H, N, d, 2 * inv_freq.shape[0]
    p.H_kv = 0 if k is None else k.shape[1]
    p.dtype = DTYPE_CODE[q.dtype]
    p.interleaved, p.backward = bool(interleaved), bool(backward)
    p.mscale, p.start = float(mscale), int(start)
    p.inv_freq = inv_freq.data_ptr()
    if positions is not None:
        p.positions, p.positions_i64 = positions.data_ptr(), positions.dtype == torch.int64
        p.pos_stride_b = positions.stride(0) if positions.shape[0] > 1 else 0
        p.pos_stride_n = positions.stride(1)
    with _on(q.device, stream) as raw:
        if out is None:
            qo = torch.empty_like(q)
            ko = None if k is None else torch.empty_like(k)
        else:
            qo, ko = (out, None) if k is None else out
            _check_out(qo, q, "q")
            if k is not None:
                _check_out(ko, k, "k")
        p.q_stride_b, p.q_stride_h, p.q_stride_n = q.stride()[:3]
        p.q_out_stride_b, p.q_out_stride_h, p.q_out_stride_n = qo.stride()[:3]
        if k is not None:
            p.k_stride_b, p.k_stride_h, p.k_stride_n = k.stride()[:3]
            p.k_out_stride_b, p.k_out_stride_h, p.k_out_stride_n = ko.stride()[:3]
        f = _fn("fa_rope", _vp, _vp, _vp, _vp, _vp, _vp)
        st = f(ctypes.addressof(p), _ptr(q), _ptr(k), _ptr(qo), _ptr(ko), raw)
    if st != FA_OK:
        raise FAError(st, "fa_rope")
    return qo if k is None else (qo, ko)


class fa_diff_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "H", "H_kv", "N", "d", "dtype", "causal", "window")] +
                [("scale", _f32), ("seqlens_k", _vp), ("lam", _vp)] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("q", "k", "v", "o", "do") for x in "bhn"])


def _set_strides(p, name, t):
    s = t.stride()
    setattr(p, name + "_stride_b", s[0])
    setattr(p, name + "_stride_h", s[1])
    setattr(p, name + "_stride_n", s[2])


def _lens(seqlens, B, device, name="seqlens_k"):
    """int32 [B] lengths on `device` (converted on the current stream where they are something else)."""
    if seqlens is None:
        return None
    if tuple(seqlens.shape) != (B,):
        raise ValueError("%s must have shape [B] = [%d]" % (name, B))
    if seqlens.dtype.is_floating_point or seqlens.dtype == torch.bool:
        raise ValueError("%s must hold whole numbers" % name)
    return seqlens.to(device=device, dtype=torch.int32).contiguous()


def _need_workspace(workspace, size, device):
    if workspace is None:
        return torch.empty(size, device=device, dtype=torch.uint8)
    if workspace.dtype != torch.uint8 or workspace.numel() < size or workspace.device != device or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor of >= %d bytes on %s" % (size, device))
    return workspace


def _diff_params(q, k, v, lam, causal, window, scale):
    _check4(q, "q")
    if q.shape[3] != 64 or q.shape[1] % 2:
        raise ValueError("q must be [B, 2H, N, 64] (the two maps of head pair h in heads 2h, 2h + 1)")
    _check4(k, "k", q.device, q.dtype)
    _check4(v, "v", q.device, q.dtype)
    B, H2, N, d = q.shape
    H, Hkv = H2 // 2, v.shape[1]
    if tuple(k.shape) != (B, 2 * Hkv, N, d) or tuple(v.shape) != (B, Hkv, N, 2 * d):
        raise ValueError("k must be [B, 2 H_kv, N, 64] and v [B, H_kv, N, 128] with the B, N of q")
    if Hkv < 1 or H % Hkv:
        raise ValueError("the number of query head pairs must be a multiple of the number of K/V pairs")
    if tuple(lam.shape) != (H,) or lam.dtype != torch.float32 or lam.device != q.device or not lam.is_contiguous():
        raise ValueError("lam must be a contiguous float32 tensor [H] on q's device")
    p = fa_diff_params()
    p.B, p.H, p.H_kv, p.N, p.d, p.dtype = B, H, Hkv, N, d, DTYPE_CODE[q.dtype]
    p.causal, p.window = bool(causal), int(window)
    p.scale = 0.0 if scale is None else float(scale)
    p.lam = lam.data_ptr()
    for n, t in (("q", q), ("k", k), ("v", v)):
        _set_strides(p, n, t)
    return p


def diff_fwd(q, k, v, lam, *, causal=False, seqlens_k=None, window=0, scale=None, need_o2=True, out=None,
             workspace=None, stream=None):
    """Differential attention (fa_diff_fwd): (o, lse, o2).

    q [B,2H,N,64] and k [B,2H_kv,N,64] hold the two maps of head pair h in
    heads 2h and 2h + 1, v [B,H_kv,N,128]; lam float32 [H].
    o = (softmax(tau q1 k1^T) - lam softmax(tau q2 k2^T)) v, [B,H,N,128];
    lse float32 [B,2H,N].  o2, the second map's own output, is what
    :func:`diff_bwd` needs besides; ``need_o2=False`` leaves it out (None).
    ``out`` = (o, lse, o2), o2 None where it is not needed; o and o2 share
    their strides."""
    p = _diff_params(q, k, v, lam, causal, window, scale)
    B, H, N, dv = p.B, p.H, p.N, 2 * p.d
    with _on(q.device, stream) as raw:
        lens = _lens(seqlens_k, B, q.device)
        p.seqlens_k = _ptr(lens)
        if out is None:
            o = torch.empty((B, H, N, dv), device=q.device, dtype=q.dtype)
            o2 = torch.empty_like(o) if need_o2 else None
            lse = torch.empty((B, 2 * H, N), device=q.device, dtype=torch.float32)
        else:
            o, lse, o2 = out
            for t, n in ((o, "o"), (o2, "o2")):
                if t is None and n == "o2" and not need_o2:
                    continue
                if t is None or tuple(t.shape) != (B, H, N, dv):
                    raise ValueError("out %s must have shape %s" % (n, (B, H, N, dv)))
                _check4(t, "out " + n, q.device, q.dtype)
            if o2 is not None and o2.stride() != o.stride():
                raise ValueError("out o and o2 must share their strides")
            _check_place(lse, "out lse", q.device, torch.float32)
            if tuple(lse.shape) != (B, 2 * H, N) or not lse.is_contiguous():
                raise ValueError("out lse must be contiguous with shape %s" % ((B, 2 * H, N),))
        _set_strides(p, "o", o)
        a = ctypes.addressof(p)
        size = _fn("fa_diff_fwd_workspace_size", _vp, restype=ctypes.c_size_t)(a)
        ws = _need_workspace(workspace, size, q.device)
        f = _fn("fa_diff_fwd", *([_vp] * 8), ctypes.c_size_t, _vp)
        st = f(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(o2), lse.data_ptr(), ws.data_ptr(),
               ws.numel(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_diff_fwd")
    diff_fwd.last_workspace = ws
    return o, lse, o2


def diff_bwd(q, k, v, lam, o, o2, do, lse, *, causal=False, seqlens_k=None, window=0, scale=None, out=None,
             workspace=None, stream=None):
    """(dq, dk, dv, dlam) of :func:`diff_fwd` (fa_diff_bwd) for the upstream
    gradient ``do`` [B,H,N,128]; o, o2, lse and the masks are the forward
    call's.  dq, dk, dv have the shapes and strides of q, k, v; dlam is
    float32 [H].  ``out`` = (dq, dk, dv, dlam)."""
    p = _diff_params(q, k, v, lam, causal, window, scale)
    B, H, N, dv_ = p.B, p.H, p.N, 2 * p.d
    for t, n in ((o, "o"), (o2, "o2"), (do, "do")):
        _check4(t, n, q.device, q.dtype)
        if tuple(t.shape) != (B, H, N, dv_):
            raise ValueError("%s must have shape %s" % (n, (B, H, N, dv_)))
    if o.stride() != o2.stride():
        raise ValueError("o and o2 must share their strides")
    _check_place(lse, "lse", q.device, torch.float32)
    if tuple(lse.shape) != (B, 2 * H, N) or not lse.is_contiguous():
        raise ValueError("lse must be the contiguous [B, 2H, N] float32 tensor diff_fwd returns")
    _set_strides(p, "o", o)
    _set_strides(p, "do", do)
    with _on(q.device, stream) as raw:
        lens = _lens(seqlens_k, B, q.device)
        p.seqlens_k = _ptr(lens)
        likes = (q, k, v)
        if out is None:
            dq, dk, dv = (torch.empty_strided(t.shape, t.stride(), device=t.device, dtype=t.dtype) for t in likes)
            dlam = torch.empty((H,), device=q.device, dtype=torch.float32)
        else:
            dq, dk, dv, dlam = out
            _check_place(dlam, "out dlam", q.device, torch.float32)
            if tuple(dlam.shape) != (H,) or not dlam.is_contiguous():
                raise ValueError("out dlam must be contiguous with shape [H]")
        for t, like, n in zip((dq, dk, dv), likes, ("dq", "dk", "dv")):
            _check_out(t, like, n)
            if t.stride() != like.stride():
                raise ValueError("out %s must have the strides %s" % (n, like.stride()))
        a = ctypes.addressof(p)
        size = _fn("fa_diff_bwd_workspace_size", _vp, restype=ctypes.c_size_t)(a)
        ws = _need_workspace(workspace, size, q.device)
        f = _fn("fa_diff_bwd", *([_vp] * 13), ctypes.c_size_t, _vp)
        st = f(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), o2.data_ptr(), do.data_ptr(), lse.data_ptr(),
               dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dlam.data_ptr(), ws.data_ptr(), ws.numel(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_diff_bwd")
    diff_bwd.last_workspace = ws
    return dq, dk, dv, dlam


class fa_prefix_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "H", "H_kv", "T", "P", "M", "d", "dtype")] +
                [("scale", _f32), ("seqlens_k", _vp)] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("q", "o", "k", "v") for x in "bhn"] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("kp", "vp") for x in "hn"])


def prefix_fwd(q, k_prefix, v_prefix, k, v, seqlens_k, *, scale=None, out=None, workspace=None, stream=None):
    """Attention of B sequences that share a prefix (fa_prefix_fwd): (o, lse).

    q [B,H,T,d] holds the T new tokens of each sequence (T = 1: one decoding
    step), k_prefix and v_prefix [H_kv,P,d] the one shared prefix, k and v
    [B,H_kv,M,d] the sequences' own caches with ``seqlens_k`` [B] rows
    filled, the new tokens' included.  Query t sees the whole prefix and the
    own keys j <= seqlens_k[b] - T + t.  P = 0 is plain cached attention;
    k_prefix, v_prefix (or k, v) may then be None.  o [B,H,T,d], lse float32
    [B,H,T].  ``out`` = (o, lse)."""
    _check4(q, "q")
    B, H, T, d = q.shape
    dev = q.device
    if (k is None) != (v is None) or (k_prefix is None) != (v_prefix is None):
        raise ValueError("k and v, and k_prefix and v_prefix, come together")
    if k is None and k_prefix is None:
        raise ValueError("neither a prefix nor caches given")
    p = fa_prefix_params()
    p.B, p.H, p.T, p.d, p.dtype = B, H, T, d, DTYPE_CODE[q.dtype]
    p.H_kv = k.shape[1] if k is not None else k_prefix.shape[0]
    p.scale = 0.0 if scale is None else float(scale)
    if p.H_kv < 1 or H % p.H_kv:
        raise ValueError("the number of query heads must be a multiple of the number of K/V heads")
    if k is not None:
        p.M = k.shape[2]
        for t, n in ((k, "k"), (v, "v")):
            _check4(t, n, dev, q.dtype)
            if tuple(t.shape) != (B, p.H_kv, p.M, d):
                raise ValueError("k, v must be [B, H_kv, M, d] with the B, d of q")
            _set_strides(p, n, t)
    if k_prefix is not None:
        p.P = k_prefix.shape[1]
        for t, n in ((k_prefix, "k_prefix"), (v_prefix, "v_prefix")):
            if t.dim() != 3 or tuple(t.shape) != (p.H_kv, p.P, d):
                raise ValueError("k_prefix, v_prefix must be [H_kv, P, d]")
            _check4(t[None], n, dev, q.dtype)
        p.kp_stride_h, p.kp_stride_n = k_prefix.stride()[:2]
        p.vp_stride_h, p.vp_stride_n = v_prefix.stride()[:2]
    _set_strides(p, "q", q)
    with _on(dev, stream) as raw:
        lens = _lens(seqlens_k, B, dev)
        if lens is None:
            raise ValueError("seqlens_k must be given")
        p.seqlens_k = lens.data_ptr()
        if out is None:
            o = torch.empty((B, H, T, d), device=dev, dtype=q.dtype)
            lse = torch.empty((B, H, T), device=dev, dtype=torch.float32)
        else:
            o, lse = out
            _check_out(o, q, "o")
            _check_place(lse, "out lse", dev, torch.float32)
            if tuple(lse.shape) != (B, H, T) or not lse.is_contiguous():
                raise ValueError("out lse must be contiguous with shape %s" % ((B, H, T),))
        _set_strides(p, "o", o)
        a = ctypes.addressof(p)
        size = _fn("fa_prefix_workspace_size", _vp, restype=ctypes.c_size_t)(a)
        ws = _need_workspace(workspace, size, dev)
        f = _fn("fa_prefix_fwd", *([_vp] * 9), ctypes.c_size_t, _vp)
        st = f(a, q.data_ptr(), _ptr(k_prefix), _ptr(v_prefix), _ptr(k), _ptr(v), o.data_ptr(), lse.data_ptr(),
               ws.data_ptr(), ws.numel(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_prefix_fwd")
    prefix_fwd.last_workspace = ws
    return o, lse
