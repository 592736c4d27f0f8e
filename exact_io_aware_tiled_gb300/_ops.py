"""ctypes binding of the operators around the attention passes (include/fa.h,
ABI 1.5): rotary positions, norms with the rotation, differential attention,
attention over a shared prefix.

As in ``_lib``: argument checks, output and workspace allocation with torch,
raw pointers and the stream; the computation runs in ``libfa_gb300.so``.
A call runs on the device of its tensors, on ``stream`` or that device's
current stream.  With ``stream`` given, outputs and workspace are allocated
on that stream, and small conversions of index arguments run on it too.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import Optional

import torch

from ._lib import DTYPE_CODE, FA_OK, FAError, int32_lengths, load

ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


def _packer(cls):
    """A function of the fields of a parameter struct, pointers as integers, that returns its bytes (a call takes
    them as they are; filling a ctypes structure costs three times as long)."""
    code = {_i32: "i", _i64: "q", _vp: "P", _f32: "f"}
    s = struct.Struct("@" + "".join(code[t] for _, t in cls._fields_) + "0q")     # padded to its alignment
    assert s.size == ctypes.sizeof(cls)
    return s.pack


class fa_rope_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "H", "H_kv", "N", "d", "rot", "dtype", "interleaved", "backward",
                                     "positions_i64")] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("q", "k", "q_out", "k_out") for x in "bhn"] +
                [("positions", _vp), ("pos_stride_b", _i64), ("pos_stride_n", _i64), ("start", _i64),
                 ("inv_freq", _vp), ("mscale", _f32)])


_pack_rope = _packer(fa_rope_params)

_typed = {}


def _fn(name, *argtypes, restype=ctypes.c_int):
    """The library's function `name` with its argument types set (once)."""
    f = _typed.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes, f.restype = list(argtypes), restype
        _typed[name] = f
    return f


def _ptrs(name, n):
    """A function of n pointers (the stream among them) that returns a status."""
    return _typed.get(name) or _fn(name, *([_vp] * n))


def _sized(name, n):
    """A function of n pointers, a workspace's size and the stream that returns a status."""
    return _typed.get(name) or _fn(name, *([_vp] * n), ctypes.c_size_t, _vp)


def _size_of(name):
    return _typed.get(name) or _fn(name, _vp, restype=ctypes.c_size_t)


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
    __slots__ = ("index",)

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        return torch._C._cuda_getCurrentRawStream(self.index)

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
    return _Plain(device.index)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _rows(t, name, like, shape):
    """Strides of a [.,.,.,d] tensor of `shape` on the device and in the dtype of the CUDA tensor `like`."""
    st = t.stride()
    if t.shape != shape or t.dtype is not like.dtype or t.get_device() != like.get_device() or \
            (st[-1] != 1 and shape[-1] > 1):
        if tuple(t.shape) != tuple(shape):
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        _check_place(t, name, like.device, like.dtype)
        raise ValueError("%s: the last dimension must be contiguous (stride 1), got strides %s" % (name, st))
    return st


def _check4(t, name):
    """The call's first tensor: 4 dimensions, on a GPU, a dtype of the library, contiguous rows."""
    if t.dim() != 4:
        raise ValueError("%s must have 4 dimensions, got shape %s" % (name, tuple(t.shape)))
    _check_place(t, name)
    if t.stride(3) != 1 and t.shape[3] > 1:
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


def _flat_f32(t, name, device, shape):
    if tuple(t.shape) != shape or t.dtype is not torch.float32 or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous float32 tensor of shape %s on %s" % (name, shape, device))


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


def _check_freq(inv_freq, q):
    if inv_freq.dim() != 1 or inv_freq.dtype is not torch.float64 or inv_freq.get_device() != q.get_device() or \
            not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 tensor [rot/2] on q's device")


def _positions(positions, q):
    """(pointer, int64?, stride over sequences, stride over tokens) of the positions of q's tokens; zeros for None."""
    if positions is None:
        return 0, 0, 0, 0
    B, N = q.shape[0], q.shape[2]
    wide = positions.dtype is torch.int64
    if not (wide or positions.dtype is torch.int32) or positions.get_device() != q.get_device():
        raise ValueError("positions must be an int32 or int64 tensor on q's device")
    ps = positions.shape
    if not (ps == (N,) or ps == (B, N) or ps == (1, N)):
        raise ValueError("positions must have shape [N], [1, N] or [B, N]")
    return positions.data_ptr(), wide, positions.stride(0) if len(ps) == 2 and ps[0] > 1 else 0, positions.stride(-1)


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
    Hkv, ks = 0, (0, 0, 0)
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must be [B, H_kv, N, d]")
        Hkv = k.shape[1]
        ks = _rows(k, "k", q, (B, Hkv, N, d))[:3]
    _check_freq(inv_freq, q)
    pos, wide, pos_b, pos_n = _positions(positions, q)
    with _on(q.device, stream) as raw:
        if out is None:
            qo = torch.empty_like(q)
            ko = None if k is None else torch.empty_like(k)
            qos, kos = qo.stride()[:3], ks if k is None else ko.stride()[:3]
        else:
            qo, ko = (out, None) if k is None else out
            qos = _rows(qo, "out q", q, q.shape)[:3]
            kos = ks if k is None else _rows(ko, "out k", q, k.shape)[:3]
        p = _pack_rope(B, H, Hkv, N, d, 2 * inv_freq.shape[0], DTYPE_CODE[q.dtype], bool(interleaved),
                       bool(backward), wide, *q.stride()[:3], *ks, *qos, *kos, pos, pos_b, pos_n, int(start),
                       inv_freq.data_ptr(), float(mscale))
        st = _ptrs("fa_rope", 6)(p, q.data_ptr(), None if k is None else k.data_ptr(), qo.data_ptr(),
                                 None if k is None else ko.data_ptr(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_rope")
    return qo if k is None else (qo, ko)


class fa_norm_rope_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "H", "H_kv", "N", "d", "rot", "dtype", "interleaved", "positions_i64")] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("q", "k", "q_out", "k_out", "dq", "dk") for x in "bhn"] +
                [("positions", _vp), ("pos_stride_b", _i64), ("pos_stride_n", _i64), ("start", _i64),
                 ("inv_freq", _vp), ("mscale", _f32), ("eps", _f32)])


_pack_norm = _packer(fa_norm_rope_params)


def _norm_args(q, k, q_weight, k_weight, inv_freq, out, what):
    """Checks of both directions' arguments: (H_kv, k's strides, rot, checked outputs or None)."""
    _check4(q, "q")
    B, H, N, d = q.shape
    Hkv, ks = 0, (0, 0, 0)
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must be [B, H_kv, N, d]")
        Hkv = k.shape[1]
        ks = _rows(k, "k", q, (B, Hkv, N, d))[:3]
    elif k_weight is not None:
        raise ValueError("k_weight is given without k")
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _flat_f32(t, n, q.device, (d,))
    if inv_freq is not None:
        _check_freq(inv_freq, q)
    if out is not None:
        out = (out, None) if k is None and isinstance(out, torch.Tensor) else out
        _rows(out[0], "out " + what[0], q, q.shape)
        if k is not None:
            _rows(out[1], "out " + what[1], q, k.shape)
    return Hkv, ks, 0 if inv_freq is None else 2 * inv_freq.shape[0], out


def norm_rope(q, k=None, *, q_weight=None, k_weight=None, eps=1e-6, inv_freq=None, positions=None, start=0, mscale=1.0,
              interleaved=False, out=None, stream=None):
    """q and k normalised for each head and rotated by their positions in one
    pass (fa_norm_rope), as (q_out, k_out); q_out alone without k.

    A row x (one token of one head) becomes R_p (w * x / sqrt(mean(x^2) + eps)).
    q [B,H,N,d], k [B,H_kv,N,d]; ``q_weight`` and ``k_weight`` float32 [d] or
    None (ones).  ``inv_freq`` (None: no rotation), ``positions``, ``start``,
    ``mscale`` and ``interleaved`` as in :func:`rope`.  ``out`` = (q_out,
    k_out), or q_out without k, may be the inputs themselves (but the backward
    pass needs q and k as they were)."""
    Hkv, ks, rot, out = _norm_args(q, k, q_weight, k_weight, inv_freq, out, ("q", "k"))
    B, H, N, d = q.shape
    pos, wide, pos_b, pos_n = _positions(positions, q)
    with _on(q.device, stream) as raw:
        qo, ko = (torch.empty_like(q), None if k is None else torch.empty_like(k)) if out is None else out
        p = _pack_norm(B, H, Hkv, N, d, rot, DTYPE_CODE[q.dtype], bool(interleaved), wide, *q.stride()[:3], *ks,
                       *qo.stride()[:3], *(ks if k is None else ko.stride()[:3]), 0, 0, 0, 0, 0, 0, pos, pos_b, pos_n,
                       int(start), 0 if inv_freq is None else inv_freq.data_ptr(), float(mscale), float(eps))
        st = _ptrs("fa_norm_rope", 8)(p, q.data_ptr(), None if k is None else k.data_ptr(), _ptr(q_weight),
                                      _ptr(k_weight), qo.data_ptr(), None if k is None else ko.data_ptr(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_norm_rope")
    return qo if k is None else (qo, ko)


def norm_rope_bwd(q, k, dq_out, dk_out=None, *, q_weight=None, k_weight=None, eps=1e-6, inv_freq=None, positions=None,
                  start=0, mscale=1.0, interleaved=False, out=None, workspace=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of :func:`norm_rope` (fa_norm_rope_bwd)
    for the gradients ``dq_out``, ``dk_out`` of its outputs; q, k and the other
    arguments are the forward call's.  The gradient of a weight that is None,
    and everything of a k that is None, is None.  The weights' gradients are
    float32 [d].  ``out`` = (dq, dk) may be the tensors dq_out, dk_out."""
    Hkv, ks, rot, out = _norm_args(q, k, q_weight, k_weight, inv_freq, out, ("dq", "dk"))
    B, H, N, d = q.shape
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out come together")
    gqs = _rows(dq_out, "dq_out", q, q.shape)[:3]
    gks = (0, 0, 0) if k is None else _rows(dk_out, "dk_out", q, k.shape)[:3]
    pos, wide, pos_b, pos_n = _positions(positions, q)
    dev = q.device
    with _on(dev, stream) as raw:
        dq, dk = (torch.empty_like(q), None if k is None else torch.empty_like(k)) if out is None else out
        dwq = None if q_weight is None else torch.empty((d,), device=dev, dtype=torch.float32)
        dwk = None if k_weight is None else torch.empty((d,), device=dev, dtype=torch.float32)
        p = _pack_norm(B, H, Hkv, N, d, rot, DTYPE_CODE[q.dtype], bool(interleaved), wide, *q.stride()[:3], *ks,
                       *dq.stride()[:3], *(ks if k is None else dk.stride()[:3]), *gqs, *gks, pos, pos_b, pos_n,
                       int(start), 0 if inv_freq is None else inv_freq.data_ptr(), float(mscale), float(eps))
        ws = _need_workspace(workspace, _size_of("fa_norm_rope_bwd_workspace_size")(p), dev)
        st = _sized("fa_norm_rope_bwd", 12)(p, q.data_ptr(), None if k is None else k.data_ptr(), dq_out.data_ptr(),
                                            None if k is None else dk_out.data_ptr(), _ptr(q_weight), _ptr(k_weight),
                                            dq.data_ptr(), None if k is None else dk.data_ptr(), _ptr(dwq), _ptr(dwk),
                                            ws.data_ptr(), ws.numel(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_norm_rope_bwd")
    return dq, dk, dwq, dwk


class fa_diff_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "H", "H_kv", "N", "d", "dtype", "causal", "window")] +
                [("scale", _f32), ("seqlens_k", _vp), ("lam", _vp)] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("q", "k", "v", "o", "do") for x in "bhn"])


_pack_diff = _packer(fa_diff_params)

def _lens(seqlens, B, device, name="seqlens_k"):
    """int32 [B] lengths on `device` (converted on the current stream where they are something else)."""
    if seqlens is None:
        return None
    if seqlens.shape != (B,):
        raise ValueError("%s must have shape [B] = [%d]" % (name, B))
    if seqlens.dtype is torch.int32 and seqlens.device == device and seqlens.is_contiguous():
        return seqlens
    if seqlens.dtype.is_floating_point or seqlens.dtype == torch.bool:
        raise ValueError("%s must hold whole numbers" % name)
    return int32_lengths(seqlens, device)


def _need_workspace(workspace, size, device):
    if workspace is None:
        return torch.empty(size, device=device, dtype=torch.uint8)
    if workspace.dtype != torch.uint8 or workspace.numel() < size or workspace.device != device or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor of >= %d bytes on %s" % (size, device))
    return workspace


def _diff_args(q, k, v, lam, causal, window, scale, lens, os, dos):
    """fa_diff_params of checked tensors; os, dos: strides of o (and o2) and of dO."""
    return _pack_diff(q.shape[0], q.shape[1] // 2, v.shape[1], q.shape[2], 64, DTYPE_CODE[q.dtype], bool(causal),
                      int(window), 0.0 if scale is None else float(scale), 0 if lens is None else lens.data_ptr(),
                      lam.data_ptr(), *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *os[:3], *dos[:3])


def _check_diff(q, k, v, lam):
    _check4(q, "q")
    B, H2, N, d = q.shape
    if d != 64 or H2 % 2 or v.dim() != 4 or v.shape[1] < 1 or (H2 // 2) % v.shape[1]:
        raise ValueError("q must be [B, 2H, N, 64] (the two maps of head pair h in heads 2h, 2h + 1), k [B, 2 H_kv, N, "
                         "64] and v [B, H_kv, N, 128], H a multiple of H_kv; got q %s, v %s" %
                         (tuple(q.shape), tuple(v.shape)))
    _rows(k, "k", q, (B, 2 * v.shape[1], N, 64))
    _rows(v, "v", q, (B, v.shape[1], N, 128))
    _flat_f32(lam, "lam", q.device, (H2 // 2,))
    return B, H2 // 2, N


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
    B, H, N = _check_diff(q, k, v, lam)
    dev = q.device
    with _on(dev, stream) as raw:
        lens = _lens(seqlens_k, B, dev)
        if out is None:
            o = torch.empty((B, H, N, 128), device=dev, dtype=q.dtype)
            o2 = torch.empty_like(o) if need_o2 else None
            lse = torch.empty((B, 2 * H, N), device=dev, dtype=torch.float32)
            os = o.stride()
        else:
            o, lse, o2 = out
            os = _rows(o, "out o", q, (B, H, N, 128))
            if o2 is None and need_o2:
                raise ValueError("out o2 is missing (need_o2=False leaves it out)")
            if o2 is not None and _rows(o2, "out o2", q, (B, H, N, 128)) != os:
                raise ValueError("out o and o2 must share their strides")
            _flat_f32(lse, "out lse", dev, (B, 2 * H, N))
        a = _diff_args(q, k, v, lam, causal, window, scale, lens, os, (0, 0, 0))
        ws = _need_workspace(workspace, _size_of("fa_diff_fwd_workspace_size")(a), dev)
        st = _sized("fa_diff_fwd", 8)(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                      None if o2 is None else o2.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
                                      raw)
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
    B, H, N = _check_diff(q, k, v, lam)
    dev = q.device
    os = _rows(o, "o", q, (B, H, N, 128))
    if _rows(o2, "o2", q, (B, H, N, 128)) != os:
        raise ValueError("o and o2 must share their strides")
    dos = _rows(do, "do", q, (B, H, N, 128))
    _flat_f32(lse, "lse", dev, (B, 2 * H, N))
    with _on(dev, stream) as raw:
        lens = _lens(seqlens_k, B, dev)
        if out is None:
            dq, dk, dv = (torch.empty_strided(t.shape, t.stride(), device=dev, dtype=t.dtype) for t in (q, k, v))
            dlam = torch.empty((H,), device=dev, dtype=torch.float32)
        else:
            dq, dk, dv, dlam = out
            for t, like, n in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
                if _rows(t, "out " + n, q, like.shape) != like.stride():
                    raise ValueError("out %s must have the strides %s" % (n, like.stride()))
            _flat_f32(dlam, "out dlam", dev, (H,))
        a = _diff_args(q, k, v, lam, causal, window, scale, lens, os, dos)
        ws = _need_workspace(workspace, _size_of("fa_diff_bwd_workspace_size")(a), dev)
        st = _sized("fa_diff_bwd", 13)(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), o2.data_ptr(),
                                       do.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                       dlam.data_ptr(), ws.data_ptr(), ws.numel(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_diff_bwd")
    diff_bwd.last_workspace = ws
    return dq, dk, dv, dlam


class fa_prefix_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "H", "H_kv", "T", "P", "M", "d", "dtype")] +
                [("scale", _f32), ("seqlens_k", _vp)] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("q", "o", "k", "v") for x in "bhn"] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("kp", "vp") for x in "hn"] + [("lam", _vp)])


_pack_prefix = _packer(fa_prefix_params)

def prefix_fwd(q, k_prefix, v_prefix, k, v, seqlens_k, *, lam=None, scale=None, out=None, workspace=None, stream=None):
    """Attention of B sequences that share a prefix (fa_prefix_fwd): (o, lse).

    q [B,H,T,d] holds the T new tokens of each sequence (T = 1: one decoding
    step), k_prefix and v_prefix [H_kv,P,d] the one shared prefix, k and v
    [B,H_kv,M,d] the sequences' own caches with ``seqlens_k`` [B] rows
    filled, the new tokens' included.  Query t sees the whole prefix and the
    own keys j <= seqlens_k[b] - T + t.  P = 0 is plain cached attention;
    k_prefix, v_prefix (or k, v) may then be None.  o [B,H,T,d], lse float32
    [B,H,T].  ``out`` = (o, lse).

    With ``lam`` (float32 [H]) it is :func:`diff_fwd`'s step for few tokens: q
    [B,2H,T,64], k_prefix [2H_kv,P,64], k [B,2H_kv,M,64], v_prefix
    [H_kv,P,128], v [B,H_kv,M,128], o [B,H,T,128], lse [B,2H,T]."""
    _check4(q, "q")
    B, SH, T, d = q.shape
    dev = q.device
    maps = 1 if lam is None else 2            # score heads per head
    H, dv = SH // maps, maps * d
    if lam is not None:
        if SH % 2 or d != 64:
            raise ValueError("with lam, q must be [B, 2H, T, 64]")
        _flat_f32(lam, "lam", dev, (H,))
    if (k is None) != (v is None) or (k_prefix is None) != (v_prefix is None):
        raise ValueError("k and v, and k_prefix and v_prefix, come together")
    P = M = 0
    ks = vs = kps = vps = (0, 0, 0)
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k, v must be [B, H_kv, M, d]")
        Hkv, M = k.shape[1] // maps, k.shape[2]
        ks, vs = _rows(k, "k", q, (B, maps * Hkv, M, d)), _rows(v, "v", q, (B, Hkv, M, dv))
    elif k_prefix is not None:
        Hkv = k_prefix.shape[0] // maps
    else:
        raise ValueError("neither a prefix nor caches given")
    if Hkv < 1 or H % Hkv:
        raise ValueError("the number of query heads must be a multiple of the number of K/V heads")
    if k_prefix is not None:
        if k_prefix.dim() != 3:
            raise ValueError("k_prefix, v_prefix must be [H_kv, P, d]")
        P = k_prefix.shape[1]
        kps = _rows(k_prefix, "k_prefix", q, (maps * Hkv, P, d))
        vps = _rows(v_prefix, "v_prefix", q, (Hkv, P, dv))
    if seqlens_k is None:
        raise ValueError("seqlens_k must be given")
    with _on(dev, stream) as raw:
        lens = _lens(seqlens_k, B, dev)
        if out is None:
            o = torch.empty((B, H, T, dv), device=dev, dtype=q.dtype)
            lse = torch.empty((B, SH, T), device=dev, dtype=torch.float32)
            os = o.stride()
        else:
            o, lse = out
            os = _rows(o, "out o", q, (B, H, T, dv))
            _flat_f32(lse, "out lse", dev, (B, SH, T))
        a = _pack_prefix(B, H, Hkv, T, P, M, d, DTYPE_CODE[q.dtype], 0.0 if scale is None else float(scale),
                         lens.data_ptr(), *q.stride()[:3], *os[:3], *ks[:3], *vs[:3], *kps[:2], *vps[:2],
                         0 if lam is None else lam.data_ptr())
        ws = _need_workspace(workspace, _size_of("fa_prefix_workspace_size")(a), dev)
        st = _sized("fa_prefix_fwd", 9)(a, q.data_ptr(), _ptr(k_prefix), _ptr(v_prefix), _ptr(k), _ptr(v), o.data_ptr(),
                                        lse.data_ptr(), ws.data_ptr(), ws.numel(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_prefix_fwd")
    prefix_fwd.last_workspace = ws
    return o, lse
