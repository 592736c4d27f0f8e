"""ctypes binding of the paged cache in 8 bits (include/fa.h, ABI 1.5).

A cache is five tensors that the program owns: ``k_cache`` and ``v_cache``
[pages,H_kv,page,d] of float8_e4m3fn (or uint8) codes, ``k_scale`` and
``v_scale`` float32 [pages,H_kv], and ``table`` int32 [B,width], whose row b
names the pages of sequence b in the order of its tokens (-1, or anything
outside [0, pages), for a page that is absent).  ``seqlens`` int32 [B] counts the
tokens, the new ones included; tokens from width * page on count as those of an
absent page.  As in ``_ops``: checks, allocation,
pointers and the stream; the computation runs in ``libfa_gb300.so``.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import DTYPE_CODE, FA_OK, FAError, _int32, int32_lengths
from ._ops import (_check4, _flat_f32, _i32, _i64, _f32, _lens, _need_workspace, _on, _packer, _ptrs, _rows, _size_of,
                   _sized, _vp)


class fa_cache8_params(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "H", "H_kv", "T", "d", "dtype", "page", "pages", "width", "window", "sinks")] +
                [("scale", _f32), ("seqlens_k", _vp), ("table", _vp), ("table_stride", _i64)] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("q", "o", "k", "v") for x in "bhn"] +
                [("%s_stride_%s" % (t, x), _i64) for t in ("kc", "vc") for x in "phn"])


_pack = _packer(fa_cache8_params)
_none3 = (0, 0, 0)
_CODES = (torch.float8_e4m3fn, torch.uint8)


def _cache(k_cache, v_cache, k_scale, v_scale, like):
    """(pages, H_kv, page, d) of a cache whose tensors fit together, on the device of the CUDA tensor `like`."""
    shape, at = k_cache.shape, like.get_device()
    if len(shape) == 4 and v_cache.shape == shape and k_cache.dtype in _CODES and v_cache.dtype in _CODES and \
            k_cache.get_device() == at and v_cache.get_device() == at and k_cache.stride(3) == 1 and \
            v_cache.stride(3) == 1 and _scales(k_scale, shape, at) and _scales(v_scale, shape, at):
        return shape
    device = like.device
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [pages, H_kv, page, d], got %s and %s" %
                         (tuple(shape), tuple(v_cache.shape)))
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype not in _CODES:
            raise ValueError("%s must be float8_e4m3fn (or uint8 codes), got %s" % (n, t.dtype))
        if t.device != device:
            raise ValueError("%s must be on %s, got %s" % (n, device, t.device))
        if t.stride(3) != 1:
            raise ValueError("%s: the last dimension must be contiguous (stride 1), got strides %s" % (n, t.stride()))
    _flat_f32(k_scale, "k_scale", device, tuple(shape[:2]))
    _flat_f32(v_scale, "v_scale", device, tuple(shape[:2]))
    raise ValueError("the cache's tensors do not fit together")


def _scales(t, shape, at):
    return t.dtype is torch.float32 and t.get_device() == at and t.shape == shape[:2] and t.is_contiguous()


def _check_table(table, B):
    if table.dim() != 2 or table.shape[0] != B or table.shape[1] < 1:
        raise ValueError("table must have shape [B, width] with B = %d, got %s" % (B, tuple(table.shape)))
    if table.dtype.is_floating_point or table.dtype == torch.bool:
        raise ValueError("table must hold whole numbers")


def _table(table, device):
    """int32 rows on `device` (converted on the current stream where they are something else; numbers that int32 does
    not hold stay outside the pages)."""
    if table.dtype is torch.int32 and table.is_cuda and table.get_device() == device.index and table.stride(1) == 1 and \
            (table.shape[0] == 1 or table.stride(0) >= table.shape[1]):
        return table
    return int32_lengths(table, device)


def _given(seqlens, B):
    if seqlens is None:
        raise ValueError("seqlens must be given")
    if seqlens.shape != (B,):
        raise ValueError("seqlens must have shape [B] = [%d]" % B)


def cache8_append(k, v, k_cache, v_cache, k_scale, v_scale, table, seqlens, *, stream=None):
    """Writes new tokens into the cache (fa_cache8_append).

    k, v [B,H_kv,T,d] (float16, bfloat16) become rows seqlens[b] - T ..
    seqlens[b] - 1 of sequence b: quantised, with the scales of the pages that
    they touch brought up to date in ``k_scale`` and ``v_scale``.  The pages must be
    in ``table`` before the call and belong to one sequence."""
    _check4(k, "k")
    B, Hkv, T, d = k.shape
    vs = _rows(v, "v", k, k.shape)
    dev = k.device
    pages, heads, page, width = _cache(k_cache, v_cache, k_scale, v_scale, k)
    if (heads, width) != (Hkv, d):
        raise ValueError("the cache has %d heads of %d, k %d of %d" % (heads, width, Hkv, d))
    _check_table(table, B)
    _given(seqlens, B)
    with _on(dev, stream) as raw:
        lens, tab = _lens(seqlens, B, dev, "seqlens"), _table(table, dev)
        p = _pack(B, Hkv, Hkv, T, d, DTYPE_CODE[k.dtype], page, pages, tab.shape[1], 0, 0, 0.0, lens.data_ptr(),
                  tab.data_ptr(), tab.stride(0), *_none3, *_none3, *k.stride()[:3], *vs[:3], *k_cache.stride()[:3],
                  *v_cache.stride()[:3])
        st = _ptrs("fa_cache8_append", 8)(p, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                          k_scale.data_ptr(), v_scale.data_ptr(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_cache8_append")


def cache8_read(k_cache, v_cache, k_scale, v_scale, table, seqlens, *, dtype=torch.bfloat16, rows=None, out=None,
                stream=None):
    """(k, v) [B,H_kv,rows,d]: the first ``rows`` tokens of every sequence out of
    the cache as values of ``dtype`` (fa_cache8_read), zeros behind seqlens[b]
    and for absent pages.  rows: width * page by default.  ``out`` = (k, v)."""
    dev = k_cache.device
    if not k_cache.is_cuda:
        raise ValueError("k_cache must be a CUDA tensor")
    pages, Hkv, page, d = _cache(k_cache, v_cache, k_scale, v_scale, k_cache)
    if table.dim() != 2:
        raise ValueError("table must have shape [B, width]")
    B = table.shape[0]
    _check_table(table, B)
    _given(seqlens, B)
    if dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("dtype must be float16 or bfloat16, got %s" % dtype)
    n = table.shape[1] * page if rows is None else int(rows)
    if n < 1:
        raise ValueError("rows must be at least 1, got %d" % n)
    with _on(dev, stream) as raw:
        lens, tab = _lens(seqlens, B, dev, "seqlens"), _table(table, dev)
        if out is None:
            k, v = (torch.empty((B, Hkv, n, d), device=dev, dtype=dtype) for _ in range(2))
        else:
            k, v = out
            for t, name in ((k, "out k"), (v, "out v")):
                if t.dtype is not dtype or not t.is_cuda:
                    raise ValueError("%s must be a CUDA tensor of %s" % (name, dtype))
            _check4(k, "out k")
            _rows(v, "out v", k, k.shape)
            if tuple(k.shape) != (B, Hkv, n, d) or k.device != dev:
                raise ValueError("out k must have shape %s on %s" % ((B, Hkv, n, d), dev))
        p = _pack(B, Hkv, Hkv, n, d, DTYPE_CODE[dtype], page, pages, tab.shape[1], 0, 0, 0.0, lens.data_ptr(),
                  tab.data_ptr(), tab.stride(0), *_none3, *_none3, *k.stride()[:3], *v.stride()[:3],
                  *k_cache.stride()[:3], *v_cache.stride()[:3])
        st = _ptrs("fa_cache8_read", 8)(p, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                        k.data_ptr(), v.data_ptr(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_cache8_read")
    return k, v


def cache8_fwd(q, k_cache, v_cache, k_scale, v_scale, table, seqlens, *, window=0, sinks=0, scale=None, out=None,
               workspace=None, stream=None):
    """Attention of T new tokens of each of B sequences over their 8-bit caches
    (fa_cache8_fwd): (o, lse).  T is meant to be a few tokens: a long chunk is
    taken, but under a short window visits several times the keys it sees.

    q [B,H,T,d] (T = 1: one decoding step), H a multiple of the cache's heads;
    seqlens [B] counts the new tokens, whose keys :func:`cache8_append` has
    written.  Query t sees the keys j <= p = seqlens[b] - T + t and, with
    ``window`` > 0, of those only j > p - window and the first ``sinks``.  o
    [B,H,T,d], lse float32 [B,H,T].  ``out`` = (o, lse)."""
    _check4(q, "q")
    B, H, T, d = q.shape
    dev = q.device
    pages, Hkv, page, width = _cache(k_cache, v_cache, k_scale, v_scale, q)
    if width != d or Hkv < 1 or H % Hkv:
        raise ValueError("the cache has %d heads of %d, q %d of %d" % (Hkv, width, H, d))
    _check_table(table, B)
    _given(seqlens, B)
    with _on(dev, stream) as raw:
        lens, tab = _lens(seqlens, B, dev, "seqlens"), _table(table, dev)
        if out is None:
            o = torch.empty((B, H, T, d), device=dev, dtype=q.dtype)
            lse = torch.empty((B, H, T), device=dev, dtype=torch.float32)
        else:
            o, lse = out
            _rows(o, "out o", q, q.shape)
            _flat_f32(lse, "out lse", dev, (B, H, T))
        p = _pack(B, H, Hkv, T, d, DTYPE_CODE[q.dtype], page, pages, tab.shape[1], _int32(window), _int32(sinks),
                  0.0 if scale is None else float(scale), lens.data_ptr(), tab.data_ptr(), tab.stride(0),
                  *q.stride()[:3], *o.stride()[:3], *_none3, *_none3, *k_cache.stride()[:3], *v_cache.stride()[:3])
        ws = _need_workspace(workspace, _size_of("fa_cache8_workspace_size")(p), dev)
        st = _sized("fa_cache8_fwd", 9)(p, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                        v_scale.data_ptr(), o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), raw)
    if st != FA_OK:
        raise FAError(st, "fa_cache8_fwd")
    cache8_fwd.last_workspace = ws
    return o, lse
