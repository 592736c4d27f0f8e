"""What the binding does before a call reaches the library: function objects and packed parameters.  CPU only."""
import ctypes
import math

import pytest
import torch

from exact_io_aware_tiled_gb300 import _lib, _ops


@pytest.mark.parametrize("module,known", [(_lib, "_raw"), (_ops, "_typed")])
def test_a_function_is_shared_only_when_its_types_are_set(module, known, monkeypatch):
    # Another thread may look the function up at any time: without argument types ctypes passes addresses as 32-bit
    # integers, and without a result type a size comes back as one.
    shared = {}
    monkeypatch.setattr(module, known, shared)

    class Function:
        def __setattr__(self, name, value):
            assert name in ("argtypes", "restype")
            assert not shared, "visible before %s is set" % name
            object.__setattr__(self, name, value)

    class Library:
        def __getattr__(self, name):
            return Function()

        def __getitem__(self, name):
            return Function()

    monkeypatch.setattr(module, "load", Library)
    if module is _lib:
        f = module._fn("fa_fwd_workspace_size", ctypes.c_size_t, ctypes.c_void_p)
    else:
        f = module._fn("fa_fwd_workspace_size", ctypes.c_void_p, restype=ctypes.c_size_t)
    assert list(shared.values()) == [f] and f.argtypes == [ctypes.c_void_p] and f.restype is ctypes.c_size_t


def _params(**kw):
    q, k = torch.zeros(1, 2, 3, 64), torch.zeros(1, 1, 3, 64)
    d = dict(causal=False, seqlens_k=None, dropout_p=0.0, seed=0, offset=0, block_mask=None, scale=None, o_f32=None,
             prof=None, window=0, fwd_kernel=0)
    d.update(kw)
    return _lib.fa_params.from_buffer_copy(_lib._packed(q, k, **d)), _lib.make_params(q, k=k, **d)


@pytest.mark.parametrize("kw", [dict(), dict(scale=0.3), dict(scale=1e39), dict(scale=-1e39), dict(scale=math.nan),
                                dict(scale=1e-50), dict(dropout_p=1e39), dict(dropout_p=0.25, seed=-1, offset=2 ** 70),
                                dict(fwd_kernel=2), dict(window=17, causal=True)])
def test_packed_parameters_are_the_structure_s(kw):
    # numbers past float32 are infinite in both: the library then takes its default scale or refuses the call
    a, b = _params(**kw)
    for name, _ in _lib.fa_params._fields_:
        x, y = getattr(a, name), getattr(b, name)
        assert x == y or (x != x and y != y), name


def test_whole_numbers_past_int32_are_its_ends():
    a, _ = _params(fwd_kernel=7)
    assert a.fwd_kernel == 7
    p = _lib.fa_params.from_buffer_copy(_lib._packed(
        torch.zeros(1, 2, 3, 64), torch.zeros(1, 1, 3, 64), False, None, 0.0, 0, 0, None, None, None, None, 2 ** 40, 2 ** 40))
    assert (p.window, p.fwd_kernel) == (2 ** 31 - 1, 2 ** 31 - 1)


def _layouts():
    base = torch.zeros(2, 9, 8, 64, dtype=torch.float16)
    yield base.transpose(1, 2)                              # dense
    yield base[:, :, 1:4].transpose(1, 2)                   # q of a fused projection
    yield torch.zeros(2, 3, 12, 80)[:, :, :9, :64]          # rows and columns of a larger tensor
    yield torch.zeros(2, 1, 9, 64)[:, :, :1]
    yield torch.zeros(9, 2, 3, 64).permute(1, 2, 0, 3)


@pytest.mark.parametrize("t", list(_layouts()), ids=range(5))
def test_outputs_have_the_strides_that_the_library_writes_with(t):
    # q's strides are what O and dQ are written with, k's what dK and dV are: their storage has to reach as far
    for o in (_lib._outputs(None, [t])[0], _lib._empty_as(t)):
        assert o.shape == t.shape and o.stride() == t.stride() and o.dtype == t.dtype
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        assert o.untyped_storage().nbytes() >= (o.storage_offset() + last + 1) * o.element_size()


def test_tensors_on_another_device_are_refused():
    # their addresses would go to the kernels as they are
    q, k = torch.zeros(1, 2, 3, 64), torch.zeros(1, 1, 3, 64)
    with pytest.raises(ValueError, match="one device"):
        _lib._layouts([q], [k, k.to("meta")])
    with pytest.raises(ValueError, match="one device"):
        _lib._layouts([q, q.to("meta"), q], [k, k])
    with pytest.raises(ValueError, match="one device"):
        _lib._layouts([q], [k.to("meta"), k.to("meta")])
    _lib._layouts([q, q], [k, k])


def test_lse_and_workspaces_of_another_kind_are_refused():
    q = torch.zeros(2, 3, 5, 64, dtype=torch.float16)
    good = torch.zeros(2, 3, 5)
    _lib._check_lse(good, q)
    for bad in (good[:, :2], good[..., None], good.double(), good.half(), good.to("meta"), good[:1].expand(2, 3, 5),
                torch.zeros(2, 5, 3).transpose(1, 2)):
        with pytest.raises(ValueError, match="lse"):
            _lib._check_lse(bad, q)
    cpu = torch.device("cpu")
    assert _lib._workspace(100, torch.zeros(100, dtype=torch.uint8), cpu).numel() == 100
    for bad in (torch.zeros(99, dtype=torch.uint8), torch.zeros(100), torch.zeros(1, dtype=torch.uint8).expand(100),
                torch.zeros(200, dtype=torch.uint8)[::2], torch.zeros(100, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            _lib._workspace(100, bad, cpu)
