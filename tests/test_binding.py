"""What the binding does before a call reaches the library: function objects and packed parameters.  CPU only."""
import ctypes

import pytest

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
