"""Workspaces at the least alignment that the operators promise to take: 16 bytes,
not 32.

CPU: the shared prefix's size leaves room to round the partial rows up to the 32
bytes of the tensor-memory kernel's stores.  GPU: every operator with a
workspace gives the bits of the default call, in a buffer of exactly its size
whose surroundings stay as they were.
"""
import ctypes

import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from exact_io_aware_tiled_gb300 import _ops
from tests import test_diff, test_prefix


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load()


def al256(n):
    return -(-n // 256) * 256


def test_prefix_workspace_leaves_room_for_aligned_rows():
    # 152 K/V heads of 33 rows fill the GPU with one split each: 152 x 33 partial rows and their statistics
    p = test_prefix._params(B=1, H=152, H_kv=152, T=33, P=4096, M=0, d=128)
    for t in ("q", "o", "k", "v", "kp", "vp"):
        setattr(p, t + "_stride_n", 128)
    rows = 152 * 33
    size = _ops._fn("fa_prefix_workspace_size", ctypes.c_void_p, restype=ctypes.c_size_t)(ctypes.addressof(p))
    assert size >= 256 + al256(rows * 16) + al256(rows * 128 * 4) + 16


class Guarded:
    """A workspace of the given size at 16 modulo 32, with filled bytes on both sides."""

    def __init__(self, size):
        self.buf = torch.full((size + 64,), 171, device="cuda", dtype=torch.uint8)
        self.at = (16 - self.buf.data_ptr()) % 32
        self.size = size
        self.ws = self.buf[self.at:self.at + size]
        assert self.ws.data_ptr() % 32 == 16

    def intact(self):
        return bool((self.buf[:self.at] == 171).all()) and bool((self.buf[self.at + self.size:] == 171).all())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,T,P", [(3, 4, 2, 2, 200),           # register products
                                         (1, 16, 4, 10, 66000),       # tensor memory, two splits a CTA at d = 64
                                         (2, 32, 4, 10, 30001)])      # tensor memory, 256-row tiles
def test_shared_prefix(d, B, H, Hkv, T, P):
    x = test_prefix.inputs(B, H, Hkv, T, P, 40, d, "bf16", 3)
    lens = torch.arange(B, device="cuda", dtype=torch.int32) * 17 + T
    want = fa.prefix_fwd(*x, lens)
    g = Guarded(fa.prefix_fwd.last_workspace.numel())
    got = fa.prefix_fwd(*x, lens, workspace=g.ws)
    assert fa.check_status(g.ws) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and g.intact()


@pytest.mark.gpu
@pytest.mark.parametrize("P", [100, 40000])
def test_shared_prefix_differential(P):
    x, lam = test_prefix.diff_inputs(1, 8, 4, 20, P, 60, "bf16", 4)
    lens = torch.tensor([60], device="cuda", dtype=torch.int32)
    want = fa.prefix_fwd(*x, lens, lam=lam)
    g = Guarded(fa.prefix_fwd.last_workspace.numel())
    got = fa.prefix_fwd(*x, lens, lam=lam, workspace=g.ws)
    assert fa.check_status(g.ws) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and g.intact()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_differential(dtype):
    q, k, v, lam, do = test_diff.inputs(2, 4, 2, 190, dtype, 6)
    want = fa.diff_fwd(q, k, v, lam, causal=True)
    g = Guarded(fa.diff_fwd.last_workspace.numel())
    got = fa.diff_fwd(q, k, v, lam, causal=True, workspace=g.ws)
    assert fa.check_status(g.ws) == 0 and g.intact()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    o, lse, o2 = want
    want = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True)
    g = Guarded(fa.diff_bwd.last_workspace.numel())
    got = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True, workspace=g.ws)
    assert fa.check_status(g.ws) == 0 and g.intact()
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    # dQ is accumulated in arrival order, then rounded: one step of the dtype apart at most, few elements
    assert test_diff.rel(got[0], want[0].double()) <= torch.finfo(test_diff.DT[dtype]).eps
