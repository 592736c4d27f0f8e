"""seqlens_k of other whole types than int32: a length that int32 does not hold
counts like any other past the keys there are (all of them), one below zero like
zero, whatever its low 32 bits are.

CPU: the binding's conversions.  GPU: calls with such lengths.
"""
import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from exact_io_aware_tiled_gb300 import _lib, _ops
from tests import test_diff, test_prefix

TOP, LOW = 2 ** 31 - 1, -2 ** 31
WIDE = [0, 5, TOP, 2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 63 - 1]


def lens_of(t):
    return _ops._lens(t, t.numel(), torch.device("cpu"))


def aux_of(t):
    return _lib._aux(t, None, torch.empty(t.numel(), 1, 1, 64))[0]


@pytest.mark.parametrize("conv", [lens_of, aux_of])
def test_wide_whole_numbers(conv):
    t = torch.tensor(WIDE + [-1, LOW, LOW - 1, -2 ** 63], dtype=torch.int64)
    got = conv(t)
    assert got.dtype == torch.int32 and got.is_contiguous()
    assert got.tolist() == [0, 5, TOP, TOP, TOP, TOP, TOP, -1, LOW, LOW, LOW]
    assert t.tolist()[3] == 2 ** 31                                # the caller's tensor stays
    assert conv(torch.tensor([0, 7, 2 ** 31, 2 ** 32 - 1], dtype=torch.uint32)).tolist() == [0, 7, TOP, TOP]
    assert conv(torch.tensor([0, 7, 2 ** 32, 2 ** 63, 2 ** 64 - 1], dtype=torch.uint64)).tolist() == [0, 7, TOP, TOP, TOP]
    assert conv(t.view(-1, 1).expand(-1, 2)[:, 0]).tolist() == got.tolist()      # not contiguous


@pytest.mark.parametrize("conv", [lens_of, aux_of])
@pytest.mark.parametrize("dtype", [torch.int8, torch.uint8, torch.int16, torch.int32])
def test_narrow_whole_numbers(conv, dtype):
    assert conv(torch.tensor([0, 1, 127], dtype=dtype)).tolist() == [0, 1, 127]


@pytest.mark.gpu
def test_calls():
    wide = torch.tensor([2 ** 31, 2 ** 32, 40, -2 ** 32 + 9], device="cuda")
    full = torch.tensor([10 ** 6, 10 ** 6, 40, 0], device="cuda", dtype=torch.int32)
    for P in (90, 0):
        x = test_prefix.inputs(4, 4, 2, 1, P, 50, 64, "bf16", 2)
        want = fa.prefix_fwd(*x, full)
        for t in (wide, torch.tensor([2 ** 31, 2 ** 32 - 1, 40, 0], dtype=torch.uint32, device="cuda")):
            got = fa.prefix_fwd(*x, t)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q, k, v, lam, do = test_diff.inputs(4, 2, 2, 70, "bf16", 3)
    got, want = (fa.diff_fwd(q, k, v, lam, seqlens_k=t) for t in (wide, full))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got, want = (fa.diff_bwd(q, k, v, lam, want[0], want[2], do, want[1], seqlens_k=t) for t in (wide, full))
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    q, k, v = (torch.randn(4, 2, 70, 64, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    got, want = (fa.fwd(q, k, v, seqlens_k=t) for t in (wide, full))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
