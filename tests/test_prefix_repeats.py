"""Results of the shared prefix do not depend on the order in which its work items
are claimed: persistent CTAs run several ragged items each, in an order that
varies with the batch's order, with what else runs and with chance.

Every row's result is held, bit for bit, to the same call on the batch in another
order, repeated and beside other work.  The batches have more items than the GPU
has CTAs, of different lengths, so that an item meets its CTA's ring of stages at
every place.
"""
import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from tests import test_prefix

pytestmark = pytest.mark.gpu


def batch(B, H, Hkv, T, P, M, d, seed):
    x = test_prefix.inputs(B, H, Hkv, T, P, M, d, "bf16", seed)
    lens = (torch.arange(B, device="cuda", dtype=torch.int32) * 197 + 31) % (M + 1)
    return x, lens


CASES = [(64, 16, 16, 1, 2000, 1024, 64),      # one row: four key groups
         (96, 8, 8, 1, 0, 1500, 128),          # without a prefix
         (48, 64, 4, 2, 500, 1000, 64),        # 32 rows: two key groups
         (24, 48, 16, 40, 0, 700, 64)]         # 120 rows: 64-row tiles beside shorter ones


@pytest.mark.parametrize("case", CASES)
def test_any_order_of_the_batch(case):
    (q, kp, vp, k, v), lens = batch(*case, seed=1)
    want = fa.prefix_fwd(q, kp, vp, k, v, lens)
    assert fa.check_status(fa.prefix_fwd.last_workspace) == 0
    for seed in range(4):
        at = torch.randperm(case[0], generator=torch.Generator().manual_seed(seed)).cuda()
        o, lse = fa.prefix_fwd(q[at], kp, vp, k[at], v[at], lens[at])
        assert torch.equal(lse, want[1][at]) and torch.equal(o, want[0][at])


@pytest.mark.parametrize("case", CASES)
def test_repeats_beside_other_work(case):
    x, lens = batch(*case, seed=2)
    want = fa.prefix_fwd(*x, lens)
    a = torch.randn(2048, 2048, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            for _ in range(4):
                a @ a
        o, lse = fa.prefix_fwd(*x, lens)
        assert torch.equal(lse, want[1]) and torch.equal(o, want[0])
    torch.cuda.synchronize()


def test_differential_step_in_any_order():
    B, H, Hkv = 64, 8, 8
    (q, kp, vp, k, v), lam = test_prefix.diff_inputs(B, H, Hkv, 1, 0, 1024, "bf16", 3)
    lens = (torch.arange(B, device="cuda", dtype=torch.int32) * 197 + 31) % 1025
    want = fa.prefix_fwd(q, None, None, k, v, lens, lam=lam)
    at = torch.arange(B - 1, -1, -1, device="cuda")
    o, lse = fa.prefix_fwd(q[at], None, None, k[at], v[at], lens[at], lam=lam)
    assert torch.equal(lse, want[1][at]) and torch.equal(o, want[0][at])
