"""Rotary positions with frequencies that are not finite: the cosine and sine of
such an angle are NaN, at position zero too (0 x infinity), so the pair's columns
are; every other column keeps its bits."""
import pytest
import torch

import exact_io_aware_tiled_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("rot", [64, 48, 42])
def test_non_finite_frequencies(dtype, interleaved, backward, rot):
    q, k = torch.randn(2, 3, 5, 64, device="cuda", dtype=dtype), torch.randn(2, 1, 5, 64, device="cuda", dtype=dtype)
    freq, _ = fa.rope_frequencies(rot)
    pos = torch.tensor([0, 1, -3, 100000, 7], device="cuda")
    kw = dict(positions=pos, mscale=1.25, interleaved=interleaved, backward=backward)
    want = fa.rope(q, k, inv_freq=freq, **kw)
    bad = freq.clone()
    where = {1: float("nan"), rot // 2 - 1: float("inf"), 8: float("-inf")}
    for i, f in where.items():
        bad[i] = f
    got = fa.rope(q, k, inv_freq=bad, **kw)
    cols = torch.zeros(64, dtype=torch.bool, device="cuda")
    for i in where:
        cols[[2 * i, 2 * i + 1] if interleaved else [i, rot // 2 + i]] = True
    for x, y in zip(got, want):
        assert bool(torch.isnan(x[..., cols]).all())
        assert torch.equal(x[..., ~cols], y[..., ~cols])
