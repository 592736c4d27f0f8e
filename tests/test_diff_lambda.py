"""Gradients of differential attention where lambda is large, of either sign, or
of different size from head to head, checked for each map by itself.

The exact dS_1 = P_1 o (dP - D_1) does not depend on lambda.  Formed as dO . O +
lambda dO . O_2 from rounded outputs, D_1 would be off by |lambda| u times
|dO| |O_2|; head pairs with |lambda| > 2 sum P_1 o dP in float32 instead.

Tolerances, relative Frobenius per head and map, u = eps / 2 of the dtype:
* map 1, |lambda| > 2: dS_1 is rounded once (u), the result once (u), the rest is
  float32: 2u;
* everything else as in test_diff.py: 4u.
"""
import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from tests.test_diff import DT, inputs, plain, rel
from tests.test_operator_ranges import Field

pytestmark = pytest.mark.gpu


def run(B, H, Hkv, N, dtype, lam, seed=0, lens=None, **mask):
    q, k, v, _, do = inputs(B, H, Hkv, N, dtype, seed)
    lam = torch.tensor(lam, device="cuda")
    sl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse, o2 = fa.diff_fwd(q, k, v, lam, seqlens_k=sl, **mask)
    g = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, seqlens_k=sl, **mask)
    assert fa.check_status(fa.diff_bwd.last_workspace) == 0
    return (q, k, v, lam, do), g, plain(q, k, v, lam, do, lens=sl, **mask)


def check(x, g, want, dtype):
    lam, Hkv = x[3], x[2].shape[1]
    u = torch.finfo(DT[dtype]).eps / 2
    dq, dk, dv, dlam = want[4]
    group = lam.numel() // Hkv
    for h in range(lam.numel()):
        tol = 2 * u if abs(float(lam[h])) > 2 else 4 * u
        assert rel(g[0][:, 2 * h], dq[:, 2 * h]) <= tol, ("dq1", h, float(lam[h]), rel(g[0][:, 2 * h], dq[:, 2 * h]) / u)
        assert rel(g[0][:, 2 * h + 1], dq[:, 2 * h + 1]) <= 4 * u, ("dq2", h)
    for h in range(Hkv):
        tol = 2 * u if bool((lam[h * group:(h + 1) * group].abs() > 2).all()) else 4 * u
        assert rel(g[1][:, 2 * h], dk[:, 2 * h]) <= tol, ("dk1", h, rel(g[1][:, 2 * h], dk[:, 2 * h]) / u)
        assert rel(g[1][:, 2 * h + 1], dk[:, 2 * h + 1]) <= 4 * u, ("dk2", h)
        assert rel(g[2][:, h], dv[:, h]) <= 4 * u, ("dv", h)
    err = (g[3].double() - dlam).abs()
    assert bool((err <= 1e-5 * want[5] + 1e-6).all()), float((err / want[5]).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lam", [2.0, -2.0, 2.5, -4.0, 10.0, -10.0, 100.0, -100.0])
def test_one_lambda(dtype, lam):
    x, g, want = run(2, 2, 1, 257, dtype, [lam, lam], seed=1, causal=True)
    check(x, g, want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hkv,lam", [(4, 4, [0.5, -30.0, 2.0, 8.0]), (4, 2, [16.0, -3.0, 0.0, 50.0]),
                                       (3, 1, [-5.0, 0.7, 20.0])])
@pytest.mark.parametrize("N,mask", [(2, dict()), (63, dict(causal=True)), (64, dict()), (129, dict(causal=True)),
                                    (300, dict(causal=True, window=100)), (300, dict(lens=[300, 0, 171])),
                                    (257, dict(causal=True, window=70, lens=[40, 257, 64])), (200, dict(scale=0.3))])
def test_heads_and_masks(dtype, H, Hkv, lam, N, mask):
    x, g, want = run(3, H, Hkv, N, dtype, lam, seed=N, **mask)
    check(x, g, want, dtype)


def test_many_heads():
    # more heads than are looked at together, one of them large
    H = 150
    lam = [0.3] * H
    lam[140] = -40.0
    x, g, want = run(1, H, H, 70, "bf16", lam, seed=4, causal=True)
    check(x, g, want, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_visible_key(dtype):
    # P_1 = 1 up to the exponential's and the logsumexp's 2^-18: dS_1 is that times dP
    x, g, want = run(2, 2, 2, 150, dtype, [100.0, -100.0], seed=5, causal=True, window=1)
    q, k, v, lam, do = x
    dp = (do.double().abs() * v.double().abs()).sum(-1, keepdim=True)
    assert bool((g[0][:, 0::2].double().abs() <= 2.0 ** -16 * 0.125 * dp * k[:, 0::2].double().abs()).all())
    assert bool((g[1][:, 0::2].double().abs() <= 2.0 ** -16 * 0.125 * dp * q[:, 0::2].double().abs()).all())


def test_rows_behind_the_sequences_may_hold_nan():
    q, k, v, _, do = inputs(3, 2, 1, 300, "bf16", 3)
    lam = torch.tensor([30.0, -7.0], device="cuda")
    lens = torch.tensor([0, 77, 256], dtype=torch.int32).cuda()
    o, lse, o2 = fa.diff_fwd(q, k, v, lam, seqlens_k=lens)
    want = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, seqlens_k=lens)
    for b, n in enumerate(lens.tolist()):
        k[b, :, n:] = float("nan")
        v[b, :, n:] = float("inf")
        v[b, :, n + 1:] = float("nan")
    got = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, seqlens_k=lens)
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    assert rel(got[0], want[0].double()) <= 2.0 ** -8


def test_strides_repeats_and_graph():
    bnhd = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    q, k, v, _, do = inputs(2, 4, 2, 190, "bf16", 6)
    lam = torch.tensor([9.0, 0.4, -20.0, 3.0], device="cuda")
    o, lse, o2 = fa.diff_fwd(q, k, v, lam, causal=True)
    want = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True)
    got = fa.diff_bwd(bnhd(q), bnhd(k), bnhd(v), lam, o, o2, bnhd(do), lse, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True)
    for _ in range(3):
        for t in c:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(c[1:], want[1:]))
    # a replay takes the lambda that is there then
    lam.mul_(0.01)
    o, lse2, o2b = fa.diff_fwd(q, k, v, lam, causal=True, out=(o, lse, o2))
    graph.replay()
    want = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(c[1:], want[1:]))


@pytest.mark.parametrize("dim", [0, 1])
def test_offsets_pass_32_bits(dim):
    f = Field()
    # two sequences of one pair, or the two maps of one pair (v and dO then have one head)
    q, k, v, _, do = inputs(2 if dim == 0 else 1, 1, 1, 200, "bf16", 3)
    lam = torch.tensor([-12.0], device="cuda")
    far = (lambda t: f.copy(t, dim) if t.shape[dim] == 2 else t)
    o, lse, o2 = fa.diff_fwd(q, k, v, lam, causal=True)
    want = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True)
    x = [far(t) for t in (q, k, v)]
    grads = [f.empty_like(t, dim) if t.shape[dim] == 2 else torch.empty_like(t) for t in (q, k, v)]
    got = fa.diff_bwd(*x, lam, o, o2, far(do), lse, causal=True, out=(*grads, torch.empty_like(lam)))
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    assert rel(got[0], want[0].double()) <= 1e-4


def test_many_sequences_of_one_token():
    B = 70000
    q, k = (torch.randn(B, 2, 1, 64, device="cuda", dtype=torch.float16) for _ in range(2))
    v, do = (torch.randn(B, 1, 1, 128, device="cuda", dtype=torch.float16) for _ in range(2))
    lam = torch.tensor([5.0], device="cuda")
    o, lse, o2 = fa.diff_fwd(q, k, v, lam)
    dq, dk, dv, _ = fa.diff_bwd(q, k, v, lam, o, o2, do, lse)
    # one key: dS_1 is 2^-18 (P_1 against 1) of dP; each weight is rounded, and their difference is
    dp = (do.double().abs() * v.double().abs()).sum(-1, keepdim=True)
    assert bool((dq[:, :1].double().abs() <= 2.0 ** -16 * 0.125 * dp * k[:, :1].double().abs() + 2.0 ** -24).all())
    assert bool((dk[:, :1].double().abs() <= 2.0 ** -16 * 0.125 * dp * q[:, :1].double().abs() + 2.0 ** -24).all())
    ref = do.double() * -4.0
    assert bool(((dv.double() - ref).abs() <= 3 * 2.0 ** -11 * do.double().abs() * 6 + 2.0 ** -24).all())


def test_two_calls_at_once():
    q, k, v, _, do = inputs(3, 4, 2, 500, "bf16", 8)
    lam = torch.tensor([0.5, -30.0, 4.0, 1.0], device="cuda")
    o, lse, o2 = fa.diff_fwd(q, k, v, lam, causal=True)
    want = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True)
    torch.cuda.synchronize()
    got = [fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True, stream=torch.cuda.Stream()) for _ in range(6)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g[1:], want[1:])) and rel(g[0], want[0].double()) <= 2.0 ** -8
