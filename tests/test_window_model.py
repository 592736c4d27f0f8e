"""The operators of a model with a sliding window as a program uses them together.

* training: q, k of a fused projection normalised and rotated, window attention with first keys forward and backward,
  the gradients back through rotation and norm;
* serving: a prompt written into the 8-bit cache in chunks and attended to from there, then single tokens, step after
  step, eagerly and as one replayed graph, with pages that have left the window taken away.

Both against 64-bit forms that start from the same 16-bit intermediates, so each rounding to 16 bits counts once,
u = eps / 2: attention's gradients 4u (tests/test_sinks.py), the norm's rounding u more.
"""
import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from tests import test_cache8, test_norm_rope, test_sinks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load()


@pytest.mark.parametrize("dtype,d,interleaved", [("bf16", 64, False), ("f16", 128, True)])
def test_a_training_step(dtype, d, interleaved):
    B, H, Hkv, N, w, s = 2, 6, 2, 700, 90, 4
    g = torch.Generator(device="cuda").manual_seed(21)
    proj = torch.randn((B, N, (H + 2 * Hkv) * d), generator=g, device="cuda").to(test_sinks.DT[dtype])
    q, k, v = (t.view(B, N, -1, d).transpose(1, 2) for t in proj.split([H * d, Hkv * d, Hkv * d], -1))
    do = torch.randn((B, H, N, d), generator=g, device="cuda").to(q.dtype)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    inv, m = fa.rope_frequencies(d, scaling="yarn", factor=4.0, original_len=256)
    kw = dict(q_weight=wq, k_weight=wk, inv_freq=inv, mscale=m, interleaved=interleaved)
    mask = dict(causal=True, window=w, sinks=s)

    qn, kn = fa.norm_rope(q, k, out=(torch.empty(B, H, N, d, device="cuda", dtype=q.dtype),
                                     torch.empty(B, Hkv, N, d, device="cuda", dtype=q.dtype)), **kw)
    vc = v.contiguous()
    o, lse = fa.fwd(qn, kn, vc, **mask)
    dqn, dkn, dv = fa.bwd(qn, kn, vc, o, do, lse, **mask)
    dq, dk, dwq, dwk = fa.norm_rope_bwd(q, k, dqn, dkn, **kw)

    pos = torch.arange(N, device="cuda")[None, None]
    for x, y, wt in ((q, qn, wq), (k, kn, wk)):
        test_norm_rope.near(y, *test_norm_rope.plain(x, wt, None, 1e-6, pos, inv, m, interleaved), dtype, -19)
    want = test_sinks.plain(qn, kn, vc, do, w, s)
    test_sinks.check((o, lse, dqn, dkn, dv), want, dtype)
    # through the norm, from the exact gradients of the attention
    u = torch.finfo(q.dtype).eps / 2
    for x, wt, exact, got, gw in ((q, wq, want[3], dq, dwq), (k, wk, want[4], dk, dwk)):
        gx, _, dw, _ = test_norm_rope.plain(x, wt, exact, 1e-6, pos, inv, m, interleaved)
        assert test_sinks.rel(got, gx) <= 5 * u
        assert test_sinks.rel(gw, dw) <= 4 * u


def pages_for(B, width, seed):
    P = B * width + 2
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(seed))[:B * width]
    return P, perm.view(B, width).to(torch.int32).cuda()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_a_prompt_and_decoding_steps(graph, d, page):
    B, H, Hkv, window, sinks, width = 3, 8, 2, 70, 4, 512 // page
    g = torch.Generator(device="cuda").manual_seed(22)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    inv, m = fa.rope_frequencies(d)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    P, table = pages_for(B, width, 23)
    kc, vc = (torch.full((P, Hkv, page, d), float("nan"), device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((P, Hkv), float("nan"), device="cuda") for _ in range(2))
    cache = (kc, vc, ks, vs, table)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step(q, k, v):
        """New tokens normalised, rotated, appended, and what they attend to."""
        T = q.shape[2]
        at = lens[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)
        lens.add_(T)
        qn, kn = fa.norm_rope(q, k, q_weight=wq, k_weight=wk, inv_freq=inv, positions=at, mscale=m)
        fa.cache8_append(kn, v, *cache, lens)
        return qn, fa.cache8_fwd(qn, *cache, lens, window=window, sinks=sinks)

    def check(qn, got):
        u8 = tuple(t.view(torch.uint8) for t in (kc, vc))
        test_cache8.check(got, test_cache8.plain_fwd(qn, u8 + (ks, vs, table), lens, page, window, sinks), "bf16")

    for T in (37, 120, 1, 64):                              # a prompt in chunks
        check(*step(r(B, H, T, d), r(B, Hkv, T, d), r(B, Hkv, T, d)))
    # what the cache holds, read back for a program that attends to it in 16 bits: the last chunk's keys near their own
    k16, v16 = fa.cache8_read(*cache, lens, rows=222)
    assert bool(torch.isfinite(k16).all()) and bool((k16[:, :, :222].abs().amax(-1) > 0).all())
    # pages before the window, but for the first, leave
    gone = (222 - window) // page
    before = fa.cache8_fwd(q0 := r(B, H, 1, d), *cache, lens, window=window, sinks=sinks)
    table[:, 1:gone] = -1
    after = fa.cache8_fwd(q0, *cache, lens, window=window, sinks=sinks)
    assert all(torch.equal(a, b) for a, b in zip(before, after))

    q, k, v = r(B, H, 1, d), r(B, Hkv, 1, d), r(B, Hkv, 1, d)
    captured = None
    if graph:
        saved = [t.clone() for t in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs, lens)]
        step(q, k, v)
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            out = step(q, k, v)
        for t, c in zip((kc.view(torch.uint8), vc.view(torch.uint8), ks, vs, lens), saved):
            t.copy_(c)
    for _ in range(40):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        if graph:
            captured.replay()
        else:
            out = step(q, k, v)
        check(*out)
    assert lens.tolist() == [262] * B


def test_values_through_the_cache_keep_e4m3s_precision():
    # a row written and read: off by half a step of E4M3, 2^-4, of what is within 2^-6 .. 448 of its page's scale
    B, Hkv, T, d, page = 2, 2, 100, 64, 32
    P, table = pages_for(B, 4, 24)
    g = torch.Generator(device="cuda").manual_seed(25)
    x = torch.randn((B, Hkv, T, d), generator=g, device="cuda").bfloat16()
    kc, vc = (torch.zeros((P, Hkv, page, d), device="cuda", dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.zeros((P, Hkv), device="cuda") for _ in range(2))
    ln = torch.full((B,), T, device="cuda", dtype=torch.int32)
    fa.cache8_append(x, 3 * x, kc, vc, ks, vs, table, ln)
    k, v = fa.cache8_read(kc, vc, ks, vs, table, ln, rows=T)
    for got, want in ((k, x), (v, 3 * x)):
        top = want.float().abs().amax()
        err = (got.double() - want.double()).abs()
        assert bool((err <= 2.0 ** -4 * want.double().abs() + 2.0 ** -10 * top.double() / 224).all())


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_a_prompt_in_chunks_reads_back_as_it_was_normed(d, page):
    # every row of the cache against the normed key and the value that it was written from: a rounding to E4M3 (2^-4
    # relative, 2^-10 of the page's scale below its normal range), and one more for each later chunk in the row's page
    B, H, Hkv, width = 3, 4, 2, 512 // page
    g = torch.Generator(device="cuda").manual_seed(26)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    inv, m = fa.rope_frequencies(d)
    wk = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    P, table = pages_for(B, width, 27)
    kc, vc = (torch.full((P, Hkv, page, d), float("nan"), device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((P, Hkv), float("nan"), device="cuda") for _ in range(2))
    cache = (kc, vc, ks, vs, table)
    chunks = (37, 120, 1, 64)
    start = torch.tensor([0, 5, 200], dtype=torch.int32, device="cuda")      # the sequences begin apart
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    keys, values, times = [], [], []
    for i, T in enumerate(chunks):
        at = lens[:, None] + start[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)
        first = sum(chunks[:i])
        lens.add_(T)
        q, k, v = r(B, H, T, d), r(B, Hkv, T, d) * 2.0 ** i, r(B, Hkv, T, d) * 2.0 ** i      # scales grow
        kn = fa.norm_rope(q, k, k_weight=wk, inv_freq=inv, positions=at, mscale=m)[1]
        fa.cache8_append(kn, v, *cache, lens)
        keys.append(kn)
        values.append(v)
        for j in range(first, first + T):
            end = (j // page + 1) * page
            times.append(1 + sum(sum(chunks[:c]) < end for c in range(i + 1, len(chunks))))
    N = sum(chunks)
    n = torch.tensor(times, device="cuda", dtype=torch.float64)[:, None]
    got = fa.cache8_read(*cache, lens, rows=N)
    for x, want, scale in zip(got, (keys, values), (ks, vs)):
        want = torch.cat(want, 2).double()
        s = scale[table.long()].transpose(1, 2).repeat_interleave(page, 2)[:, :, :N, None].double()
        bound = ((1 + 2.0 ** -4) ** n - 1) * want.abs() + n * 2.0 ** -10 * s
        assert bool(((x.double() - want).abs() <= bound).all())
        for other in (want.roll(1, 2), want.roll(1, 1), want.roll(1, 0)):      # rows, heads, sequences of others do not pass
            assert not bool(((x.double() - other).abs() <= bound).all(-1).any())
