"""Rotary positions, differential attention and the shared prefix at the ends of
their ranges: rows more than 2^32 elements apart, two calls at once, many
sequences of one token.

Each call is held to the same call on compact tensors (itself tested against the
plain forms): layouts and neighbours must not change a bit, dQ apart, which is
accumulated in an order that varies.
"""
import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from tests import test_diff, test_prefix

pytestmark = pytest.mark.gpu
FAR = 2 ** 32 + 64                       # elements


class Field:
    """One buffer in which tensors lie with `dim` FAR elements apart, side by side in the rest."""

    def __init__(self, dtype=torch.bfloat16):
        self.buf = torch.empty(FAR + (1 << 26), device="cuda", dtype=dtype)
        self.at = 0

    def empty_like(self, t, dim):
        assert t.shape[dim] == 2
        inner = [n for i, n in enumerate(t.shape) if i != dim]
        strides, s = [], 1
        for n in reversed(inner):
            strides.insert(0, s)
            s *= n
        strides.insert(dim, FAR)
        out = self.buf.as_strided(t.shape, strides, self.at)
        self.at += -(-s // 64) * 64
        assert self.at <= 1 << 26
        return out

    def copy(self, t, dim):
        return self.empty_like(t, dim).copy_(t)


@pytest.mark.parametrize("dim", [0, 1])
def test_rope_offsets_pass_32_bits(dim):
    f = Field()
    q, k = (torch.randn(2, 2, 70, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    freq, m = fa.rope_frequencies(64)
    want = fa.rope(q, k, inv_freq=freq, mscale=m, start=9)
    got = fa.rope(f.copy(q, dim), f.copy(k, dim), inv_freq=freq, mscale=m, start=9,
                  out=(f.empty_like(q, dim), f.empty_like(k, dim)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dim", [0, 1])
def test_differential_offsets_pass_32_bits(dim):
    f = Field()
    # two sequences of one pair, or the two maps of one pair (v and o then have one head)
    q, k, v, lam, do = test_diff.inputs(2 if dim == 0 else 1, 1, 1, 200, "bf16", 3)
    far = (lambda t: f.copy(t, dim) if t.shape[dim] == 2 else t)
    o, lse, o2 = fa.diff_fwd(q, k, v, lam, causal=True)
    g = fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True)
    x = [far(t) for t in (q, k, v)]
    outs = [f.empty_like(t, dim) if t.shape[dim] == 2 else torch.empty_like(t) for t in (o, o2)]
    got = fa.diff_fwd(*x, lam, causal=True, out=(outs[0], torch.empty_like(lse), outs[1]))
    assert torch.equal(got[0], o) and torch.equal(got[1], lse) and torch.equal(got[2], o2)
    grads = [f.empty_like(t, dim) if t.shape[dim] == 2 else torch.empty_like(t) for t in (q, k, v)]
    got = fa.diff_bwd(*x, lam, outs[0], outs[1], far(do), lse, causal=True, out=(*grads, torch.empty_like(lam)))
    assert all(torch.equal(a, b) for a, b in zip(got[1:], g[1:]))
    assert test_diff.rel(got[0], g[0].double()) <= 1e-4


@pytest.mark.parametrize("dim", [0, 1])
def test_caches_offsets_pass_32_bits(dim):
    f = Field()
    q, kp, vp, k, v = test_prefix.inputs(2, 4, 2, 3, 300, 500, 128, "bf16", 5)
    lens = torch.tensor([500, 77], device="cuda", dtype=torch.int32)
    want = fa.prefix_fwd(q, kp, vp, k, v, lens)
    heads = (lambda t: f.copy(t, 0))                  # the prefix's K/V heads
    got = fa.prefix_fwd(q, heads(kp), heads(vp), f.copy(k, dim), f.copy(v, dim), lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    far_q = f.copy(q[:, :2], dim)                     # two heads, so that either dimension can be far
    out = f.empty_like(far_q, dim)
    want = fa.prefix_fwd(q[:, :2], kp, vp, k, v, lens)
    got = fa.prefix_fwd(far_q, kp, vp, k, v, lens, out=(out, torch.empty_like(want[1])))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_cache_of_more_than_2_32_elements():
    # the last keys of one long row: 2^25 + 100 of 128 columns
    M, d = 2 ** 25 + 100, 128
    k = torch.zeros(1, 1, M, d, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    q = torch.ones(1, 1, 1, d, device="cuda", dtype=torch.bfloat16)
    k[0, 0, M - 2] = 4.0                              # score 4 sqrt(128) = 45: the others weigh e^-45 each
    v[0, 0, M - 2], v[0, 0, M - 1] = 3.0, 9.0
    o, lse = fa.prefix_fwd(q, None, None, k, v, torch.tensor([M], device="cuda", dtype=torch.int32))
    assert fa.check_status(fa.prefix_fwd.last_workspace) == 0
    # 2^25 e^-45.25 < 2^-40
    assert bool((o == 3.0).all()) and abs(float(lse) - 4 * 128 ** 0.5) <= 2.0 ** -18 * 46
    # as a prefix
    o, lse = fa.prefix_fwd(q.repeat(1, 1, 40, 1), k[0], v[0], None, None, torch.zeros(1, device="cuda", dtype=torch.int32))
    assert bool((o == 3.0).all()) and bool(((lse - 4 * 128 ** 0.5).abs() <= 2.0 ** -18 * 46).all())


def test_two_calls_at_once():
    a = test_diff.inputs(4, 4, 2, 700, "bf16", 1)
    b = test_prefix.inputs(40, 8, 2, 1, 30000, 300, 128, "bf16", 2)
    lens = (torch.arange(40, device="cuda", dtype=torch.int32) * 7) % 301

    def train(stream):
        q, k, v, lam, do = a
        o, lse, o2 = fa.diff_fwd(q, k, v, lam, causal=True, stream=stream)
        return [o, lse, o2] + list(fa.diff_bwd(q, k, v, lam, o, o2, do, lse, causal=True, stream=stream))

    def decode(stream):
        return list(fa.prefix_fwd(*b, lens, stream=stream))

    here = torch.cuda.current_stream()
    want = [train(here), decode(here)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(3):
        for i, s in enumerate(streams):
            got.append((i % 2, (train, decode)[i % 2](s)))
    torch.cuda.synchronize()
    for kind, outs in got:
        for i, (x, y) in enumerate(zip(outs, want[kind])):
            if kind == 0 and i == 3:
                assert test_diff.rel(x, y.double()) <= 1e-4
            else:
                assert torch.equal(x, y)


def test_many_sequences_of_one_token():
    B = 70000                                         # more than a grid's second dimension takes
    q, k, v, lam, do = (torch.randn(s, device="cuda", dtype=t) for s, t in (
        ((B, 2, 1, 64), torch.float16), ((B, 2, 1, 64), torch.float16), ((B, 1, 1, 128), torch.float16),
        ((1,), torch.float32), ((B, 1, 1, 128), torch.float16)))
    o, lse, o2 = fa.diff_fwd(q, k, v, lam)
    u = 2.0 ** -11
    ref = v.double() * (1 - lam.double())
    assert bool(((o.double() - ref).abs() <= 3 * u * v.double().abs() * (1 + lam.double().abs()) + 2.0 ** -24).all())
    dq, dk, dv, dlam = fa.diff_bwd(q, k, v, lam, o, o2, do, lse)
    # one key: the weights are 1 and lam; each is rounded, and their difference is
    ref = do.double() * (1 - lam.double())
    assert bool(((dv.double() - ref).abs() <= 3 * u * do.double().abs() * (1 + lam.double().abs()) + 2.0 ** -24).all())
    want = -(do.double() * v.double()).sum()
    assert abs(float(dlam) - float(want)) <= 1e-5 * float((do.double() * v.double()).sum(-1).norm())
    lens = torch.ones(B, device="cuda", dtype=torch.int32)
    o, _ = fa.prefix_fwd(do, None, None, k.new_zeros(B, 1, 1, 128), v, lens)
    assert torch.equal(o, v)
    freq, _ = fa.rope_frequencies(64)
    r = fa.rope(q, inv_freq=freq, positions=torch.zeros(B, 1, device="cuda", dtype=torch.int32))
    assert torch.equal(r, q)
