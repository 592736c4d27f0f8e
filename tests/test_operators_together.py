"""The operators as a program uses them together.

* training: q, k of a fused projection rotated by their positions, differential
  attention forward and backward, the gradients rotated back;
* serving: keys rotated and appended to the caches, attention over the shared
  prefix and the caches, step after step, eagerly and as one replayed graph.

Both against 64-bit forms that start from the same 16-bit intermediates, so each
rounding to 16 bits counts once: u = eps / 2.  Gradients: 4u for the attention's
(tests/test_diff.py), u for the rotation's rounding.  Outputs: as in
tests/test_prefix.py.
"""
import pytest
import torch

import exact_io_aware_tiled_gb300 as fa
from tests import test_diff, test_prefix, test_rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fa.build()
    fa.load()


@pytest.mark.parametrize("interleaved,scaling", [(False, "none"), (True, "yarn")])
def test_a_training_step(interleaved, scaling):
    B, H, Hkv, N = 2, 4, 2, 333
    g = torch.Generator(device="cuda").manual_seed(5)
    width = 2 * H * 64 + 2 * Hkv * 64 + Hkv * 128
    proj = torch.randn((B, N, width), generator=g, device="cuda").bfloat16()       # a fused projection
    q = proj[..., :2 * H * 64].view(B, N, 2 * H, 64).transpose(1, 2)
    k = proj[..., 2 * H * 64:2 * (H + Hkv) * 64].view(B, N, 2 * Hkv, 64).transpose(1, 2)
    v = proj[..., 2 * (H + Hkv) * 64:].view(B, N, Hkv, 128).transpose(1, 2)
    lam = torch.rand(H, generator=g, device="cuda") * 0.5 + 0.2
    do = torch.randn((B, H, N, 128), generator=g, device="cuda").bfloat16()
    inv, m = fa.rope_frequencies(64, scaling=scaling, factor=4.0, original_len=128)
    pos = (torch.arange(N, device="cuda")[None] + torch.tensor([[0], [777]], device="cuda"))
    kw = dict(inv_freq=inv, positions=pos, mscale=m, interleaved=interleaved)

    qr, kr = fa.rope(q, k, **kw)
    o, lse, o2 = fa.diff_fwd(qr, kr, v, lam, causal=True)
    dqr, dkr, dv, dlam = fa.diff_bwd(qr, kr, v, lam, o, o2, do, lse, causal=True)
    dq, dk = fa.rope(dqr, dkr, backward=True, **kw)

    for x, y in ((q, qr), (k, kr)):
        test_rope.check(y, *test_rope.plain(x, pos.cpu(), inv.cpu().numpy(), m, interleaved, False))
    want = test_diff.plain(qr, kr, v, lam, do, causal=True)
    test_diff.check_fwd((o, lse, o2), want, "bf16")
    test_diff.check_grads((dqr, dkr, dv, dlam), want, "bf16")
    u = 2.0 ** -8
    for got, exact in ((dq, want[4][0]), (dk, want[4][1])):
        turned = test_rope.plain(exact, pos.cpu(), inv.cpu().numpy(), m, interleaved, True)[0].cuda()
        assert test_diff.rel(got, turned) <= 5 * u
    # in place, into the projection's own memory, as a training program would
    fa.rope(q, k, out=(q, k), **kw)
    assert torch.equal(q, qr) and torch.equal(k, kr)


@pytest.mark.parametrize("graph", [False, True])
def test_decoding_steps(graph):
    B, H, Hkv, P, M, d, steps, T = 5, 8, 2, 300, 40, 64, 12, 2
    g = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    inv, m = fa.rope_frequencies(d, scaling="ntk", factor=2.0)
    kp, vp = r(Hkv, P, d), r(Hkv, P, d)
    kp = fa.rope(kp[None], inv_freq=inv)[0]                                # the prefix at positions 0 .. P - 1
    kc, vc = torch.full((B, Hkv, M, d), float("nan"), device="cuda").bfloat16(), torch.empty(0)
    vc = kc.clone()
    lens = torch.tensor([0, 3, 7, 1, 15], dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens.tolist()):                                  # what each sequence has said so far
        kc[b, :, :n], vc[b, :, :n] = r(Hkv, n, d), r(Hkv, n, d)
    q, k, v = r(B, H, T, d), r(B, Hkv, T, d), r(B, Hkv, T, d)
    rows = torch.arange(B, device="cuda")[:, None]

    def step():
        """Rotate the new tokens, append them, attend; the lengths grow by T."""
        at = lens.long()[:, None] + torch.arange(T, device="cuda")         # own rows of the new tokens
        qr, kr = fa.rope(q, k, inv_freq=inv, positions=at + P)
        kc[rows, :, at] = kr.transpose(1, 2)
        vc[rows, :, at] = v.transpose(1, 2)
        lens.add_(T)
        return qr, fa.prefix_fwd(qr, kp, vp, kc, vc, lens)

    captured = None
    if graph:
        saved = kc.clone(), vc.clone(), lens.clone()
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            out = step()
        for t, s in zip((kc, vc, lens), saved):
            t.copy_(s)
    for _ in range(steps):
        q.copy_(r(B, H, T, d))
        k.copy_(r(B, Hkv, T, d))
        v.copy_(r(B, Hkv, T, d))
        if graph:
            captured.replay()
        else:
            out = step()
        qr, got = out
        test_prefix.check(got, test_prefix.plain(qr, kp, vp, kc, vc, lens), "bf16")
