"""Cases, inputs, plain forms and 64-bit values of three groups of operators that stand next to the attention
kernels: rotary positions, differential attention and attention over a shared prefix.

``rope``     q and k rotated by their positions (and the gradients rotated back).
``diff``     O = (softmax(tau Q1 K1^T) - lambda softmax(tau Q2 K2^T)) V per head pair, forward alone or forward
             and backward (dQ, dK, dV, dlambda).
``prefix``   T new tokens of each of B sequences attend to one prefix that all share and to their own cache rows.

With ``own`` false, ``run`` is the plain form: elementary torch operations in 32 bits (angles in 64), rounded once
at the end.  With ``own`` true it makes the framework's calls on the same state.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CAP = 1.8e12        # flop-equivalents (flops + 300 x bytes) no drawn case goes over


def _fa():
    import exact_io_aware_tiled_gb300 as fa
    return fa


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _rope(name, **kw):
    c = dict(op="rope", B=1, H=16, Hkv=16, N=1024, d=64, rot=64, dtype="bf16", interleaved=False, backward=False,
             base=10000.0, scaling="none", factor=1.0, orig=0, start=0, perseq=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _diff(name, **kw):
    c = dict(op="diff", B=1, H=8, Hkv=8, N=1024, dtype="bf16", causal=True, window=0, lo=-1, hi=-1, backward=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def _prefix(name, **kw):
    c = dict(op="prefix", B=8, H=16, Hkv=16, d=64, T=1, P=1024, M=256, lo=1, hi=256, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of 64 sequences at far, different positions of a context stretched eightfold: latency alone
        _rope("rope one token", B=64, N=1, scaling="yarn", factor=8.0, orig=16384, start=100000, perseq=True),
        # q and k of the GPT-2-medium training step
        _rope("rope gpt2-medium", B=64),
        # the gradients of a long ragged batch, grouped heads, a third of a wide head rotated, pairs interleaved
        _rope("rope back interleaved", B=3, H=32, Hkv=4, N=7001, d=128, rot=48, dtype="f16", interleaved=True,
              backward=True, scaling="linear", factor=4.0),
        # float32 training, odd length, stretched base
        _rope("rope f32 ntk", B=5, H=12, Hkv=12, N=2047, dtype="f32", scaling="ntk", factor=4.0),
        # a short prompt through one small layer: latency alone
        _diff("diff short prompt", H=4, Hkv=2, N=77, dtype="f16", backward=False),
        # GPT-2-medium width as 8 head pairs (2 x 64 for q and k, 128 for v): the training step
        _diff("diff gpt2-medium train", B=64),
        # BERT-large length, dense with padded sequences, fp16: the training step
        _diff("diff padded train", B=32, N=509, dtype="f16", causal=False, lo=0, hi=509),
        # a long prompt with a sliding window and grouped heads
        _diff("diff long window", B=1, H=8, Hkv=2, N=8191, window=1024, backward=False),
        # two sequences that share little: latency alone
        _prefix("prefix two sequences", B=2, P=129, M=33, hi=33),
        # GPT-2-medium heads, 64 sequences over a shared document, own caches of very different length
        _prefix("prefix 64 sequences", B=64, P=8193, M=1024, lo=1, hi=1024),
        # 128 sequences, 8 query heads per K/V head, wide heads, long prefix
        _prefix("prefix 128 grouped", B=128, H=16, Hkv=2, d=128, P=32769, M=2048, lo=0, hi=2047),
        # a 23,400-step day shared by 6 continuations of 5 tokens each, 12 heads, fp16
        _prefix("prefix five tokens", B=6, H=12, Hkv=12, T=5, P=23400, M=700, lo=5, hi=699, dtype="f16"),
    ]


def _cost(c):
    w = work(c)
    return w["flops"] + 300 * w["bytes"]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    while True:
        op = rng.choice(["rope", "diff", "prefix"])
        if op == "rope":
            d = rng.choice([64, 128])
            hkv = rng.choice([1, 2, 4, 8, 12])
            rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
            sc = rng.choice(["none", "linear", "ntk", "yarn"])
            c = _rope(None, B=log(1, 64), Hkv=hkv, H=hkv * rng.choice([1, 2, 4]), N=log(1, 9000), d=d, rot=rot,
                      dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), interleaved=rng.random() < 0.5,
                      backward=rng.random() < 0.4, base=rng.choice([10000.0, 500000.0]), scaling=sc,
                      factor=1.0 if sc == "none" else rng.choice([2.0, 4.0, 8.0]), orig=log(1024, 32768),
                      start=rng.choice([0, log(1, 1000000)]), perseq=rng.random() < 0.5)
        elif op == "diff":
            hkv = rng.choice([2, 3, 4, 8])
            n = log(2, 6000)        # one key alone has P = 1 and no gradient to compare
            causal = rng.random() < 0.7
            pad = rng.random() < 0.4
            c = _diff(None, B=log(1, 32), Hkv=hkv, H=hkv * rng.choice([1, 1, 2, 4]), N=n,
                      dtype=rng.choice(["bf16", "bf16", "f16"]), causal=causal,
                      window=log(2, n) if causal and rng.random() < 0.3 else 0, lo=0 if pad else -1,
                      hi=n if pad else -1, backward=rng.random() < 0.6)
            if c["B"] * c["H"] * n * n > 64 * 8 * 1024 * 1024:   # the plain form holds the score maps
                continue
        else:
            hkv = rng.choice([1, 2, 8, 12, 16])
            t = rng.choice([1, 1, 1, rng.randint(2, 9)])
            m = log(max(t, 2), 2048)
            c = _prefix(None, B=log(1, 128), Hkv=hkv, H=hkv * rng.choice([1, 1, 4, 8]), d=rng.choice([64, 128]), T=t,
                        P=rng.choice([0, log(1, 40000), log(100, 40000), log(100, 40000)]), M=m, lo=0,
                        hi=rng.randint(t, m), dtype=rng.choice(["bf16", "bf16", "f16"]))
            if c["B"] * c["H"] * c["T"] * (c["P"] + m) > 128 * 16 * 40000:
                continue
        if _cost(c) <= CAP:
            return c


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n lengths spread evenly over lo..hi (the same sum for every seed)."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64) if n > 1 else np.array([hi], dtype=np.int64)


def _freqs(c):
    """Inverse frequencies (float64) and the factor on cos and sin of a rotation of `rot` dimensions.

    none: base^(-2i/rot).  linear: divided by factor.  ntk: the base grows so that the slowest pair is slowed by
    factor and the fastest not at all.  yarn: pairs that turn more than 32 times within the original length stay,
    those that turn less than once are slowed by factor, a ramp between; cos and sin grow by 0.1 ln(factor) + 1."""
    rot, f = c["rot"], c["factor"]
    i = np.arange(rot // 2, dtype=np.float64)
    base = c["base"]
    if c["scaling"] == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2.0))
    inv = base ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        inv = inv / f
    if c["scaling"] == "yarn":
        def dim(turns):
            return rot * math.log(c["orig"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        inv = inv / f * ramp + inv * (1.0 - ramp)
        return inv, 0.1 * math.log(f) + 1.0
    return inv, 1.0


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng([seed, 7])
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = dict(c)
    B, H, Hkv = c["B"], c["H"], c["Hkv"]
    if c["op"] == "rope":
        N = c["N"]
        s["q"], s["k"] = normal(B, H, N, c["d"]), normal(B, Hkv, N, c["d"])
        inv, s["mscale"] = _freqs(c)
        s["inv_freq"] = torch.from_numpy(inv).cuda()
        pos = np.arange(N, dtype=np.int64) + c["start"]
        if c["perseq"]:
            pos = pos[None, :] + rng.integers(0, 1 + c["start"] // 2 + 64, size=(B, 1))
        s["positions"] = torch.from_numpy(pos.astype(np.int32)).cuda()
    elif c["op"] == "diff":
        N = c["N"]
        s["q"], s["k"], s["v"] = normal(B, 2 * H, N, 64), normal(B, 2 * Hkv, N, 64), normal(B, Hkv, N, 128)
        s["do"] = normal(B, H, N, 128)
        s["lam"] = torch.rand((H,), generator=g, device="cuda", dtype=torch.float32) * 0.7 + 0.1
        s["lens"] = None
        if c["hi"] >= 0:
            s["lens"] = torch.from_numpy(rng.permutation(_spread(c["lo"], c["hi"], B)).astype(np.int32)).cuda()
    else:
        d = c["d"]
        s["q"] = normal(B, H, c["T"], d)
        s["kp"], s["vp"] = normal(Hkv, c["P"], d), normal(Hkv, c["P"], d)
        s["k"], s["v"] = normal(B, Hkv, c["M"], d), normal(B, Hkv, c["M"], d)
        s["lens"] = torch.from_numpy(rng.permutation(_spread(c["lo"], c["hi"], B)).astype(np.int32)).cuda()
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def _plain_rope(s, x):
    """cos / sin of 64-bit angles, held in 32 bits; the rotation (or its transpose) in 32 bits."""
    rot = s["rot"]
    a = s["positions"].double()[..., None] * s["inv_freq"]                  # [N, rot/2] or [B, N, rot/2]
    cos, sin = (torch.cos(a) * s["mscale"]).float(), (torch.sin(a) * s["mscale"]).float()
    if a.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]                               # over the heads
    if s["backward"]:
        sin = -sin
    xf = x.float()
    y = xf.clone()
    if s["interleaved"]:
        x0, x1 = xf[..., 0:rot:2], xf[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    else:
        x0, x1 = xf[..., :rot // 2], xf[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    return y.to(x.dtype)


def _visible(s, N):
    """[1 or B, N, N]: which keys a query sees."""
    i = torch.arange(N, device="cuda")
    see = torch.ones((1, N, N), dtype=torch.bool, device="cuda")
    if s["causal"]:
        see = see & (i[None, :] <= i[:, None])
    if s["window"] > 0:
        see = see & (i[None, :] > i[:, None] - s["window"])
    if s["lens"] is not None:
        see = see & (i[None, None, :] < s["lens"][:, None, None])
    return see


def _plain_softmax(scores, see):
    """P and the logsumexp over the visible keys: zeros and -inf for a row that sees none."""
    x = scores.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return p / torch.where(total == 0, torch.ones_like(total), total), lse


def _plain_diff(s):
    B, H, Hkv, N = s["B"], s["H"], s["Hkv"], s["N"]
    G, dt, tau = H // Hkv, s["q"].dtype, 0.125
    q = s["q"].float().view(B, Hkv, G, 2, N, 64)
    k = s["k"].float().view(B, Hkv, 1, 2, N, 64)
    v = s["v"].float().view(B, Hkv, 1, N, 128)
    lam = s["lam"].view(1, Hkv, G, 1, 1)
    see = _visible(s, N)[:, None, None, None]
    p, lse = _plain_softmax(torch.matmul(q, k.transpose(-1, -2)) * tau, see)
    p1, p2 = p[:, :, :, 0], p[:, :, :, 1]
    w = p1 - lam * p2
    o = torch.matmul(w, v)
    out = [o.reshape(B, H, N, 128).to(dt), lse.reshape(B, 2 * H, N)]
    if not s["backward"]:
        return out
    do = s["do"].float().view(B, Hkv, G, N, 128)
    dv = torch.matmul(w.transpose(-1, -2), do).sum(2)
    del w
    dp = torch.matmul(do, v.transpose(-1, -2))
    d1, d2 = (p1 * dp).sum(-1, keepdim=True), (p2 * dp).sum(-1, keepdim=True)
    ds = torch.stack((p1 * (dp - d1) * tau, p2 * (dp - d2) * (-tau * lam)), 3)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    dlam = -d2.sum((0, 3, 4)).reshape(H)
    return out + [dq.reshape(B, 2 * H, N, 64).to(dt), dk.reshape(B, 2 * Hkv, N, 64).to(dt),
                  dv.reshape(B, Hkv, N, 128).to(dt), dlam]


def _plain_prefix(s):
    B, H, Hkv, T, P, M, d = (s[n] for n in ("B", "H", "Hkv", "T", "P", "M", "d"))
    G, dt, tau = H // Hkv, s["q"].dtype, 1.0 / math.sqrt(d)
    q = s["q"].float().view(B, Hkv, G * T, d)
    kp, vp = s["kp"].float(), s["vp"].float()
    shared = q.transpose(0, 1).reshape(Hkv, B * G * T, d)                   # every sequence's rows against one prefix
    sp = torch.matmul(shared, kp.transpose(-1, -2)).view(Hkv, B, G * T, P).transpose(0, 1)
    so = torch.matmul(q, s["k"].float().transpose(-1, -2))
    j, t = torch.arange(M, device="cuda"), torch.arange(T, device="cuda")
    see = j[None, None, :] <= (s["lens"][:, None, None] - T + t[None, :, None])          # [B, T, M]
    see = see[:, None, None].expand(B, 1, G, T, M).reshape(B, 1, G * T, M)
    see = torch.cat((torch.ones((B, 1, G * T, P), dtype=torch.bool, device="cuda"), see), -1)
    p, lse = _plain_softmax(torch.cat((sp, so), -1) * tau, see)
    o = torch.matmul(p[..., P:], s["v"].float())
    op = torch.matmul(p[..., :P].transpose(0, 1).reshape(Hkv, B * G * T, P), vp)
    o = o + op.view(Hkv, B, G * T, d).transpose(0, 1)
    return [o.reshape(B, H, T, d).to(dt), lse.reshape(B, H, T)]


def run(state):
    s = state
    if s["op"] == "rope":
        if own:
            return list(_fa().rope(s["q"], s["k"], positions=s["positions"], inv_freq=s["inv_freq"],
                                   mscale=s["mscale"], interleaved=s["interleaved"], backward=s["backward"]))
        return [_plain_rope(s, s["q"]), _plain_rope(s, s["k"])]
    if s["op"] == "diff":
        if own:
            fa = _fa()
            mask = dict(causal=s["causal"], window=s["window"], seqlens_k=s["lens"])
            if not s["backward"]:
                return list(fa.diff_fwd(s["q"], s["k"], s["v"], s["lam"], need_o2=False, **mask)[:2])
            o, lse, o2 = fa.diff_fwd(s["q"], s["k"], s["v"], s["lam"], **mask)
            return [o, lse] + list(fa.diff_bwd(s["q"], s["k"], s["v"], s["lam"], o, o2, s["do"], lse, **mask))
        return _plain_diff(s)
    if own:
        return list(_fa().prefix_fwd(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lens"]))
    return _plain_prefix(s)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def _pairs(c):
    """Visible (query, key) pairs of one head, summed over the batch."""
    N, w = c["N"], c["window"]
    i = np.arange(N, dtype=np.int64)
    total = 0
    lens = _spread(c["lo"], c["hi"], c["B"]) if c["hi"] >= 0 else np.full(c["B"], N, dtype=np.int64)
    for n in lens:
        last = np.minimum(i, n - 1) if c["causal"] else np.full(N, n - 1)
        first = np.maximum(i - w + 1, 0) if w > 0 else np.zeros(N, dtype=np.int64)
        total += int(np.maximum(last - first + 1, 0).sum())
    return total


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    B, H, Hkv = c["B"], c["H"], c["Hkv"]
    if c["op"] == "rope":
        n = B * (H + Hkv) * c["N"]
        return {"bytes": 2 * n * c["d"] * e + 4 * c["N"] * (B if c["perseq"] else 1) + 4 * c["rot"],
                "flops": 3 * n * c["rot"]}
    if c["op"] == "diff":
        qo, kv = B * H * c["N"] * 128 * e, B * Hkv * c["N"] * 128 * e
        lse, pairs = 4 * B * 2 * H * c["N"], H * _pairs(c)
        bytes_, flops = 2 * qo + 2 * kv + lse, 512 * pairs
        if c["backward"]:       # dO in; dQ, dK, dV out; both score maps again, dP, dV, dQ, dK
            bytes_, flops = bytes_ + 2 * qo + 2 * kv, flops + 1280 * pairs
        return {"bytes": bytes_, "flops": flops}
    d, T = c["d"], c["T"]
    lens = _spread(c["lo"], c["hi"], B)
    keys = int(lens.sum())
    pairs = B * T * c["P"] + sum(int(max(0, n - T + t + 1)) for n in lens for t in range(T))
    return {"bytes": 2 * B * H * T * d * e + 4 * B * H * T + 2 * Hkv * (c["P"] + keys) * d * e,
            "flops": 4 * d * H * pairs}


# ---------------------------------------------------------------------------------------------------------------
# the same outputs in 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------------------------
def _exact_rope(s, x):
    # a pair as a complex number, turned by exp(+-i angle)
    rot = s["rot"]
    sign = -1.0 if s["backward"] else 1.0
    turn = torch.polar(torch.full_like(s["inv_freq"], s["mscale"]).expand(s["positions"].shape + (rot // 2,)).contiguous(),
                       sign * s["positions"].to(torch.float64).unsqueeze(-1) * s["inv_freq"])
    if turn.dim() == 3:
        turn = turn.unsqueeze(1)
    y = x.to(torch.float64)
    head = y[..., :rot]
    if s["interleaved"]:
        z = torch.view_as_complex(head.reshape(head.shape[:-1] + (rot // 2, 2)).contiguous()) * turn
        head = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        head = torch.cat((z.real, z.imag), -1)
    return torch.cat((head, y[..., rot:]), -1)


def _exact_diff(s):
    # one head pair of one sequence at a time; the gradients by differentiating the forward
    B, H, Hkv, N = s["B"], s["H"], s["Hkv"], s["N"]
    G, grad = H // Hkv, s["backward"]
    lv = {n: s[n].detach().to(torch.float64).requires_grad_(grad) for n in ("q", "k", "v", "lam")}
    do = s["do"].to(torch.float64)
    o = torch.zeros((B, H, N, 128), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, 2 * H, N), dtype=torch.float64, device="cuda")
    sums = {n: torch.zeros_like(t) for n, t in lv.items()}
    seen = _visible(s, N)
    for b in range(B):
        see = seen[b % seen.shape[0]]
        none = ~see.any(-1, keepdim=True)
        for h in range(H):
            hk = h // G
            q, k = lv["q"][b, 2 * h:2 * h + 2], lv["k"][b, 2 * hk:2 * hk + 2]
            x = torch.einsum("mid,mjd->mij", q, k) / 8.0
            x = torch.where(see | none, x, torch.full_like(x, -math.inf))
            p = torch.softmax(x, -1) * (~none)
            y = (p[0] - lv["lam"][h] * p[1]) @ lv["v"][b, hk]
            o[b, h] = y.detach()
            lse[b, 2 * h:2 * h + 2] = torch.logsumexp(x.detach(), -1).masked_fill(none.squeeze(-1), -math.inf)
            if grad:
                leaf = [q, k, lv["v"], lv["lam"]]
                got = torch.autograd.grad(y, leaf, do[b, h])
                sums["q"][b, 2 * h:2 * h + 2] += got[0]
                sums["k"][b, 2 * hk:2 * hk + 2] += got[1]
                sums["v"] += got[2]
                sums["lam"] += got[3]
    return [o, lse] + ([sums["q"], sums["k"], sums["v"], sums["lam"]] if grad else [])


def _exact_prefix(s):
    # each sequence's keys in one row, one sequence after the other
    B, H, Hkv, T, d = s["B"], s["H"], s["Hkv"], s["T"], s["d"]
    G = H // Hkv
    o = torch.zeros((B, H, T, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    kp, vp = s["kp"].to(torch.float64), s["vp"].to(torch.float64)
    for b, n in enumerate(s["lens"].tolist()):
        k = torch.cat((kp, s["k"][b, :, :n].to(torch.float64)), 1)
        v = torch.cat((vp, s["v"][b, :, :n].to(torch.float64)), 1)
        for t in range(T):
            seen = s["P"] + max(0, n - T + t + 1)
            if seen == 0:
                continue
            q = s["q"][b, :, t].to(torch.float64).view(Hkv, G, d)
            x = torch.bmm(q, k[:, :seen].transpose(1, 2)) * d ** -0.5
            lse[b, :, t] = torch.logsumexp(x, -1).view(H)
            o[b, :, t] = torch.bmm(torch.softmax(x, -1), v[:, :seen]).view(H, d)
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        return [_exact_rope(s, s["q"]), _exact_rope(s, s["k"])]
    if s["op"] == "diff":
        if s["backward"]:
            # one sequence's leaves at a time keep the gradients' zero fill small
            return _by_sequence(s)
        return _exact_diff(s)
    return _exact_prefix(s)


def _by_sequence(s):
    parts = []
    for b in range(s["B"]):
        one = dict(s, B=1, lens=None if s["lens"] is None else s["lens"][b:b + 1])
        one.update({n: s[n][b:b + 1] for n in ("q", "k", "v", "do")})
        parts.append(_exact_diff(one))
    return [torch.cat([p[i] for p in parts]) for i in range(5)] + [sum(p[5] for p in parts)]
