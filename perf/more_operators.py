"""Cases, inputs, plain forms and 64-bit values of the operators of a model with a sliding window: what it trains with
and what it serves from.

``norm``    q and k normalised for each head and rotated by their positions in one pass, or the gradients of that
            (q, k and both weight vectors).
``sink``    attention with a sliding window whose first tokens stay visible, forward alone or forward and backward.
``append``  new keys and values written into a paged cache of 8-bit codes with a scale for each page and head, then
            the sequences' caches read back in 16 bits (a prompt in chunks attends to what the cache holds).
``cache``   T new tokens of each of B sequences attend to their 8-bit caches, with or without window and sinks.

With ``own`` false, ``run`` is the plain form: elementary torch operations in 32 bits (angles in 64), rounded once
at the end.  With ``own`` true it makes the framework's calls on the same state.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def _fa():
    import exact_io_aware_tiled_gb300 as fa
    return fa


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _norm(name, **kw):
    c = dict(op="norm", B=1, H=16, Hkv=16, N=1024, d=64, rot=64, dtype="bf16", interleaved=False, backward=False,
             base=10000.0, start=0, perseq=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _sink(name, **kw):
    c = dict(op="sink", B=1, H=16, Hkv=16, N=1024, d=64, dtype="bf16", window=256, sinks=4, lo=-1, hi=-1, backward=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _append(name, **kw):
    c = dict(op="append", B=8, Hkv=16, d=64, T=1, M=512, lo=1, hi=512, page=64, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _cache(name, **kw):
    c = dict(op="cache", B=8, H=16, Hkv=16, d=64, T=1, M=1024, lo=1, hi=1024, page=64, window=0, sinks=0, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of 64 sequences at far, different positions, grouped heads: latency alone
        _norm("norm one token", B=64, Hkv=4, N=1, start=100000, perseq=True),
        # q and k of the GPT-2-medium training step
        _norm("norm gpt2-medium", B=64),
        # their gradients
        _norm("norm back gpt2-medium", B=64, backward=True),
        # gradients of a long ragged batch: grouped heads of 128, half of a head rotated, pairs interleaved, fp16
        _norm("norm back interleaved", B=3, H=32, Hkv=4, N=7001, d=128, rot=64, dtype="f16", interleaved=True,
              backward=True),
        # a short prompt through one small layer: latency alone
        _sink("sink short prompt", H=4, Hkv=2, N=300, dtype="f16", window=64),
        # GPT-2-medium heads on longer sequences: the training step
        _sink("sink train", B=4, N=4096, window=512, backward=True),
        # grouped heads, padded sequences of an odd length, more first tokens than one tile: the training step
        _sink("sink padded train", B=8, H=12, Hkv=4, N=2047, window=300, sinks=150, lo=0, hi=2047, dtype="f16",
              backward=True),
        # a long prompt, wide grouped heads
        _sink("sink long prompt", H=8, Hkv=2, N=16383, d=128, window=4096),
        # one decoding step of 64 sequences, then their caches
        _append("append one token", B=64, M=512, lo=1, hi=509, page=16),
        # a chunk of 2,047 tokens of four prompts behind what was there before
        _append("append chunk", B=4, Hkv=8, d=128, T=2047, M=8192, lo=2047, hi=8190),
        # 64 sequences of very different length, GPT-2-medium heads
        _cache("cache 64 sequences", B=64, M=8192, lo=1, hi=8191),
        # a 23,400-step day, 6 continuations of 5 tokens each, 12 heads, fp16, a window with 4 first tokens
        _cache("cache window", B=6, H=12, Hkv=12, T=5, M=23424, lo=5, hi=23400, window=4096, sinks=4, page=32,
               dtype="f16"),
    ]


def _cost(c):
    w = work(c)
    return w["flops"] + 300 * w["bytes"]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    cap = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "sink", "append", "cache"])
        if op == "norm":
            d = rng.choice([64, 128])
            hkv = rng.choice([1, 2, 4, 8, 12])
            c = _norm(None, B=log(1, 64), Hkv=hkv, H=hkv * rng.choice([1, 2, 4]), N=log(1, 9000), d=d,
                      rot=rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]),
                      dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), interleaved=rng.random() < 0.5,
                      backward=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]),
                      start=rng.choice([0, log(1, 1000000)]), perseq=rng.random() < 0.5)
        elif op == "sink":
            hkv = rng.choice([1, 2, 4, 8])
            n = log(8, 8000)        # a row of one key has P = 1 and no gradient to compare
            pad = rng.random() < 0.4
            d = rng.choice([64, 64, 128])
            c = _sink(None, B=log(1, 16), Hkv=hkv, H=hkv * rng.choice([1, 1, 2, 4]), N=n, d=d,
                      dtype=rng.choice(["bf16", "bf16", "f16"] + (["f32"] if d == 64 else [])),
                      window=log(2, max(2, n // 2)), sinks=rng.choice([1, 4, log(1, 300)]), lo=0 if pad else -1,
                      hi=n if pad else -1, backward=rng.random() < 0.6)
            if c["B"] * c["H"] * n * n > 64 * 8 * 1024 * 1024:   # the plain form holds the score maps
                continue
        else:
            hkv = rng.choice([1, 2, 8, 12, 16])
            page = rng.choice([16, 32, 64, 128])
            d = rng.choice([64, 128])
            if op == "append":
                t = rng.choice([1, 1, rng.randint(2, 9), log(1, 2000)])
                m = page * log(-(-max(t, 2) // page), 8192 // page)
                c = _append(None, B=log(1, 64), Hkv=hkv, d=d, T=t, M=m, lo=min(t, m), hi=rng.randint(min(t, m), m),
                            page=page, dtype=rng.choice(["bf16", "bf16", "f16"]))
            else:
                t = rng.choice([1, 1, 1, rng.randint(2, 9)])
                m = page * log(-(-max(t, 2) // page), 32768 // page)
                win = rng.random() < 0.4
                c = _cache(None, B=log(1, 128), Hkv=hkv, H=hkv * rng.choice([1, 1, 4, 8]), d=d, T=t, M=m, lo=0,
                           hi=rng.randint(t, m), page=page, window=log(1, m) if win else 0,
                           sinks=rng.choice([0, 4, log(1, 200)]) if win else 0,
                           dtype=rng.choice(["bf16", "bf16", "f16"]))
            if c["B"] * c["Hkv"] * c["M"] * d > 64 * 16 * 8192 * 64:   # the plain form holds the caches in 32 bits
                continue
            if op == "cache" and c["B"] * c["H"] * c["T"] * c["M"] > 128 * 16 * 40000:
                continue
        if _cost(c) <= cap:
            return c


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n lengths spread evenly over lo..hi (the same sum for every seed)."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64) if n > 1 else np.array([hi], dtype=np.int64)


def _e4m3(y):
    """y (|y| <= 448) rounded to the nearest value of the E4M3 grid, ties to even: 3 bits behind the leading one,
    from 2^-6 down a fixed step of 2^-9."""
    _, k = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (k - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step


def _exponent(amax):
    """The scale's exponent: the smallest whole e with amax <= 448 2^e, -126 at least."""
    m, k = torch.frexp(amax)
    e = k - 9 + (m > 0.875).to(k.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng([seed, 7])
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = dict(c)
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "norm":
        H, N = c["H"], c["N"]
        s["q"], s["k"] = normal(B, H, N, d), normal(B, Hkv, N, d)
        s["wq"], s["wk"] = (1.0 + 0.2 * torch.randn((d,), generator=g, device="cuda") for _ in range(2))
        if c["backward"]:
            s["dq"], s["dk"] = normal(B, H, N, d), normal(B, Hkv, N, d)
        i = np.arange(c["rot"] // 2, dtype=np.float64)
        s["inv_freq"] = torch.from_numpy(c["base"] ** (-2.0 * i / c["rot"])).cuda()
        pos = np.arange(N, dtype=np.int64) + c["start"]
        if c["perseq"]:
            pos = pos[None, :] + rng.integers(0, 1 + c["start"] // 2 + 64, size=(B, 1))
        s["positions"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        return s
    lens = None
    if c["hi"] >= 0:
        lens = rng.permutation(_spread(c["lo"], c["hi"], B))
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    if c["op"] == "sink":
        H, N = c["H"], c["N"]
        s["q"], s["k"], s["v"] = normal(B, H, N, d), normal(B, Hkv, N, d), normal(B, Hkv, N, d)
        s["do"] = normal(B, H, N, d)
        if lens is None:
            s["lens"] = None
        return s
    # a pool of pages in no order; the pages of a sequence lie anywhere in it, what it has no page for is -1
    page, W = c["page"], -(-c["M"] // c["page"])
    need = -(-lens // page)
    pool = rng.permutation(int(need.sum()) + 3)
    table = np.full((B, W), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = pool[at:at + need[b]]
        at += need[b]
    s["table"] = torch.from_numpy(table).cuda()
    NP = len(pool)
    for n in ("k", "v"):
        x = torch.randn((NP, Hkv, page, d), generator=g, device="cuda", dtype=torch.float32)
        x *= torch.exp(0.5 * torch.randn((NP, Hkv, 1, 1), generator=g, device="cuda", dtype=torch.float32))
        e = _exponent(x.abs().amax((2, 3)))
        s[n + "s"] = torch.ldexp(torch.ones_like(x[:, :, 0, 0]), e)
        s[n + "c"] = _e4m3(x / s[n + "s"][:, :, None, None]).to(torch.float8_e4m3fn)
        del x
    if c["op"] == "append":
        # the new rows are larger than most of the old ones: some pages have to take a larger scale
        s["k"], s["v"] = 2 * normal(B, Hkv, c["T"], d), 2 * normal(B, Hkv, c["T"], d)
    else:
        s["q"] = normal(B, c["H"], c["T"], d)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def _turns(s):
    a = s["positions"].double()[..., None] * s["inv_freq"]                  # [N, rot/2] or [B, N, rot/2]
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    return (cos[:, None], sin[:, None]) if a.dim() == 3 else (cos, sin)     # over the heads


def _rotated(s, x, cos, sin):
    rot, y = s["rot"], x.clone()
    if s["interleaved"]:
        x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    else:
        x0, x1 = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    return y


def _plain_norm(s, x, w, dy):
    cos, sin = _turns(s)
    xf = x.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    h = xf * r
    if dy is None:
        return _rotated(s, h * w, cos, sin).to(x.dtype)
    dz = _rotated(s, dy.float(), cos, -sin)
    dh = dz * w
    dx = r * (dh - h * (dh * h).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dz * h).sum((0, 1, 2))


def _plain_softmax(scores, see):
    """P and the logsumexp over the visible keys: zeros and -inf for a row that sees none."""
    x = scores.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return p / torch.where(total == 0, torch.ones_like(total), total), lse


def _plain_sink(s):
    B, H, Hkv, N, d = s["B"], s["H"], s["Hkv"], s["N"], s["d"]
    G, dt, tau = H // Hkv, s["q"].dtype, 1.0 / math.sqrt(d)
    q, do = (s[n].float().view(B, Hkv, G, N, d) for n in ("q", "do"))
    k, v = (s[n].float().view(B, Hkv, 1, N, d) for n in ("k", "v"))
    i = torch.arange(N, device="cuda")
    see = (i[None, :] <= i[:, None]) & ((i[None, :] > i[:, None] - s["window"]) | (i[None, :] < s["sinks"]))
    if s["lens"] is not None:
        see = see & (i[None, None, :] < s["lens"][:, None, None])
        see = see[:, None, None]
    p, lse = _plain_softmax(torch.matmul(q, k.transpose(-1, -2)) * tau, see)
    o = torch.matmul(p, v)
    out = [o.reshape(B, H, N, d).to(dt), lse.reshape(B, H, N)]
    if not s["backward"]:
        return out
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    dp = torch.matmul(do, v.transpose(-1, -2))
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * tau
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return out + [dq.reshape(B, H, N, d).to(dt), dk.to(dt), dv.to(dt)]


def _cached(s, n, scaled=True):
    """[B, Hkv, W page, d] float32: each sequence's cache in the order of its tokens, absent pages as page 0."""
    B, Hkv, d, page = s["B"], s["Hkv"], s["d"], s["page"]
    ids = s["table"].long().clamp(min=0)
    x = s[n + "c"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
    if scaled:
        x = x * s[n + "s"][ids][..., None, None]
    return x.transpose(1, 2).reshape(B, Hkv, -1, d)


def _plain_append(s):
    B, Hkv, d, T, page = s["B"], s["Hkv"], s["d"], s["T"], s["page"]
    W = s["table"].shape[1]
    j = torch.arange(W * page, device="cuda")
    first = (s["lens"] - T)[:, None]
    new, old = (j[None] >= first) & (j[None] < s["lens"][:, None]), j[None] < first            # [B, M]
    row = (j[None] - first).clamp(0, T - 1)[:, None, :, None].expand(B, Hkv, W * page, d).long()
    ids = s["table"].long()
    kept = old.view(B, W, page).any(-1)[:, None]                                               # [B, 1, W]
    write = new.view(B, W, page).any(-1) & (ids >= 0)                                          # pages to write
    out = []
    for n in ("k", "v"):
        x = torch.gather(s[n].float(), 2, row)
        amax = (x.abs() * new[:, None, :, None]).view(B, Hkv, W, page, d).amax((-2, -1))
        was = s[n + "s"][ids.clamp(min=0)].transpose(1, 2)                                     # [B, Hkv, W]
        e = _exponent(amax)
        scale = torch.ldexp(torch.ones_like(was), e)
        scale = torch.where(kept, torch.maximum(scale, was), scale)
        wide = scale.repeat_interleave(page, 2)[..., None]
        ratio = torch.where(kept, was / scale, torch.ones_like(was)).repeat_interleave(page, 2)[..., None]
        codes = _cached(s, n, scaled=False)
        codes = torch.where(old[:, None, :, None], _e4m3(codes * ratio), codes)
        codes = torch.where(new[:, None, :, None], _e4m3(x / wide), codes)
        codes = codes.view(B, Hkv, W, page, d).transpose(1, 2)[write].to(torch.float8_e4m3fn)
        s[n + "c"].view(torch.uint8)[ids[write]] = codes.view(torch.uint8)
        s[n + "s"][ids[write]] = scale.transpose(1, 2)[write]
        read = _cached(s, n) * (j[None] < s["lens"][:, None])[:, None, :, None]
        out.append(read.to(s["k"].dtype))
    return out


def _plain_cache(s):
    B, H, Hkv, T, d = (s[n] for n in ("B", "H", "Hkv", "T", "d"))
    G, dt = H // Hkv, s["q"].dtype
    k, v = _cached(s, "k"), _cached(s, "v")
    M = k.shape[2]
    q = s["q"].float().view(B, Hkv, G * T, d)
    j, t = torch.arange(M, device="cuda"), torch.arange(T, device="cuda")
    p = (s["lens"][:, None] - T + t)[:, :, None]                                               # [B, T, 1]
    see = j <= p
    if s["window"] > 0:
        see = see & ((j > p - s["window"]) | (j < s["sinks"]))
    see = see[:, None, None].expand(B, 1, G, T, M).reshape(B, 1, G * T, M)
    w, lse = _plain_softmax(torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d)), see)
    return [torch.matmul(w, v).reshape(B, H, T, d).to(dt), lse.reshape(B, H, T)]


def run(state):
    s = state
    if s["op"] == "norm":
        if own:
            kw = dict(q_weight=s["wq"], k_weight=s["wk"], eps=EPS, inv_freq=s["inv_freq"], positions=s["positions"],
                      interleaved=s["interleaved"])
            if s["backward"]:
                return list(_fa().norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], **kw))
            return list(_fa().norm_rope(s["q"], s["k"], **kw))
        if s["backward"]:
            (dq, dwq), (dk, dwk) = _plain_norm(s, s["q"], s["wq"], s["dq"]), _plain_norm(s, s["k"], s["wk"], s["dk"])
            return [dq, dk, dwq, dwk]
        return [_plain_norm(s, s["q"], s["wq"], None), _plain_norm(s, s["k"], s["wk"], None)]
    if s["op"] == "sink":
        if own:
            mask = dict(causal=True, window=s["window"], sinks=s["sinks"], seqlens_k=s["lens"])
            o, lse = _fa().fwd(s["q"], s["k"], s["v"], **mask)
            if not s["backward"]:
                return [o, lse]
            return [o, lse] + list(_fa().bwd(s["q"], s["k"], s["v"], o, s["do"], lse, **mask))
        return _plain_sink(s)
    if s["op"] == "append":
        if own:
            cache = (s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"])
            _fa().cache8_append(s["k"], s["v"], *cache)
            return list(_fa().cache8_read(*cache, dtype=s["k"].dtype))
        return _plain_append(s)
    if own:
        return list(_fa().cache8_fwd(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"],
                                     window=s["window"], sinks=s["sinks"]))
    return _plain_cache(s)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def _seen(n, rows, window, sinks):
    """Of the n first keys: how many the queries at positions `rows` see, in all."""
    last = np.minimum(rows, n - 1)
    total = np.maximum(last + 1, 0)
    if window > 0:
        hidden = np.maximum(np.minimum(rows - window, last) + 1 - np.minimum(sinks, np.maximum(last + 1, 0)), 0)
        total = total - hidden
    return int(np.maximum(total, 0).sum())


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "norm":
        n = B * (c["H"] + Hkv) * c["N"]
        moved = 3 if c["backward"] else 2
        return {"bytes": moved * n * d * e + 4 * c["N"] * (B if c["perseq"] else 1) + 4 * c["rot"],
                "flops": (12 if c["backward"] else 4) * n * d + 3 * n * c["rot"]}
    lens = _spread(c["lo"], c["hi"], B) if c["hi"] >= 0 else np.full(B, c.get("N", 0), dtype=np.int64)
    if c["op"] == "sink":
        H, N = c["H"], c["N"]
        rows = np.arange(N, dtype=np.int64)
        pairs = H * sum(_seen(int(n), rows, c["window"], c["sinks"]) for n in lens)
        qo, kv = B * H * N * d * e, B * Hkv * N * d * e
        bytes_, flops = 2 * qo + 2 * kv + 4 * B * H * N, 4 * d * pairs
        if c["backward"]:       # dO in; dQ, dK, dV out; the scores again, dP, dV, dQ, dK
            bytes_, flops = bytes_ + 2 * qo + 2 * kv, flops + 10 * d * pairs
        return {"bytes": bytes_, "flops": flops}
    T = c["T"]
    if c["op"] == "append":
        new = 2 * B * Hkv * T * d
        rows = 2 * Hkv * d * int(lens.sum())
        out = 2 * B * Hkv * (-(-c["M"] // c["page"]) * c["page"]) * d
        # the new rows in; every filled row in as a code, out in 16 bits, zeros behind them
        return {"bytes": new * e + rows + out * e, "flops": 4 * new + rows}
    t = np.arange(T, dtype=np.int64)
    pairs = keys = 0
    for n in (int(x) for x in lens):
        pairs += c["H"] * _seen(n, n - T + t, c["window"], c["sinks"])
        low = max(0, n - T - c["window"] + 1) if c["window"] > 0 else 0
        keys += n - low + min(low, c["sinks"])
    qo = B * c["H"] * T * d
    return {"bytes": 2 * qo * e + 4 * B * c["H"] * T + 2 * Hkv * keys * d, "flops": 4 * d * pairs}


# ---------------------------------------------------------------------------------------------------------------
# the same outputs in 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------------------------
def _exact_norm(s):
    # pairs as complex numbers, turned by exp(i angle); gradients by differentiating the forward, head by head
    rot, back = s["rot"], s["backward"]
    angle = s["positions"].to(torch.float64).unsqueeze(-1) * s["inv_freq"]
    turn = torch.polar(torch.ones_like(angle), angle)
    outs, sums = [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(x.shape[-1], dtype=torch.float64, device="cuda")
        for h in range(x.shape[1]):
            leaf = x[:, h].to(torch.float64).requires_grad_(back)
            lw = w.to(torch.float64).requires_grad_(back)
            z = leaf * lw / torch.sqrt((leaf * leaf).sum(-1, keepdim=True) / x.shape[-1] + EPS)
            head = z[..., :rot]
            if s["interleaved"]:
                head = head.reshape(head.shape[:-1] + (rot // 2, 2))
                u = torch.view_as_real(torch.complex(head[..., 0], head[..., 1]) * turn).flatten(-2)
            else:
                u = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * turn
                u = torch.cat((u.real, u.imag), -1)
            z = torch.cat((u, z[..., rot:]), -1)
            if back:
                gx, gw = torch.autograd.grad(z, [leaf, lw], dy[:, h].to(torch.float64))
                y[:, h], dw = gx, dw + gw
            else:
                y[:, h] = z
        outs.append(y)
        sums.append(dw)
    return outs + sums if back else outs


def _exact_sink(s):
    # one head of one sequence at a time, blocks of queries against the keys they may see; gradients by differentiating
    B, H, Hkv, N, d = s["B"], s["H"], s["Hkv"], s["N"], s["d"]
    G, grad, w, ns = H // Hkv, s["backward"], s["window"], s["sinks"]
    f8 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros((B, H, N, d), **f8), torch.full((B, H, N), -math.inf, **f8)
    dq, dk, dv = torch.zeros((B, H, N, d), **f8), torch.zeros((B, Hkv, N, d), **f8), torch.zeros((B, Hkv, N, d), **f8)
    lens = [N] * B if s["lens"] is None else s["lens"].tolist()
    step = 1024
    for b in range(B):
        for h in range(H):
            hk = h // G
            for i0 in range(0, N, step):
                i = torch.arange(i0, min(N, i0 + step), device="cuda")
                low = max(0, i0 - w + 1)
                j = torch.cat((torch.arange(min(ns, low), device="cuda"), torch.arange(low, int(i[-1]) + 1, device="cuda")))
                j = j[j < lens[b]]
                if len(j) == 0:
                    continue
                lq = s["q"][b, h, i].to(torch.float64).requires_grad_(grad)
                lk = s["k"][b, hk, j].to(torch.float64).requires_grad_(grad)
                lv = s["v"][b, hk, j].to(torch.float64).requires_grad_(grad)
                ahead = (i[:, None] - j[None, :])
                see = (ahead >= 0) & ((ahead < w) | (j[None, :] < ns))
                some = see.any(-1)
                x = torch.einsum("id,jd->ij", lq, lk) * d ** -0.5
                x = x.masked_fill(~see & some[:, None], -math.inf)
                y = (torch.softmax(x, -1) * some[:, None]) @ lv
                o[b, h, i] = y.detach()
                lse[b, h, i] = torch.logsumexp(x.detach(), -1).masked_fill(~some, -math.inf)
                if grad:
                    gq, gk, gv = torch.autograd.grad(y, [lq, lk, lv], s["do"][b, h, i].to(torch.float64))
                    dq[b, h, i] = gq
                    dk[b, hk].index_add_(0, j, gk)
                    dv[b, hk].index_add_(0, j, gv)
    return [o, lse] + ([dq, dk, dv] if grad else [])


def _grid():
    """The values of E4M3 from 0 up, by their codes, and the middles between them."""
    v = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]
    v = torch.tensor(v, dtype=torch.float64, device="cuda")
    return v, (v[1:] + v[:-1]) / 2


def _nearest(y):
    v, mid = _grid()
    a = y.abs()
    n = torch.searchsorted(mid, a.contiguous())                 # a tie takes the lower code here
    tie = (n < 126) & (mid[n.clamp(max=125)] == a) & (n % 2 == 1)
    return v[n + tie.long()] * torch.sign(y)


def _exact_append(s):
    # page by page of every sequence
    B, Hkv, d, T, page = s["B"], s["Hkv"], s["d"], s["T"], s["page"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    out = []
    for n in ("k", "v"):
        codes, scale, x = s[n + "c"].to(torch.float64), s[n + "s"].to(torch.float64), s[n].to(torch.float64)
        y = torch.zeros((B, Hkv, len(table[0]) * page, d), dtype=torch.float64, device="cuda")
        for b in range(B):
            for at in range(0, lens[b], page):
                p, end, new = table[b][at // page], min(at + page, lens[b]), max(at, lens[b] - T)
                held = codes[p, :, :end - at] * scale[p][:, None, None]
                if new < end:
                    rows = x[b, :, new - lens[b] + T:end - lens[b] + T]
                    top = rows.abs().amax((1, 2))
                    e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), torch.full_like(top, -126.0))
                    e = torch.where(448 * 2.0 ** (e - 1) >= top, e - 1, e).clamp(min=-126.0)      # log2's own rounding
                    sc = 2.0 ** e
                    if new > at:
                        sc = torch.maximum(sc, scale[p])
                    sc = sc[:, None, None]
                    held = torch.cat((_nearest(held[:, :new - at] / sc), _nearest(rows / sc)), 1) * sc
                y[b, :, at:end] = held
        out.append(y)
    return out


def _exact_cache(s):
    # each sequence's keys in one row, one sequence after the other
    B, H, Hkv, T, d, page = (s[n] for n in ("B", "H", "Hkv", "T", "d", "page"))
    o = torch.zeros((B, H, T, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        k, v = ((s[x + "c"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).to(torch.float64) *
                 s[x + "s"][ids].to(torch.float64)[..., None, None]).transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
                for x in ("k", "v"))
        for t in range(T):
            p = n - T + t
            if p < 0:
                continue
            low = max(0, p - s["window"] + 1) if s["window"] > 0 else 0
            j = torch.cat((torch.arange(min(low, s["sinks"]), device="cuda"), torch.arange(low, p + 1, device="cuda")))
            x = torch.bmm(s["q"][b, :, t].to(torch.float64).view(Hkv, H // Hkv, d), k[:, j].transpose(1, 2)) * d ** -0.5
            lse[b, :, t] = torch.logsumexp(x, -1).view(H)
            o[b, :, t] = torch.bmm(torch.softmax(x, -1), v[:, j]).view(H, d)
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "sink": _exact_sink, "append": _exact_append, "cache": _exact_cache}[s["op"]](s)
