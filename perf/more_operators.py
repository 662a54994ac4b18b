"""Measured cases of the 4-bit cache and of the step with head norms: attention
over a paged cache held in 4 bits, the append that norms, rotates and quantises
a step's keys and values into it, and the append of normed and rotated keys to
the 16-bit cache.

listed() and draw() give cases (dicts of plain values), prepare() what a
serving program has in hand before the call, run() one call, work() the bytes
and operations that the call cannot do without, exact() its result in 64 bits.
run() computes the plain form in elementary torch operations, or, where `own`
is true, calls the library.

The 4-bit cache: a head of 128 dims is held as value_d = s (n_d - z) with codes
n_d and a zero point z from 0 to 15, s an fp16 whose low four bits are zero, at
most 4096; z lies in those four bits.  A row is 64 bytes, dim d in the low (even
d) or high nibble of byte d // 2.  A block holds B = min(page, 32) slots of one
head: B rows of k, B rows of v, B words (s | z) of k, B words of v, padded to a
multiple of 16 bytes; a page of a head is page / B blocks, and the cache uint8
[pages, heads, bytes of a page].  The quantiser, with lo = min(x, 0) and hi =
max(x, 0) over the head: s is (hi - lo) / 15 in fp16, its bits rounded up to a
multiple of 16; z = rint(-lo / s) and n = rint(x / s) + z, both kept in 0 .. 15.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_EPS = 1e-6
_D = 128  # dims of a head of the 4-bit cache


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few short requests, one token each: the latency of one call
        dict(name="kv4_decode_small", op="attend", dtype="fp16", batch=4, prefills=0, q_lo=1, q_hi=1, prefix=0, kv_lo=1,
             kv_hi=512, heads=8, kv_heads=2, page=16, causal=False, window=-1, sink=0, lens=1),
        # a serving batch of 64 single-token requests, lengths from 512 to 32768
        dict(name="kv4_decode_batch", op="attend", dtype="bf16", batch=64, prefills=0, q_lo=1, q_hi=1, prefix=0,
             kv_lo=512, kv_hi=32768, heads=32, kv_heads=8, page=16, causal=False, window=-1, sink=0, lens=2),
        # two long contexts, eight query heads per key head: the keys have to be split over the card
        dict(name="kv4_decode_long", op="attend", dtype="bf16", batch=2, prefills=0, q_lo=1, q_hi=1, prefix=0,
             kv_lo=99991, kv_hi=131072, heads=64, kv_heads=8, page=64, causal=False, window=-1, sink=0, lens=3),
        # 64 branches with a short private part on pages of one token
        dict(name="kv4_decode_page1", op="attend", dtype="bf16", batch=64, prefills=0, q_lo=1, q_hi=1, prefix=0,
             kv_lo=64, kv_hi=512, heads=32, kv_heads=8, page=1, causal=False, window=-1, sink=0, lens=4),
        # prompts being read, some behind an earlier part of the conversation
        dict(name="kv4_prefill", op="attend", dtype="bf16", batch=8, prefills=8, q_lo=128, q_hi=2048, prefix=2048,
             kv_lo=0, kv_hi=0, heads=32, kv_heads=8, page=16, causal=True, window=-1, sink=0, lens=5),
        # a mixed step with a sliding window and sink tokens: four prompt parts beside 24 decoding requests
        dict(name="kv4_mixed_window", op="attend", dtype="fp16", batch=28, prefills=4, q_lo=100, q_hi=256, prefix=4000,
             kv_lo=16, kv_hi=4096, heads=16, kv_heads=4, page=16, causal=True, window=1023, sink=4, lens=6),
        # one decode step: 64 new tokens normed, rotated and quantised into the 4-bit cache
        dict(name="kv4_append_decode", op="append4", dtype="bf16", tokens=64, pad=0, heads=32, kv_heads=8, rot=128,
             interleaved=False, norm=True, theta=1000000.0, far=131072, page=16),
        # a long prompt's tokens
        dict(name="kv4_append_prefill", op="append4", dtype="bf16", tokens=8192, pad=0, heads=32, kv_heads=8, rot=128,
             interleaved=False, norm=True, theta=1000000.0, far=16384, page=64),
        # half a head turned in neighbouring pairs, no norms, an odd count padded to a captured size
        dict(name="kv4_append_partial", op="append4", dtype="fp16", tokens=1111, pad=41, heads=16, kv_heads=16, rot=64,
             interleaved=True, norm=False, theta=10000.0, far=1000000, page=8),
        # one decode step into the 16-bit cache: 64 new tokens normed and rotated
        dict(name="norm_append_decode", op="append16", dtype="bf16", tokens=64, pad=0, heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, per_head=False, theta=1000000.0, far=131072, page=16),
        # a long prompt's tokens
        dict(name="norm_append_prefill", op="append16", dtype="bf16", tokens=16384, pad=0, heads=32, kv_heads=8,
             dim=128, rot=128, interleaved=False, per_head=False, theta=1000000.0, far=16384, page=16),
        # heads of 80 dims with weights of their own, partly turned, an odd count with padding
        dict(name="norm_append_partial", op="append16", dtype="fp16", tokens=1111, pad=41, heads=24, kv_heads=24,
             dim=80, rot=32, interleaved=True, per_head=True, theta=10000.0, far=1000000, page=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append4", "append4", "append16"])
    while op == "attend":
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 8, 16])
        if heads > 64:
            continue
        batch = _log(rng, 1, 64)
        kind = rng.choice(["decode", "decode", "prefill", "mixed"])
        prefills = {"decode": 0, "prefill": batch, "mixed": max(1, batch // 6)}[kind]
        q_hi = _log(rng, 2, 2048) if prefills else 1
        prefix = _log(rng, 1, 4096) if prefills else 0
        kv_hi = _log(rng, 64, 4096 if prefills else 131072)
        window = _log(rng, 16, 4096) if rng.random() < 0.25 else -1
        c = dict(op="attend", dtype=rng.choice(["bf16", "fp16"]), batch=batch, prefills=prefills,
                 q_lo=max(1, q_hi // 8), q_hi=q_hi, prefix=prefix, kv_lo=max(1, kv_hi // 64), kv_hi=kv_hi,
                 heads=heads, kv_heads=kv_heads, page=rng.choice([1, 4, 8, 16, 16, 32, 64, 128]), causal=prefills > 0,
                 window=window, sink=rng.choice([0, 4]) if window >= 0 else 0, lens=rng.randrange(1 << 20))
        rows = c["batch"] * max(l[1] for l in _lens(c))
        w = _attend_work(c)
        if (rows * kv_heads <= 64 * 32768 * 8 and rows * q_hi * heads <= 8 * 2048 * 4096 * 32
                and w["flops"] <= 2.0e11 and w["bytes"] <= 4.0e8):
            return c
    kv_heads = rng.choice([1, 2, 4, 8])
    c = dict(dtype=rng.choice(["bf16", "fp16"]), pad=rng.choice([0, 0, 1, 7]), heads=kv_heads * rng.choice([1, 2, 4]),
             kv_heads=kv_heads, interleaved=rng.random() < 0.5, theta=rng.choice([10000.0, 500000.0, 1000000.0]),
             page=rng.choice([1, 8, 16, 64]))
    if op == "append4":
        c.update(op=op, tokens=_log(rng, 1, 8192), norm=rng.random() < 0.6, rot=rng.choice([128, 128, 32, 64]))
    else:
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        c.update(op=op, tokens=_log(rng, 1, 16384 if dim <= 128 else 8192), dim=dim, rot=rng.choice([dim, dim, 32, 64]),
                 per_head=rng.random() < 0.3)
    c["far"] = max(c["tokens"], _log(rng, 1000, 1000000))
    return c


def _lens(c):
    """(query tokens, keys with those tokens) of each request of an attend case."""
    r = random.Random(c["lens"])
    got = []
    for b in range(c["batch"]):
        if b < c["prefills"]:
            q = r.randint(c["q_lo"], c["q_hi"])
            got.append((q, q + r.randint(0, c["prefix"])))
        else:
            got.append((1, _log(r, c["kv_lo"], c["kv_hi"])))
    return got


def _visible(c):
    """Pairs of a query token and a key that its mask leaves, and the keys that any token of its request sees."""
    pairs = keys = 0
    for q, kv in _lens(c):
        w, s = c["window"], c["sink"]
        for t in ([0] if q == 1 else range(q)):
            pos = kv - q + t
            hi = pos + 1 if c["causal"] else kv
            if w < 0:
                pairs += hi
            else:
                lo = max(0, pos - w)
                pairs += hi - lo + min(s, lo)
        lo = 0 if w < 0 else max(0, kv - q - w)
        keys += kv - lo + min(s, lo)
    return pairs, keys


def _attend_work(c):
    pairs, keys = _visible(c)
    tokens = sum(l[0] for l in _lens(c))
    return {"bytes": keys * c["kv_heads"] * 132 + tokens * c["heads"] * (512 + 4), "flops": pairs * c["heads"] * 512}


def work(c):
    if c["op"] == "attend":
        return _attend_work(c)
    H, Hk = c["heads"], c["kv_heads"]
    if c["op"] == "append4":  # q in and out, k and v in, their codes out; then the codes read and their values written
        row = 2 * H * 256 + Hk * 512 + Hk * 132 + Hk * (132 + 512)
        return {"bytes": c["tokens"] * (row + 8), "flops": c["tokens"] * _D * (7 * (H + Hk) + 8 * Hk)}
    row = 2 * c["dim"] * (H + 2 * Hk)
    return {"bytes": c["tokens"] * (2 * row + 8), "flops": 7 * c["tokens"] * (H + Hk) * c["dim"]}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _indptr(xs):
    got = [0]
    for x in xs:
        got.append(got[-1] + x)
    return got


def prepare(c, seed):
    return {"attend": _prepare_attend, "append4": _prepare_append, "append16": _prepare_append}[c["op"]](c, seed)


def _prepare_attend(c, seed):
    g, dt, P, Hk = _gen(seed), _DT[c["dtype"]], c["page"], c["kv_heads"]
    lens = _lens(c)
    qs, ks = [l[0] for l in lens], [l[1] for l in lens]
    pages = [-(-k // P) for k in ks]
    used = sum(pages)
    pool = used + 7
    qo, kvp = _indptr(qs), _indptr(pages)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    # keys with a few dims larger than the others, as keys have them
    wide = torch.ones(_D, device="cuda")
    wide[torch.randperm(_D, generator=g, device="cuda")[:4]] = 3.0
    cache = torch.zeros((pool, Hk, _page_bytes(P)), dtype=torch.uint8, device="cuda")
    some = max(1, (1 << 17) // P)
    for at in range(0, pool, some):
        n = min(some, pool - at)
        k = _normal(g, (n, P, Hk, _D), dt).float() * wide
        v = _normal(g, (n, P, Hk, _D), dt).float()
        cache[at:at + n] = _packed(*_codes(k), *_codes(v), P)
    s = {"c": c, "qo_indptr": _i32(qo), "kv_indptr": _i32(kvp), "kv_lens": _i32(ks), "cache": cache,
         "kv_indices": perm[:used].contiguous(), "q": _normal(g, (qo[-1], c["heads"], _D), dt),
         "scale": 1 / math.sqrt(_D), "max_q": max(qs), "max_kv": max(ks)}
    if own:  # the plan of the step and its workspace, made once for all layers
        import serving_attention_gb300 as fi

        cfg = fi.default_plan_config(0, max_batch=256, max_items=1 << 14, max_merge_units=1 << 13,
                                     max_partial_rows=1 << 17, kv_bits=4, window_left=c["window"],
                                     sink_tokens=c["sink"])
        s["ws"] = fi.Workspace(cfg)
        last = [k - (p - 1) * P if p else 0 for k, p in zip(ks, pages)]
        s["info"] = fi.plan(s["ws"], qo, kvp, [], last, c["heads"], Hk, _D, P, int(c["causal"]))
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((qo[-1], c["heads"]), dtype=torch.float32, device="cuda")
    return s


def _prepare_append(c, seed):
    g, dt, P, T, four = _gen(seed), _DT[c["dtype"]], c["page"], c["tokens"], c["op"] == "append4"
    H, Hk, n = c["heads"], c["kv_heads"], c["tokens"] + c["pad"]
    D = _D if four else c["dim"]
    f = [c["theta"] ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)]
    pool = -(-T // P) + 3
    # q, k and v as the projection leaves them: parts of one row
    qkv = _normal(g, (n, (H + 2 * Hk) * D), dt)
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[:T] = torch.randperm(pool * P, generator=g, device="cuda")[:T].to(torch.int32)
    positions = torch.zeros(n, dtype=torch.int32, device="cuda")
    positions[:T] = torch.randint(0, c["far"], (T,), generator=g, device="cuda").to(torch.int32)
    s = {"c": c, "q": qkv[:, :H * D].unflatten(1, (H, D)), "k": qkv[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D)),
         "v": qkv[:, (H + Hk) * D:].unflatten(1, (Hk, D)), "slots": slots, "positions": positions,
         "freq": torch.tensor(f, dtype=torch.float64, device="cuda"),
         # the rates in turns a position, as 64-bit fractions
         "turns": torch.tensor([_signed(int(math.ldexp(x / (2 * math.pi), 64) + 0.5)) for x in f], device="cuda"),
         "q_out": torch.zeros((n, H, D), dtype=dt, device="cuda")}
    if not four or c["norm"]:
        per_head = not four and c["per_head"]
        for name, heads in (("q_weight", H), ("k_weight", Hk)):
            s[name] = 1 + 0.1 * torch.randn((heads, D) if per_head else (D,), generator=g, device="cuda")
    else:
        s["q_weight"] = s["k_weight"] = None
    if four:
        s["cache"] = torch.zeros((pool, Hk, _page_bytes(P)), dtype=torch.uint8, device="cuda")
        s["all"] = torch.arange(pool * P, dtype=torch.int32, device="cuda")
        s["k_out"], s["v_out"] = (torch.zeros((pool * P, Hk, D), dtype=dt, device="cuda") for _ in range(2))
    else:
        s["k_cache"], s["v_cache"] = (_normal(g, (pool, P, Hk, D), dt) for _ in range(2))
    if own:
        from serving_attention_gb300 import step

        s["setup"] = step.rotary_setup(D, c["rot"], interleaved=c["interleaved"], theta=c["theta"])
    return s


def _signed(x):
    return x - (1 << 64) if x >= 1 << 63 else x


# ------------------------------------------------------- the 4-bit format

def _page_bytes(P):
    B = min(P, 32)
    return P // B * ((132 * B + 15) // 16 * 16)


def _codes(x):
    """Codes and words (s | z) of rows of 128 fp32 values.  Single fp32 operations in a fixed order: next to a border
    a code goes by the last bit."""
    lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
    bits = ((hi - lo) * (1 / 15)).to(torch.float16).view(torch.int16).to(torch.int32)
    bits = ((bits + 15) & ~15).clamp(max=0x6C00)  # 4096
    s = bits.to(torch.int16).view(torch.float16).float()
    inv = torch.where(s > 0, 1 / s, 0.0)
    z = torch.round(-lo * inv).clamp(0, 15)
    n = (torch.round(x * inv) + z).clamp(0, 15).to(torch.uint8)
    return n, (bits | z.to(torch.int32)).squeeze(-1).to(torch.int16)


def _packed(kn, kw, vn, vw, P):
    """Pages [N, Hk, bytes] from codes [N, P, Hk, 128] and words [N, P, Hk] of k and v."""
    N, B, Hk = kn.shape[0], min(P, 32), kn.shape[2]

    def part(x, width):  # [N, P, Hk, width] bytes -> [N, Hk, P / B, B * width]
        return x.view(N, P // B, B, Hk, width).permute(0, 3, 1, 2, 4).reshape(N, Hk, P // B, B * width)

    rows = [part(n[..., 0::2] | n[..., 1::2] << 4, 64) for n in (kn, vn)]
    words = [part(w.contiguous().view(torch.uint8).view(N, P, Hk, 2), 2) for w in (kw, vw)]
    out = torch.cat(rows + words, -1)
    return torch.nn.functional.pad(out, (0, _page_bytes(P) // (P // B) - out.shape[-1])).flatten(2)


def _parts(cache, P):
    """Views of a cache's rows of k and v [N, Hk, P / B, B, 64] and words [N, Hk, P / B, B, 2], all bytes."""
    B = min(P, 32)
    x = cache.view(*cache.shape[:2], P // B, -1)
    cut = [0, 64 * B, 128 * B, 130 * B, 132 * B]
    return [x[..., a:b].unflatten(-1, (B, -1)) for a, b in zip(cut, cut[1:])]


def _values(rows, words):
    """fp32 values [N * P, Hk, 128] of rows and words as _parts gives them (exact: at most 11 bits each)."""
    n = torch.stack([rows & 15, rows >> 4], -1).flatten(-2)
    w = words.contiguous().view(torch.int16)
    s = (w & ~15).view(torch.float16).float()
    x = (n.float() - (w & 15).float()) * s
    return x.flatten(2, 3).transpose(1, 2).flatten(0, 1)


# ------------------------------------------------------------------- runs

def run(s):
    return {"attend": _run_attend, "append4": _run_append4, "append16": _run_append16}[s["c"]["op"]](s)


def _run_attend(s):
    c = s["c"]
    if own:
        from serving_attention_gb300 import kv4

        kv4.run(s["ws"], s["info"], s["q"], s["cache"], s["kv_indices"], s["o"], s["lse"], s["scale"])
        return {"o": s["o"], "lse": s["lse"]}
    B, H, Hk, P, Lq, Lk = c["batch"], c["heads"], c["kv_heads"], c["page"], s["max_q"], s["max_kv"]
    G = H // Hk
    qo, kvp, kv_lens = s["qo_indptr"].long(), s["kv_indptr"].long(), s["kv_lens"].long()
    q_lens = qo[1:] - qo[:-1]
    j = torch.arange(Lk, device="cuda")
    t = torch.arange(Lq, device="cuda")
    there = j < kv_lens[:, None]
    page = s["kv_indices"].long()[(kvp[:-1, None] + j // P).clamp(max=s["kv_indices"].numel() - 1)]
    row = torch.where(there, page * P + j % P, 0)
    krows, vrows, kwords, vwords = _parts(s["cache"], P)
    zero = torch.zeros((), device="cuda")
    keys = _values(krows, kwords)[row]
    q = s["q"][(qo[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.view(B, Lq, Hk, G, _D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * Lq, _D)
    x = torch.matmul(q, keys.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, Hk, G, Lq, Lk)
    del keys
    pos = (kv_lens - q_lens)[:, None] + t
    see = there[:, None, :] & ((j <= pos[:, :, None]) if c["causal"] else torch.ones_like(pos, dtype=torch.bool)[:, :, None])
    if c["window"] >= 0:
        see = see & ((j >= pos[:, :, None] - c["window"]) | (j < c["sink"]))
    x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, zero, m)).exp_()
    l = x.sum(-1, keepdim=True)
    vals = _values(vrows, vwords)[row].permute(0, 2, 1, 3)
    o = torch.matmul(x.view(B, Hk, G * Lq, Lk), vals).view(B, Hk, G, Lq, _D)
    o = torch.where(l > 0, o / l, zero)
    lse = (m + l.log())[..., 0]
    n = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(qo[1:], n, right=True)
    return {"o": o.permute(0, 3, 1, 2, 4)[b, n - qo[b]].reshape(-1, H, _D).to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2)[b, n - qo[b]].reshape(-1, H)}


def _cos_sin(s):
    """cos and sin of each token's pairs: the angle's part of a turn from 64-bit integers."""
    turn = s["positions"].long()[:, None] * s["turns"]
    angle = (turn >> 32).float() * 2.0 ** -31 * math.pi
    return angle.cos(), angle.sin()


def _rotated(x, cos, sin, rot, interleaved):
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos[:, None] - x[..., b] * sin[:, None]
    y[..., b] = x[..., b] * cos[:, None] + x[..., a] * sin[:, None]
    return y


def _pairwise(y):
    """Sums of 128 values in pairs: halves of the row, then inside groups of 8, then over the groups."""
    y = (y[..., :64] + y[..., 64:]).unflatten(-1, (8, 8))
    y = y[..., :4] + y[..., 4:]
    y = y[..., :2] + y[..., 2:]
    y = y[..., 0] + y[..., 1]
    y = y[..., :4] + y[..., 4:]
    y = y[..., :2] + y[..., 2:]
    return y[..., :1] + y[..., 1:]


def _run_append4(s):
    c = s["c"]
    if own:
        from serving_attention_gb300 import kv4

        kv4.append(s["setup"], s["positions"], s["slots"], s["q"], s["q_out"], s["k"], s["v"], s["cache"], c["page"],
                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=_EPS)
        kv4.read(s["all"], s["cache"], c["page"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    cos, sin = _cos_sin(s)
    q, k = s["q"].float(), s["k"].float()
    if c["norm"]:  # sums in a fixed order, and single operations: the codes go by the last bit
        q = q * (1 / torch.sqrt(_pairwise(q * q) * (1 / _D) + _EPS)) * s["q_weight"]
        k = k * (1 / torch.sqrt(_pairwise(k * k) * (1 / _D) + _EPS)) * s["k_weight"]
    s["q_out"].copy_(_rotated(q, cos, sin, c["rot"], c["interleaved"]))
    kn, kw = _codes(_rotated(k, cos, sin, c["rot"], c["interleaved"]))
    vn, vw = _codes(s["v"].float())
    # rows without a slot (padding) are not written: they repeat the first token's write
    at = torch.where(s["slots"] >= 0, torch.arange(s["slots"].numel(), device="cuda"), 0)
    slot = s["slots"].long()[at]
    P, B = c["page"], min(c["page"], 32)
    krows, vrows, kwords, vwords = _parts(s["cache"], P)
    page, block, place = slot // P, slot % P // B, slot % B
    krows[page, :, block, place] = (kn[..., 0::2] | kn[..., 1::2] << 4)[at]
    vrows[page, :, block, place] = (vn[..., 0::2] | vn[..., 1::2] << 4)[at]
    kwords[page, :, block, place] = kw.contiguous().view(torch.uint8).unflatten(-1, (-1, 2))[at]
    vwords[page, :, block, place] = vw.contiguous().view(torch.uint8).unflatten(-1, (-1, 2))[at]
    s["k_out"].copy_(_values(krows, kwords))
    s["v_out"].copy_(_values(vrows, vwords))
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _run_append16(s):
    c = s["c"]
    if own:
        from serving_attention_gb300 import step

        step.norm_append(s["setup"], s["positions"], s["slots"], s["q"], s["q_out"], s["q_weight"], s["k"],
                         s["k_weight"], s["v"], s["k_cache"], s["v_cache"], eps=_EPS)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    cos, sin = _cos_sin(s)
    q, k = s["q"].float(), s["k"].float()
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + _EPS) * s["q_weight"]
    k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + _EPS) * s["k_weight"]
    at = torch.where(s["slots"] >= 0, torch.arange(s["slots"].numel(), device="cuda"), 0)
    slot = s["slots"].long()[at]
    s["q_out"].copy_(_rotated(q, cos, sin, c["rot"], c["interleaved"]))
    k = _rotated(k, cos, sin, c["rot"], c["interleaved"]).to(s["k"].dtype)
    s["k_cache"].view(-1, *k.shape[1:])[slot] = k[at]
    s["v_cache"].view(-1, *s["v"].shape[1:])[slot] = s["v"][at]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ------------------------------------------------------------------ exact

def exact(c, seed):
    s = prepare(c, seed)
    return {"attend": _exact_attend, "append4": _exact_append, "append16": _exact_append}[c["op"]](s)


def _held(cache, P, h, ids, n, which):
    """fp64 values [n, 128] of the first n slots of pages `ids`, head h: which = 0 for k, 1 for v."""
    B = min(P, 32)
    blocks = cache[ids, h].view(-1, cache.shape[-1] * B // P).long()
    codes = blocks[:, 64 * B * which:64 * B * (which + 1)].reshape(-1, 64)
    at = 128 * B + 2 * B * which
    word = blocks[:, at:at + 2 * B:2] + 256 * blocks[:, at + 1:at + 2 * B:2]
    word = word.reshape(-1, 1)[:n]
    e, f = word >> 10, (word & 0x3F0).double() / 1024
    s = torch.where(e == 0, torch.ldexp(f, e - 14), torch.ldexp(1 + f, e - 15))
    out = torch.empty(n, _D, dtype=torch.float64, device="cuda")
    out[:, 0::2] = (codes[:n] % 16 - word % 16) * s
    out[:, 1::2] = (codes[:n] // 16 - word % 16) * s
    return out


def _exact_attend(s):
    """Request by request and key head by key head."""
    c = s["c"]
    H, Hk, P = c["heads"], c["kv_heads"], c["page"]
    G, out, lses = H // Hk, [], []
    qo, kvp = s["qo_indptr"].tolist(), s["kv_indptr"].tolist()
    for b, n in enumerate(s["kv_lens"].tolist()):
        ids = s["kv_indices"][kvp[b]:kvp[b + 1]].long()
        q = s["q"][qo[b]:qo[b + 1]].double()
        L = q.shape[0]
        pos = torch.arange(L, device="cuda")[:, None] + (n - L)
        key = torch.arange(n, device="cuda")[None]
        see = key <= pos if c["causal"] else key < n + 0 * pos
        if c["window"] >= 0:
            see = see & ((key >= pos - c["window"]) | (key < c["sink"]))
        o = torch.zeros(L, H, _D, dtype=torch.float64, device="cuda")
        lse = torch.full((L, H), -math.inf, dtype=torch.float64, device="cuda")
        for h in range(Hk):
            k, v = _held(s["cache"], P, h, ids, n, 0), _held(s["cache"], P, h, ids, n, 1)
            for a in range(h * G, (h + 1) * G):
                x = (q[:, a] @ k.T * s["scale"]).masked_fill(~see, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[:, a] = z
                o[:, a] = torch.exp(x - torch.where(z.isinf(), 0.0, z)[:, None]) @ v
        out.append(o)
        lses.append(lse)
    return {"o": torch.cat(out), "lse": torch.cat(lses)}


def _exact_append(s):
    """Norm, then pairs as complex numbers, each turned by its angle; of the 4-bit cache, the definition of its codes."""
    c, n = s["c"], s["c"]["tokens"]
    angle = s["positions"].double()[:, None, None] * s["freq"]
    turn = torch.polar(torch.ones_like(angle), angle)

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + _EPS).sqrt() * w.double()
        head, tail = x[..., :c["rot"]], x[..., c["rot"]:]
        pairs = head.unflatten(-1, (-1, 2)) if c["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, tail], -1)

    def held(x):
        x = x.double()
        lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
        near = ((hi - lo) / 15).to(torch.float16).double()
        # seven significant bits, upwards (a step of 2^-20 below the smallest normal number)
        step = torch.ldexp(torch.ones_like(near), torch.frexp(near.clamp(min=2.0 ** -14))[1] - 7)
        s = (torch.ceil(near / step) * step).clamp(max=4096.0)
        z = torch.where(s > 0, torch.round(-lo / s), 0).clamp(0, 15)
        return torch.where(s > 0, ((torch.round(x / s) + z).clamp(0, 15) - z) * s, 0)

    slot = s["slots"][:n].long()
    if c["op"] == "append4":
        k, v = (torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
        k[slot], v[slot] = held(turned(s["k"], s["k_weight"]))[:n], held(s["v"])[:n]
        return {"q": turned(s["q"], s["q_weight"]), "k": k, "v": v}
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k_cache.flatten(0, 1)[slot] = turned(s["k"], s["k_weight"])[:n]
    v_cache.flatten(0, 1)[slot] = s["v"][:n].double()
    return {"q": turned(s["q"], s["q_weight"]), "k_cache": k_cache, "v_cache": v_cache}
