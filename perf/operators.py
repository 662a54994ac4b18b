"""Measured cases of the step operators: differential attention over the paged
cache, rotary positions written with the keys and values into that cache, and
the page tables and slot maps of a step built on the GPU.

listed() and draw() give cases (dicts of plain values), prepare() what a
serving program has in hand before the call, run() one call, work() the bytes
and operations that the call cannot do without, exact() its result in 64 bits.
run() computes the plain form in elementary torch operations, or, where `own`
is true, calls the library.

Differential attention, per query row and head h with halves q = [q1 | q2] and
keys k = [k1 | k2] of 64 dims each, values of 128:
    o = S1 - lambda_h S2,  S_i = softmax(scale q_i k_i^T + mask) V
    o = out_scale * o                                   without a norm, or
    o = out_scale * o / sqrt(mean(o^2) + eps) * w       with one.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few short requests, one token each: the latency of one call
        dict(name="diff_decode_small", op="diff", dtype="fp16", batch=4, prefills=0, q_lo=1, q_hi=1, prefix=0, kv_lo=1,
             kv_hi=512, heads=8, kv_heads=2, page=16, causal=False, norm=True, window=-1, sink=0, lens=1),
        # a serving batch of 64 single-token requests, lengths from 512 to 32768
        dict(name="diff_decode_batch", op="diff", dtype="bf16", batch=64, prefills=0, q_lo=1, q_hi=1, prefix=0,
             kv_lo=512, kv_hi=32768, heads=32, kv_heads=8, page=16, causal=False, norm=True, window=-1, sink=0,
             lens=2),
        # two long contexts, eight query heads per key head: the keys have to be split over the card
        dict(name="diff_decode_long", op="diff", dtype="bf16", batch=2, prefills=0, q_lo=1, q_hi=1, prefix=0,
             kv_lo=99991, kv_hi=131072, heads=64, kv_heads=8, page=64, causal=False, norm=False, window=-1, sink=0,
             lens=3),
        # 64 branches with a short private part on pages of one token
        dict(name="diff_decode_page1", op="diff", dtype="bf16", batch=64, prefills=0, q_lo=1, q_hi=1, prefix=0,
             kv_lo=64, kv_hi=512, heads=32, kv_heads=8, page=1, causal=False, norm=True, window=-1, sink=0, lens=4),
        # prompts being read, some behind an earlier part of the conversation
        dict(name="diff_prefill", op="diff", dtype="bf16", batch=8, prefills=8, q_lo=128, q_hi=2048, prefix=2048,
             kv_lo=0, kv_hi=0, heads=32, kv_heads=8, page=16, causal=True, norm=True, window=-1, sink=0, lens=5),
        # a mixed step with a sliding window and sink tokens: four prompt parts beside 24 decoding requests
        dict(name="diff_mixed_window", op="diff", dtype="fp16", batch=28, prefills=4, q_lo=100, q_hi=256, prefix=4000,
             kv_lo=16, kv_hi=4096, heads=16, kv_heads=4, page=16, causal=True, norm=True, window=1023, sink=4,
             lens=6),
        # one decode step: 64 new tokens rotated and written to the cache
        dict(name="rope_append_decode", op="rope", dtype="bf16", tokens=64, pad=0, heads=32, kv_heads=8, dim=128,
             v_dim=128, rot=128, interleaved=False, scaling="by_parts", factor=8.0, theta=500000.0, far=131072,
             page=16),
        # a long prompt's tokens
        dict(name="rope_append_prefill", op="rope", dtype="bf16", tokens=16384, pad=0, heads=32, kv_heads=8, dim=128,
             v_dim=128, rot=128, interleaved=False, scaling="none", factor=1.0, theta=500000.0, far=16384, page=16),
        # part of a head of 80 dims, neighbouring pairs, an odd count padded to a captured size
        dict(name="rope_append_partial", op="rope", dtype="fp16", tokens=1111, pad=41, heads=24, kv_heads=24, dim=80,
             v_dim=80, rot=32, interleaved=True, scaling="yarn", factor=16.0, theta=10000.0, far=1000000, page=8),
        # a latent cache: one rotated key of 64 dims for all 128 heads, the latent row beside it
        dict(name="rope_append_latent", op="rope", dtype="bf16", tokens=333, pad=3, heads=128, kv_heads=1, dim=64,
             v_dim=512, rot=64, interleaved=True, scaling="yarn", factor=40.0, theta=10000.0, far=163840, page=64),
        # the tables of a decode step of 64 requests
        dict(name="tables_decode", op="tables", batch=64, prefills=0, chunk=1, kv_lo=512, kv_hi=32768, page=16, pad=0,
             lens=7),
        # a full house: 4096 requests, some of them reading prompts
        dict(name="tables_large", op="tables", batch=4096, prefills=32, chunk=512, kv_lo=128, kv_hi=32768, page=16,
             pad=480, lens=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["diff", "diff", "diff", "rope", "rope", "tables"])
    if op == "diff":
        while True:
            kv_heads = rng.choice([1, 2, 4, 8])
            heads = kv_heads * rng.choice([1, 2, 4, 4, 8, 16])
            if heads > 64:
                continue
            batch = _log(rng, 1, 64)
            kind = rng.choice(["decode", "decode", "prefill", "mixed"])
            prefills = {"decode": 0, "prefill": batch, "mixed": max(1, batch // 6)}[kind]
            q_hi = _log(rng, 2, 2048) if prefills else 1
            prefix = _log(rng, 1, 4096) if prefills else 0
            kv_hi = _log(rng, 64, 4096 if prefills else 131072)
            window = _log(rng, 16, 4096) if rng.random() < 0.25 else -1
            c = dict(op="diff", dtype=rng.choice(["bf16", "fp16"]), batch=batch, prefills=prefills,
                     q_lo=max(1, q_hi // 8), q_hi=q_hi, prefix=prefix, kv_lo=max(1, kv_hi // 64), kv_hi=kv_hi,
                     heads=heads, kv_heads=kv_heads, page=rng.choice([1, 8, 16, 16, 32, 64]), causal=prefills > 0,
                     norm=rng.random() < 0.6, window=window, sink=rng.choice([0, 4]) if window >= 0 else 0,
                     lens=rng.randrange(1 << 20))
            rows = c["batch"] * max(l[1] for l in _lens(c))
            if (rows * kv_heads <= 64 * 32768 * 8 and rows * q_hi * heads <= 8 * 2048 * 4096 * 32
                    and _diff_work(c)["flops"] <= 3.0e11 and _diff_work(c)["bytes"] <= 1.6e9):
                return c
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        rot = rng.choice([dim, dim, 32, 64])
        kv_heads = rng.choice([1, 2, 4, 8])
        tokens = _log(rng, 1, 16384 if dim <= 128 else 8192)
        return dict(op="rope", dtype=rng.choice(["bf16", "fp16"]), tokens=tokens, pad=rng.choice([0, 0, 1, 7]),
                    heads=kv_heads * rng.choice([1, 2, 4]), kv_heads=kv_heads, dim=dim, v_dim=dim,
                    rot=rot, interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "by_parts", "yarn"]),
                    factor=rng.choice([2.0, 8.0, 32.0]), theta=rng.choice([10000.0, 500000.0]),
                    far=max(tokens, _log(rng, 1000, 1000000)), page=rng.choice([1, 8, 16, 64]))
    batch = _log(rng, 1, 4096)
    return dict(op="tables", batch=batch, prefills=rng.choice([0, min(batch, 8)]), chunk=_log(rng, 2, 1024),
                kv_lo=16, kv_hi=_log(rng, 64, 32768), page=rng.choice([8, 16, 32, 64]), pad=rng.randrange(64),
                lens=rng.randrange(1 << 20))


def _lens(c):
    """(query tokens, keys with those tokens) of each request of a diff or tables case."""
    r = random.Random(c["lens"])
    got = []
    for b in range(c["batch"]):
        if b < c["prefills"] and c["op"] == "diff":
            q = r.randint(c["q_lo"], c["q_hi"])
            got.append((q, q + r.randint(0, c["prefix"])))
        else:
            kv = _log(r, c["kv_lo"], c["kv_hi"])
            got.append((min(kv, r.randint(1, c["chunk"])) if b < c["prefills"] else 1, kv))
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


def _diff_work(c):
    pairs, keys = _visible(c)
    tokens = sum(l[0] for l in _lens(c))
    return {"bytes": keys * c["kv_heads"] * 512 + tokens * c["heads"] * (512 + 8), "flops": pairs * c["heads"] * 768}


def work(c):
    if c["op"] == "diff":
        return _diff_work(c)
    if c["op"] == "rope":
        row = 2 * c["heads"] * c["dim"] + 2 * c["kv_heads"] * (c["dim"] + c["v_dim"])
        return {"bytes": c["tokens"] * (2 * row + 8), "flops": 3 * c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rot"]}
    lens = _lens(c)
    P = c["page"]
    pages = sum(-(-kv // P) for _, kv in lens)
    tokens = sum(q for q, _ in lens)
    return {"bytes": 4 * (2 * c["batch"] + 3 * c["batch"] + 2 * pages + 2 * (tokens + c["pad"])), "flops": 4 * pages}


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
    return {"diff": _prepare_diff, "rope": _prepare_rope, "tables": _prepare_tables}[c["op"]](c, seed)


def _prepare_diff(c, seed):
    g, dt, P = _gen(seed), _DT[c["dtype"]], c["page"]
    lens = _lens(c)
    qs, ks = [l[0] for l in lens], [l[1] for l in lens]
    pages = [-(-k // P) for k in ks]
    used = sum(pages)
    pool = used + 7
    qo, kvp = _indptr(qs), _indptr(pages)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    s = {"c": c, "qo_indptr": _i32(qo), "kv_indptr": _i32(kvp), "kv_lens": _i32(ks), "kv_indices": perm[:used].contiguous(),
         "q": _normal(g, (qo[-1], c["heads"], 128), dt), "scale": 0.125, "max_q": max(qs), "max_kv": max(ks),
         "k": _normal(g, (pool, P, c["kv_heads"], 128), dt), "v": _normal(g, (pool, P, c["kv_heads"], 128), dt),
         "lam": 0.2 + 0.6 * torch.rand(c["heads"], generator=g, device="cuda"),
         "w": 1 + 0.1 * torch.randn(128, generator=g, device="cuda") if c["norm"] else None, "out_scale": 0.2}
    if own:  # the plan of the step and its workspace, made once for all layers
        import serving_attention_gb300 as fi

        cfg = fi.default_plan_config(0, max_batch=256, max_items=1 << 14, max_merge_units=1 << 13,
                                     max_partial_rows=1 << 17, differential=1, window_left=c["window"],
                                     sink_tokens=c["sink"])
        s["ws"] = fi.Workspace(cfg)
        last = [k - (p - 1) * P if p else 0 for k, p in zip(ks, pages)]
        s["info"] = fi.plan(s["ws"], qo, kvp, [], last, c["heads"], c["kv_heads"], 128, P, int(c["causal"]))
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((qo[-1], c["heads"], 2), dtype=torch.float32, device="cuda")
    return s


def _frequencies(c):
    """Radians per position of each rotated pair, and the factor on cos and sin."""
    rot, theta, s, kind = c["rot"], c["theta"], c["factor"], c["scaling"]
    n, orig = rot // 2, 8192
    if kind == "ntk":
        theta *= s ** (rot / (rot - 2))
    f = [theta ** (-2.0 * i / rot) for i in range(n)]
    amp = 1.0
    if kind == "linear":
        f = [x / s for x in f]
    elif kind == "by_parts":  # pairs that turn over 4 times in the old length keep their rate, under once: slowed
        keep = [min(1.0, max(0.0, (orig * x / (2 * math.pi) - 1.0) / 3.0)) for x in f]
        f = [x * k + x / s * (1 - k) for x, k in zip(f, keep)]
    elif kind == "yarn":  # between the pairs that turn 32 times and once, linearly in the pair's number
        at = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
        slow = [min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 1e-3))) for i in range(n)]
        f = [x / s * k + x * (1 - k) for x, k in zip(f, slow)]
        amp = 0.1 * math.log(s) + 1.0
    return f, amp


def _prepare_rope(c, seed):
    g, dt, P, T = _gen(seed), _DT[c["dtype"]], c["page"], c["tokens"]
    H, Hk, D, Dv, n = c["heads"], c["kv_heads"], c["dim"], c["v_dim"], c["tokens"] + c["pad"]
    f, amp = _frequencies(c)
    pool = -(-T // P) * 2 + 3
    # q, k and v as the projection leaves them: parts of one row
    qkv = _normal(g, (n, H * D + Hk * D + Hk * Dv), dt)
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[:T] = torch.randperm(pool * P, generator=g, device="cuda")[:T].to(torch.int32)
    positions = torch.zeros(n, dtype=torch.int32, device="cuda")
    positions[:T] = torch.randint(0, c["far"], (T,), generator=g, device="cuda").to(torch.int32)
    s = {"c": c, "q": qkv[:, :H * D].unflatten(1, (H, D)), "k": qkv[:, H * D:H * D + Hk * D].unflatten(1, (Hk, D)),
         "v": qkv[:, H * D + Hk * D:].unflatten(1, (Hk, Dv)), "slots": slots, "positions": positions,
         "freq": torch.tensor(f, dtype=torch.float64, device="cuda"), "amp": amp,
         "q_out": torch.zeros((n, H, D), dtype=dt, device="cuda"), "k_cache": _normal(g, (pool, P, Hk, D), dt),
         "v_cache": _normal(g, (pool, P, Hk, Dv), dt)}
    if own:
        from serving_attention_gb300 import step

        s["setup"] = step.rotary_setup(D, c["rot"], interleaved=c["interleaved"], theta=c["theta"], scaling=c["scaling"],
                                     factor=c["factor"], original_positions=8192)
    return s


def _prepare_tables(c, seed):
    g, P = _gen(seed), c["page"]
    lens = _lens(c)
    B = c["batch"]
    pages = [-(-kv // P) for _, kv in lens]
    old = [-(-(kv - q) // P) for q, kv in lens]
    width, taken, first = max(pages) + 3, sum(pages) - sum(old), 11
    ids = torch.randperm(B * width + taken + 64, generator=g, device="cuda").to(torch.int32)
    table = ids[:B * width].view(B, width).contiguous()
    col = torch.arange(width, device="cuda")
    table[col >= _i32(old)[:, None]] = -1  # not given out yet
    s = {"c": c, "qo_lens": _i32([q for q, _ in lens]), "kv_lens": _i32([kv for _, kv in lens]), "table": table,
         "free": ids[B * width:].contiguous(), "head": _i32([first]), "max_pages": sum(pages) + 5,
         "max_tokens": sum(q for q, _ in lens) + c["pad"]}
    if own:
        from serving_attention_gb300 import step

        s["out"] = step.StepTables(B, s["max_pages"], s["max_tokens"])
    return s


# ------------------------------------------------------------------- runs

def run(s):
    return {"diff": _run_diff, "rope": _run_rope, "tables": _run_tables}[s["c"]["op"]](s)


def _run_diff(s):
    c = s["c"]
    if own:
        from serving_attention_gb300 import differential

        differential.run(s["ws"], s["info"], s["q"], s["k"], s["v"], s["kv_indices"], s["lam"], s["o"], s["lse"],
                         s["scale"], norm_weight=s["w"], norm_eps=_EPS, out_scale=s["out_scale"])
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
    zero = torch.zeros((), device="cuda")
    keys = torch.where(there[:, :, None, None], s["k"].view(-1, Hk, 128)[row].float(), zero)
    vals = torch.where(there[:, :, None, None], s["v"].view(-1, Hk, 128)[row].float(), zero)
    q = s["q"][(qo[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.view(B, Lq, Hk, G, 2, 64).permute(0, 2, 4, 3, 1, 5).reshape(B, Hk, 2, G * Lq, 64)
    keys = keys.view(B, Lk, Hk, 2, 64).permute(0, 2, 3, 4, 1)
    x = torch.matmul(q, keys).mul_(s["scale"]).view(B, Hk, 2, G, Lq, Lk)
    del keys
    pos = (kv_lens - q_lens)[:, None] + t
    see = there[:, None, :] & ((j <= pos[:, :, None]) if c["causal"] else torch.ones_like(pos, dtype=torch.bool)[:, :, None])
    if c["window"] >= 0:
        see = see & ((j >= pos[:, :, None] - c["window"]) | (j < c["sink"]))
    x.masked_fill_(~see[:, None, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, zero, m)).exp_()
    l = x.sum(-1, keepdim=True)
    vals = vals.permute(0, 2, 1, 3)[:, :, None]
    o = torch.matmul(x.view(B, Hk, 2, G * Lq, Lk), vals).view(B, Hk, 2, G, Lq, 128)
    o = torch.where(l > 0, o / l, zero)
    lse = m + l.log()
    y = o[:, :, 0] - s["lam"].view(1, Hk, G, 1, 1) * o[:, :, 1]
    if s["w"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS) * s["w"]
    y = y * s["out_scale"]
    n = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(qo[1:], n, right=True)
    return {"o": y.permute(0, 3, 1, 2, 4)[b, n - qo[b]].reshape(-1, H, 128).to(s["q"].dtype),
            "lse": lse[..., 0].permute(0, 4, 1, 3, 2)[b, n - qo[b]].reshape(-1, H, 2)}


def _rotated(x, cos, sin, rot, interleaved):
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos[:, None] - x[..., b] * sin[:, None]
    y[..., b] = x[..., b] * cos[:, None] + x[..., a] * sin[:, None]
    return y


def _run_rope(s):
    c = s["c"]
    if own:
        from serving_attention_gb300 import step

        step.append(s["setup"], s["positions"], s["slots"], s["q"], s["q_out"], s["k"], s["v"], s["k_cache"],
                    s["v_cache"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    dt = s["q"].dtype
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = (angle.cos() * s["amp"]).float(), (angle.sin() * s["amp"]).float()
    # rows without a slot (padding) are not written: they repeat the first token's write
    at = torch.where(s["slots"] >= 0, torch.arange(s["slots"].numel(), device="cuda"), 0)
    slot = s["slots"].long()[at]
    s["q_out"].copy_(_rotated(s["q"].float(), cos, sin, c["rot"], c["interleaved"]))
    k = _rotated(s["k"].float(), cos, sin, c["rot"], c["interleaved"]).to(dt)
    s["k_cache"].view(-1, *k.shape[1:])[slot] = k[at]
    s["v_cache"].view(-1, *s["v"].shape[1:])[slot] = s["v"][at]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _run_tables(s):
    c = s["c"]
    if own:
        from serving_attention_gb300 import step

        t = s["out"]
        step.build_tables(t, s["qo_lens"], s["kv_lens"], s["table"], c["page"], s["free"], s["head"])
        return {"qo_indptr": t.qo_indptr, "kv_indptr": t.kv_indptr, "last_page_len": t.last_page_len,
                "kv_indices": t.kv_indices, "positions": t.positions, "slots": t.slots, "table": s["table"],
                "counts": t.counts[:4]}
    P = c["page"]
    q, kv = s["qo_lens"].long(), s["kv_lens"].long()
    old = kv - q
    pages, had = (kv + P - 1) // P, (old + P - 1) // P
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    qo, kvp = torch.cat([zero, q.cumsum(0)]), torch.cat([zero, pages.cumsum(0)])
    new = (pages - had).cumsum(0)
    col = torch.arange(s["table"].shape[1], device="cuda")
    take = (col >= had[:, None]) & (col < pages[:, None])
    src = s["head"].long() + (new - (pages - had))[:, None] + col - had[:, None]
    s["table"].copy_(torch.where(take, s["free"][src.clamp(0, s["free"].numel() - 1)], s["table"]))
    e = torch.arange(s["max_pages"], device="cuda")
    b = torch.searchsorted(kvp[1:], e, right=True).clamp(max=c["batch"] - 1)
    ids = torch.where(e < kvp[-1], s["table"][b, (e - kvp[b]).clamp(max=s["table"].shape[1] - 1)], -1)
    n = torch.arange(s["max_tokens"], device="cuda")
    b = torch.searchsorted(qo[1:], n, right=True).clamp(max=c["batch"] - 1)
    pos = torch.where(n < qo[-1], old[b] + n - qo[b], 0)
    slots = torch.where(n < qo[-1], s["table"][b, pos // P] * P + pos % P, -1)
    i = torch.int32
    return {"qo_indptr": qo.to(i), "kv_indptr": kvp.to(i), "kv_indices": ids.to(i), "positions": pos.to(i),
            "slots": slots.to(i), "table": s["table"],
            "last_page_len": torch.where(pages > 0, kv - (pages - 1) * P, 0).to(i),
            "counts": torch.stack([qo[-1], kvp[-1], new[-1], s["head"][0] + new[-1]]).to(i)}


# ------------------------------------------------------------------ exact

def exact(c, seed):
    if c["op"] == "tables":
        return None  # whole numbers
    s = prepare(c, seed)
    return _exact_diff(s) if c["op"] == "diff" else _exact_rope(s)


def _exact_diff(s):
    """Request by request and key head by key head."""
    c = s["c"]
    H, Hk, P = c["heads"], c["kv_heads"], c["page"]
    G, out, lses = H // Hk, [], []
    qo, kvp = s["qo_indptr"].tolist(), s["kv_indptr"].tolist()
    lam = s["lam"].double()
    for b, n in enumerate(s["kv_lens"].tolist()):
        ids = s["kv_indices"][kvp[b]:kvp[b + 1]].long()
        q = s["q"][qo[b]:qo[b + 1]].double()
        L = q.shape[0]
        pos = torch.arange(L, device="cuda")[:, None] + (n - L)
        key = torch.arange(n, device="cuda")[None]
        see = key <= pos if c["causal"] else key < n + 0 * pos
        if c["window"] >= 0:
            see = see & ((key >= pos - c["window"]) | (key < c["sink"]))
        o = torch.zeros(L, H, 128, dtype=torch.float64, device="cuda")
        lse = torch.full((L, H, 2), -math.inf, dtype=torch.float64, device="cuda")
        for h in range(Hk):
            k = s["k"][ids, :, h].reshape(-1, 128)[:n].double()
            v = s["v"][ids, :, h].reshape(-1, 128)[:n].double()
            for a in range(h * G, (h + 1) * G):
                for half, sign in ((0, 1.0), (1, -lam[a])):
                    d = slice(64 * half, 64 * half + 64)
                    x = (q[:, a, d] @ k[:, d].T * s["scale"]).masked_fill(~see, -math.inf)
                    z = torch.logsumexp(x, -1)
                    lse[:, a, half] = z
                    o[:, a] += sign * (torch.exp(x - torch.where(z.isinf(), 0.0, z)[:, None]) @ v)
        out.append(o)
        lses.append(lse)
    o = torch.cat(out)
    if s["w"] is not None:
        o = o / (o.square().mean(-1, keepdim=True) + _EPS).sqrt() * s["w"].double()
    return {"o": o * s["out_scale"], "lse": torch.cat(lses)}


def _exact_rope(s):
    """Pairs as complex numbers, each turned by its angle."""
    c, n = s["c"], s["c"]["tokens"]
    angle = s["positions"].double()[:, None, None] * s["freq"]
    turn = torch.polar(torch.full_like(angle, s["amp"]), angle)

    def rotated(x):
        x = x.double()
        head, tail = x[..., :c["rot"]], x[..., c["rot"]:]
        pairs = head.unflatten(-1, (-1, 2)) if c["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, tail], -1)

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    slot = s["slots"][:n].long()
    k_cache.flatten(0, 1)[slot] = rotated(s["k"])[:n]
    v_cache.flatten(0, 1)[slot] = s["v"][:n].double()
    return {"q": rotated(s["q"]), "k_cache": k_cache, "v_cache": v_cache}
