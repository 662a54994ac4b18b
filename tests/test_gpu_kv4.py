"""The 4-bit cache on the GPU against its oracle.

The append's codes are compared to the bit where no rotation comes before them
(a rotation's cos and sin are not the oracle's): then by their definition.

Attention, per row: a softmax weight enters as fp16, off by at most 2^-11 of
itself (2^-12 for half a step: doubled where the sum that divides it is of the
rounded weights) or, below 2^-14 of the largest weight in store, by 2^-25 of the
unit of its values; logits, sums and exponentials in fp32 add less than 1e-4
(528 products' magnitudes of up to 46 at 2^-23 each are 3e-5).  So
|o - ref| <= (2^-11 + 1e-4) sum_j p_j |v_j| + n 2^-24 max |v| + half a step of the output."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_attention_gb300 as fi
import workloads
from oracle import kv4 as oracle_kv4
from oracle import step as oracle_step
from serving_attention_gb300 import kv4, step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * std).to(DT[dtype])


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ append

def _strided_cache(pages, page, heads, fill=0xA5):
    """A cache inside a larger buffer, heads outside pages, with bytes around every page."""
    n = kv4.page_bytes(page)
    buf = torch.full((heads + 1, pages, n + 32), fill, dtype=torch.uint8, device=DEV)
    return buf[:heads, :, 16:16 + n].transpose(0, 1), buf


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(6, 3), (0, 8), (16, 1)])
def test_append_to_the_bit(dtype, page, heads, kv_heads):
    """Norms and quantiser without a rotation, padding tokens, strided operands: every byte of the cache."""
    T, pages = 41, -(-41 // page) + 2
    cache, buf = _strided_cache(pages, page, kv_heads)
    rng = np.random.default_rng(page)
    slots = rng.permutation(pages * page)[:T]
    slots[::7] = [-1, pages * page, -2**31, 2**31 - 1, -5, pages * page + 7][: len(slots[::7])]
    wide = _randn((T, heads + 2 * kv_heads, 136), dtype, page + heads)
    wide *= torch.exp(torch.linspace(-9, 9, T, device=DEV))[:, None, None].to(wide.dtype)  # rows of every size
    q, k, v = wide[:, :heads, :128], wide[:, heads:heads + kv_heads, 8:], wide[:, heads + kv_heads:, :128]
    qw, kw = 1 + 0.2 * torch.randn(max(heads, 1), 128, generator=_gen(1), device=DEV), \
        1 + 0.2 * torch.randn(128, generator=_gen(2), device=DEV)
    qw = qw[:heads] if heads else None
    q_out = torch.full_like(q, 3.0) if heads else None
    kv4.append(None, None, _i32(slots), q if heads else None, q_out, k, v, cache, page, q_weight=qw, k_weight=kw,
               eps=1e-5)
    want = np.full(cache.shape, 0xA5, np.uint8)
    kn = oracle_kv4.norm_exact_order(k.float().cpu().numpy(), kw.cpu().numpy(), 1e-5)
    vn = v.float().cpu().numpy()
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            for h in range(kv_heads):
                oracle_kv4.put(want, page, int(s), h, kn[t, h], vn[t, h])
    assert np.array_equal(cache.cpu().numpy(), want)
    around = buf.clone()
    around[:kv_heads, :, 16:-16] = 0xA5
    assert (around == 0xA5).all()  # nothing outside the cache
    if heads:
        ref = torch.from_numpy(oracle_kv4.norm_exact_order(q.float().cpu().numpy(), qw.cpu().numpy(), 1e-5))
        assert torch.equal(q_out.cpu(), ref.to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_extremes(dtype):
    """Zeros, one value, infinities, NaN, subnormals and the largest numbers."""
    top = torch.finfo(DT[dtype]).max
    tiny = torch.finfo(DT[dtype]).smallest_normal
    rows = torch.zeros((12, 1, 128), device=DEV)
    rows[1, 0, 7] = 1.0
    rows[2, 0, 7], rows[2, 0, 9] = float("inf"), 1.0
    rows[3, 0, 7], rows[3, 0, 9] = float("-inf"), 1.0
    rows[4] = float("nan")
    rows[5, 0, ::2], rows[5, 0, 1::2] = float("nan"), 2.0
    rows[6], rows[7] = top, -top
    rows[8, 0, 0], rows[8, 0, 1] = top, -top
    rows[9] = tiny
    rows[10, 0, 3] = tiny / 4
    rows[11, 0] = torch.linspace(-2.0**-20, 2.0**-20, 128, device=DEV)
    x = rows.to(DT[dtype])
    cache = kv4.empty_cache(2, 8, 1, DEV)
    kv4.append(None, None, _i32(range(12)), None, None, x, x, cache, 8)
    want = np.zeros(cache.shape, np.uint8)
    for t in range(12):
        oracle_kv4.put(want, 8, t, 0, x[t, 0].float().cpu().numpy(), x[t, 0].float().cpu().numpy())
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (64, True), (16, False), (80, False),
                                             (112, False), (96, True), (32, False)])
@pytest.mark.parametrize("norm", [False, True])
def test_append_rotated(dtype, rot, interleaved, norm):
    T, H, Hk, P = 37, 5, 3, 16
    r = step.rotary_setup(128, rot, interleaved, 500000.0, "yarn", 8.0, 8192)
    f, amp = oracle_step.rates(rot, 500000.0, "yarn", 8.0, 8192, 1.0, 32.0)
    pos = [0, 1, 2, 131071, 1000003, 2**31 - 1, -5] + list(range(100, 100 + T - 7))
    qkv = _randn((T, H + 2 * Hk, 128), dtype, rot + norm)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    w = [1 + 0.2 * torch.randn(128, generator=_gen(i), device=DEV) for i in (5, 6)] if norm else [None, None]
    pages = 4
    cache, _ = _strided_cache(pages, P, Hk)
    slots = np.random.default_rng(rot).permutation(pages * P)[:T]
    q_out = torch.empty_like(q)
    kv4.append(r, _i32(pos), _i32(slots), q, q_out, k, v, cache, P, q_weight=w[0], k_weight=w[1])

    def turned(x, weight):
        x = _f64(x)
        if weight is not None:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * _f64(weight)
        return oracle_step.rotate(x, pos, f, amp, rot, interleaved)

    # an angle's fp32 rounding (2^-24 of half a turn, up to pi 2^-24 = 2e-7), cosf and sinf (2 ulp), the norm's factor
    # (2^-23) and the products' roundings: below 1e-6 of the pair
    size = 2 * amp * 4.5 * 1e-6
    ref = turned(q, w[0])
    half = torch.finfo(DT[dtype]).eps / 2
    assert (np.abs(_f64(q_out) - ref) <= size + half * np.abs(ref) * (1 + 1e-6) + 1e-7).all()
    ref = turned(k, w[1])
    got_bytes = cache.cpu().numpy()
    for t in range(T):
        for h in range(Hk):
            got, got_v = oracle_kv4.get(got_bytes, P, int(slots[t]), h)
            want_v = oracle_kv4.values(*oracle_kv4.quantise(v[t, h].float().cpu().numpy()[None]))[0]
            assert np.array_equal(got_v, want_v)
            at = oracle_kv4.places(P, int(slots[t]) % P)[2]
            page = got_bytes[int(slots[t]) // P, h]
            word = int(page[at]) + 256 * int(page[at + 1])
            s = float(np.uint16(word & 0xFFF0).view(np.float16))
            exact = (max(ref[t, h].max(), 0) - min(ref[t, h].min(), 0)) / 15
            assert exact * (1 - 2.0**-11) - size <= s <= exact * (1 + 2.0**-11 + 15 / 1024) + size
            z = word & 15
            t0 = ref[t, h] / s + z  # the code before it is rounded
            n = got / s + z
            assert (np.abs(n - np.clip(t0, 0, 15)) <= 0.5 + size / s + 1e-4).all()


def test_append_does_not_depend_on_the_batch():
    """A token's bytes are the same alone and among thousands, whatever warps share it."""
    T, H, Hk, P = 5000, 8, 4, 32
    r = step.rotary_setup(128, theta=1e6)
    qkv = _randn((T, H + 2 * Hk, 128), "bf16", 3)
    w = 1 + 0.1 * torch.randn(128, generator=_gen(1), device=DEV)
    pos, slots = torch.arange(T, device=DEV).int(), torch.randperm(T + 88, generator=_gen(2), device=DEV)[:T].int()
    a, b = kv4.empty_cache(159, P, Hk, DEV), kv4.empty_cache(159, P, Hk, DEV)
    qa, qb = torch.empty_like(qkv[:, :H]), torch.empty_like(qkv[:, :H])
    args = lambda s: (r, pos[s], slots[s], qkv[s, :H])  # noqa: E731
    kv4.append(*args(slice(0, T)), qa, qkv[:, H:H + Hk], qkv[:, H + Hk:], a, P, q_weight=w, k_weight=w)
    for s in (slice(0, 1), slice(1, 70), slice(70, 1000), slice(1000, T)):
        kv4.append(*args(s), qb[s], qkv[s, H:H + Hk], qkv[s, H + Hk:], b, P, q_weight=w, k_weight=w)
    assert torch.equal(a, b) and torch.equal(qa, qb)


def test_append_in_place():
    r = step.rotary_setup(128)
    q, kv = _randn((9, 4, 128), "fp16", 1), _randn((9, 2, 128), "fp16", 2)
    pos, out, cache = torch.arange(9, device=DEV).int(), torch.empty_like(q), kv4.empty_cache(2, 8, 2, DEV)
    kv4.append(r, pos, pos, q, out, kv, kv, cache, 8)
    kv4.append(r, pos, pos, q, q, kv, kv, cache, 8)
    assert torch.equal(q, out)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page,heads", [(1, 1), (4, 3), (16, 8), (64, 2), (128, 5)])
def test_read(dtype, page, heads):
    pages = 3
    cache, _ = _strided_cache(pages, page, heads)
    cache.copy_(torch.randint(0, 256, cache.shape, generator=_gen(page), device=DEV).to(torch.uint8))
    raw = cache.cpu().numpy()
    for p in range(pages):  # words with a finite s
        for h in range(heads):
            for s in range(page):
                for at in oracle_kv4.places(page, s)[2:]:
                    raw[p, h, at + 1] = min(raw[p, h, at + 1], 0x6B)
    cache.copy_(torch.from_numpy(raw))
    slots = [0, pages * page - 1, -1, pages * page, 2**31 - 1, -2**31] + [s % (pages * page) for s in range(3, 40)]
    buf = torch.full((len(slots), heads + 1, 136), 7.0, dtype=DT[dtype], device=DEV)
    k_out, v_out = buf[:, :heads, :128], torch.empty((len(slots), heads, 128), dtype=DT[dtype], device=DEV)
    kv4.read(_i32(slots), cache, page, k_out, v_out)
    kv4.read(_i32(slots), cache, page, None, v_out)
    for i, s in enumerate(slots):
        for h in range(heads):
            k, v = oracle_kv4.get(raw, page, s, h) if 0 <= s < pages * page else (np.zeros(128), np.zeros(128))
            assert torch.equal(k_out[i, h].cpu(), torch.from_numpy(k).to(DT[dtype]))
            assert torch.equal(v_out[i, h].cpu(), torch.from_numpy(v).to(DT[dtype]))
    assert (buf[:, heads] == 7).all() and (buf[..., 128:] == 7).all()


# --------------------------------------------------------------- attention

def _config(**kw):
    return fi.default_plan_config(0, kv_bits=4, max_items=1 << 15, max_merge_units=1 << 13, max_partial_rows=1 << 17, **kw)


class Batch:
    """Requests over a 4-bit cache of normal values, every slot that holds no key filled with 0xFF."""

    def __init__(self, seed, qo, kv, hq, hkv, page, dtype, causal=0, v_std=1.0, scale=128.0**-0.5, strided=False):
        rng = np.random.default_rng(seed)
        pages = [-(-n // page) for n in kv]
        self.qo = np.concatenate([[0], np.cumsum(qo)]).astype(np.int32)
        self.kvp = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.last = np.array([n - (p - 1) * page if p else 1 for n, p in zip(kv, pages)], np.int32)
        pool = int(self.kvp[-1]) + 3
        self.ids = rng.permutation(pool)[:int(self.kvp[-1])].astype(np.int32)
        self.hq, self.hkv, self.page, self.causal, self.pool, self.scale = hq, hkv, page, causal, pool, scale
        self.q = _randn((int(self.qo[-1]) + 2, hq, 128), dtype, seed)
        if strided:
            self.cache, _ = _strided_cache(pool, page, hkv, 0xFF)
        else:
            self.cache = torch.full((pool, hkv, kv4.page_bytes(page)), 0xFF, dtype=torch.uint8, device=DEV)
        slots = [int(self.ids[self.kvp[b] + j // page]) * page + j % page for b, n in enumerate(kv) for j in range(n)]
        if slots:
            k, v = _randn((len(slots), hkv, 128), dtype, seed + 1), _randn((len(slots), hkv, 128), dtype, seed + 2, v_std)
            kv4.append(None, None, _i32(slots), None, None, k, v, self.cache, page)

    def plan(self, ws, stream=None):
        return fi.plan(ws, self.qo, self.kvp, self.ids, self.last, self.hq, self.hkv, 128, self.page, self.causal,
                       self.pool, stream=stream)

    def run(self, cfg, stream=None, ws=None, lse=True):
        ws = ws or fi.Workspace(cfg, device=DEV)
        info = self.plan(ws, stream)
        o = torch.full_like(self.q, float("nan"))
        l = torch.full(self.q.shape[:2], float("nan"), device=DEV) if lse else None
        self.idx = _i32(self.ids if self.ids.size else [0])
        kv4.run(ws, info, self.q, self.cache, self.idx, o, l, self.scale, stream=stream)
        return o, l, info, ws

    def check(self, o, lse, window=-1, sink=0, ids=None):
        n = int(self.qo[-1])
        k, v = oracle_kv4.all_values(self.cache.cpu().numpy(), self.page)
        k, v = np.nan_to_num(k, posinf=0, neginf=0), np.nan_to_num(v, posinf=0, neginf=0)
        ro, rl, size = oracle_kv4.attention(self.qo, self.kvp, self.ids if ids is None else ids, self.last, self.page,
                                            self.causal, self.scale, _f64(self.q), k, v, window, sink, self.pool)
        ro, rl, size = ro[:n], rl[:n], size[:n]
        og, lg = _f64(o[:n]), _f64(lse[:n])
        assert np.isfinite(og).all()
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lg), empty) and (og[empty] == 0).all()
        keys = max([0] + [int(self.kvp[b + 1] - self.kvp[b]) * self.page for b in range(len(self.qo) - 1)])
        half = torch.finfo(o.dtype).eps / 2
        top = np.abs(v[np.unique(self.ids[(self.ids >= 0) & (self.ids < self.pool)])]).max(initial=0)
        tol = (2.0**-11 + 1e-4) * size + keys * 2.0**-24 * min(top, 15 * 4096.0)
        tol = tol * (1 + half) + half * np.abs(ro) + torch.finfo(o.dtype).smallest_normal * 2 * half
        assert (np.abs(og - ro) <= tol).all(), float((np.abs(og - ro) - tol).max())
        assert np.abs(lg[~empty] - rl[~empty]).max(initial=0) <= 2e-4
        assert torch.isnan(o[n:]).all() and torch.isnan(lse[n:]).all()  # rows behind the last sequence


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hkv,group", [(2, 1), (1, 4), (2, 8), (1, 16), (2, 5), (1, 9)])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128])
def test_decode(dtype, hkv, group, page):
    kv = [1, 16, 17, 31, 32, 33, 127, 128, 129, 300, 0, 1001]
    b = Batch(10 + page + group, [1] * len(kv), kv, hkv * group, hkv, page, dtype, strided=page in (4, 64))
    o, lse, info, ws = b.run(_config())
    assert fi.device_status(ws) == 0
    b.check(o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page,group", [(16, 4), (1, 8), (128, 16)])
def test_split_decode(dtype, page, group):
    """Chunks of 64 keys: every request is merged from many partial states."""
    b = Batch(3, [1] * 5, [2000, 64, 65, 1, 777], 2 * group, 2, page, dtype)
    o, lse, info, ws = b.run(_config(decode_min_chunk=64, split_factor=8))
    assert info.num_merge_units > 0 and fi.device_status(ws) == 0
    b.check(o, lse)
    again = b.run(_config(decode_min_chunk=64, split_factor=8), ws=ws)
    n = int(b.qo[-1])
    assert torch.equal(again[0][:n], o[:n]) and torch.equal(again[1][:n], lse[:n])  # chunks merge in one order


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page,hkv,group", [(16, 2, 4), (8, 1, 8), (64, 1, 1), (1, 2, 2), (16, 1, 3), (128, 1, 16),
                                            (4, 1, 5), (32, 2, 1)])
@pytest.mark.parametrize("causal", [0, 1])
def test_prefill(dtype, page, hkv, group, causal):
    qo, kv = [1, 2, 33, 70, 130, 9], [5, 2, 300, 70, 257, 140]
    b = Batch(20 + page + group, qo, kv, hkv * group, hkv, page, dtype, causal)
    o, lse, info, ws = b.run(_config())
    assert fi.device_status(ws) == 0
    b.check(o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_split_prefill(dtype):
    """Chunks of 128 keys: late merge units."""
    b = Batch(7, [100, 1, 300], [1100, 700, 300], 8, 2, 16, dtype, 1)
    o, lse, info, ws = b.run(_config(prefill_min_chunk=128, decode_min_chunk=64, split_factor=16))
    assert info.num_late_merge_units > 0 and fi.device_status(ws) == 0
    b.check(o, lse)


def test_rows_without_keys():
    """More queries than keys under the causal mask, and requests without keys or without queries."""
    b = Batch(5, [40, 3, 1, 20, 0], [10, 0, 0, 1, 50], 8, 2, 16, "bf16", 1)
    o, lse, info, ws = b.run(_config())
    b.check(o, lse)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 0), (100, 4), (37, 300), (5000, 2), (2**31 - 1, 0)])
def test_window(window, sink, split):
    kw = dict(prefill_min_chunk=128, decode_min_chunk=64, split_factor=16) if split else {}
    b = Batch(8, [1, 3, 40, 1, 200], [1000, 257, 900, 64, 420], 8, 2, 16, "fp16", 1)
    o, lse, info, ws = b.run(_config(window_left=window, sink_tokens=sink, **kw))
    assert fi.device_status(ws) == 0
    b.check(o, lse, window, sink)


@pytest.mark.parametrize("qo", [1, 40])
def test_steep_logits_and_values(qo):
    """Running maxima that move in every stage, value scales from 2^-13 to 2^8, requests of tiny values alone."""
    b = Batch(9, [qo] * 4, [700] * 4, 8, 2, 16, "bf16", 1, scale=1.5)
    b.check(*b.run(_config())[:2])
    for std in (2.0**-12, 300.0):
        b = Batch(11, [qo] * 2, [300] * 2, 8, 2, 16, "fp16", 0, v_std=std)
        b.check(*b.run(_config())[:2])


@pytest.mark.parametrize("qo", [1, 40])
def test_queries_of_every_size(qo):
    """Rows of 2^-20 and 2^15 beside each other: each has its own power of two."""
    b = Batch(12, [qo], [300], 8, 2, 16, "bf16", 0, scale=2.0**-15)
    b.q *= torch.exp2(torch.linspace(-20, 15, 8, device=DEV))[None, :, None].to(b.q.dtype)
    o, lse, *_ = b.run(_config())
    b.check(o, lse)


@pytest.mark.parametrize("qo", [1, 40])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_page_ids_outside_the_cache(qo, page):
    b = Batch(13, [qo, qo], [333, 200], 8, 2, page, "bf16", 0)
    good = b.ids.copy()
    bad = good.copy()
    bad[3 % len(bad)], bad[len(bad) // 2], bad[-1] = -1, b.pool, 2**31 - 1
    ws = fi.Workspace(_config(), device=DEV)
    info = b.plan(ws)
    o, lse = torch.full_like(b.q, float("nan")), torch.full(b.q.shape[:2], float("nan"), device=DEV)
    kv4.run(ws, info, b.q, b.cache, _i32(bad), o, lse, b.scale)
    b.ids = good
    b.check(o, lse, ids=bad)


def test_captured_step_replays_later_plans():
    """Tables, append and attention as a serving loop has them, one graph for every step."""
    P, Hk, G, B, width = 8, 2, 4, 3, 40
    cfg = _config()
    ws = fi.Workspace(cfg, device=DEV)
    cache = kv4.empty_cache(B * width, P, Hk, DEV)
    tables = step.StepTables(B, B * width, B)
    r = step.rotary_setup(128, theta=1e6)
    w = 1 + 0.1 * torch.randn(128, generator=_gen(1), device=DEV)
    q, k, v = _randn((B, Hk * G, 128), "bf16", 1), _randn((B, Hk, 128), "bf16", 2), _randn((B, Hk, 128), "bf16", 3)
    q_rot, o = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty((B, Hk * G), device=DEV)
    free = torch.randperm(B * width, generator=_gen(4), device=DEV).int()
    block = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    head, qo_lens, kv_lens = _i32([0]), _i32([1] * B), _i32([0] * B)

    def calls():
        step.build_tables(tables, qo_lens, kv_lens, block, P, free, head)
        kv4.append(r, tables.positions, tables.slots, q, q_rot, k, v, cache, P, q_weight=w, k_weight=w)
        kv4.run(ws, info, q_rot, cache, tables.kv_indices, o, lse, 0.1)
        head.copy_(tables.counts[3:4])

    graph, keys, held = None, [0, 0, 0], [[], [], []]
    for it in range(25):
        g = _gen(100 + it)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        keys = [n + 1 for n in keys]
        kv_lens.copy_(_i32(keys))
        pages = [-(-n // P) for n in keys]
        info = fi.plan(ws, list(range(B + 1)), np.concatenate([[0], np.cumsum(pages)]), [],
                       [n - (p - 1) * P for n, p in zip(keys, pages)], Hk * G, Hk, 128, P, 0)
        if it == 3:
            torch.cuda.synchronize()
            saved = [t.clone() for t in (cache, block, head)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                calls()
            for t, s in zip((cache, block, head), saved):
                t.copy_(s)
        if graph:
            graph.replay()
        else:
            calls()
        assert fi.device_status(ws) == 0 and int(tables.counts[4]) == 0
        slots = tables.slots.cpu().numpy()
        raw = cache.cpu().numpy()
        for b in range(B):
            held[b].append([oracle_kv4.get(raw, P, int(slots[b]), h) for h in range(Hk)])
            kb = np.array([[x[h][0] for h in range(Hk)] for x in held[b]])
            vb = np.array([[x[h][1] for h in range(Hk)] for x in held[b]])
            ro, rl, size = oracle_kv4.attention([0, 1], [0, 1], [0], [len(kb)], len(kb), 0, 0.1, _f64(q_rot[b:b + 1]),
                                                kb[None], vb[None])
            assert (np.abs(_f64(o[b:b + 1]) - ro) <= (2.0**-11 + 1e-4) * size + 2.0**-8 * np.abs(ro) + 1e-5).all()
            assert np.abs(_f64(lse[b:b + 1]) - rl).max() <= 2e-4


@pytest.mark.parametrize("first", [0, 1])
def test_captured_run_serves_plans_of_the_other_class(first):
    """A run captured on a plan of single tokens serves one whose prompt parts are split, and the other way round."""
    bs = [Batch(50, [1] * 5, [300, 20, 700, 1, 64], 8, 2, 16, "bf16", 1),
          Batch(51, [60, 1, 150], [900, 300, 260], 8, 2, 16, "bf16", 1)]
    cfg = _config(prefill_min_chunk=128, decode_min_chunk=64, split_factor=4)
    ws = fi.Workspace(cfg, device=DEV)
    rows, pool = max(len(b.q) for b in bs), max(b.pool for b in bs)
    q = torch.zeros((rows, 8, 128), dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros((pool, 2, kv4.page_bytes(16)), dtype=torch.uint8, device=DEV)
    idx = torch.zeros(max(len(b.ids) for b in bs), dtype=torch.int32, device=DEV)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)

    def stage(b):
        q[:len(b.q)].copy_(b.q)
        cache[:b.pool].copy_(b.cache)
        idx[:len(b.ids)].copy_(_i32(b.ids))
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        return b.plan(ws)

    info = stage(bs[first])
    assert (info.num_late_merge_units > 0) == (first == 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv4.run(ws, info, q, cache, idx, o, lse, bs[0].scale)
    for turn in (first, 1 - first, first, 1 - first):
        b = bs[turn]
        stage(b)
        graph.replay()
        torch.cuda.synchronize()
        assert fi.device_status(ws) == 0
        b.check(o[:len(b.q)], lse[:len(b.q)])


@pytest.mark.parametrize("group", [3, 4, 16])
def test_strided_queries_and_outputs(group):
    """Rows of q and o with room between heads and tokens: the values of contiguous ones, and nothing else written."""
    b = Batch(60 + group, [1, 70, 5, 200], [400, 300, 5, 200], 2 * group, 2, 16, "bf16", 1)
    o, lse, info, ws = b.run(_config())
    n = int(b.qo[-1])
    wide = [torch.full((len(b.q), 2 * group + 1, 136), 3.0, dtype=b.q.dtype, device=DEV) for _ in range(2)]
    q, out = (x[:, 1:, :128] for x in wide)
    q.copy_(b.q)
    kv4.run(ws, info, q, b.cache, b.idx, out, None, b.scale)
    assert torch.equal(out[:n], o[:n]) and fi.device_status(ws) == 0
    assert (wide[1][n:] == 3).all() and (wide[1][:, 0] == 3).all() and (wide[1][..., 128:] == 3).all()


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams give what each gives alone."""
    bs = [Batch(30 + i, [1] * 6 + [60], [500, 3, 900, 77, 1500, 31, 400], 8, 2, 16, "bf16", 1) for i in range(2)]
    alone = [b.run(_config()) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    wss = [fi.Workspace(_config(), device=DEV) for _ in bs]
    torch.cuda.synchronize()
    got = [[] for _ in bs]
    for _ in range(5):
        for i, b in enumerate(bs):
            with torch.cuda.stream(streams[i]):
                got[i].append(b.run(None, ws=wss[i])[:2])
    torch.cuda.synchronize()
    for i, b in enumerate(bs):
        n = int(b.qo[-1])
        for o, l in got[i]:
            assert torch.equal(o[:n], alone[i][0][:n]) and torch.equal(l[:n], alone[i][1][:n])


def test_foreign_plans_write_nothing():
    b = Batch(14, [1, 1], [40, 50], 8, 2, 16, "bf16")
    cfg = _config()
    ws = fi.Workspace(cfg, device=DEV)
    info = b.plan(ws)
    o = torch.full_like(b.q, 5.0)
    other = fi.Workspace(cfg, device=DEV)  # no plan in it
    kv4.run(other, info, b.q, b.cache, _i32(b.ids), o, None, b.scale)
    assert fi.device_status(other) == 6 and (o == 5).all()
    fi.plan(other, b.qo, b.kvp, b.ids, b.last, 4, 2, 128, 16, 0, b.pool)  # of other heads
    kv4.run(other, info, b.q, b.cache, _i32(b.ids), o, None, b.scale)
    assert fi.device_status(other) == 6 and (o == 5).all()


def test_large_offsets():
    """A cache of over 4 GB whose last pages a request uses."""
    P, Hk, pages = 128, 8, 34000
    cache = torch.empty((pages, Hk, kv4.page_bytes(P)), dtype=torch.uint8, device=DEV)
    assert cache.numel() > 1 << 32
    ids = [pages - 1, pages - 2, 0, pages // 2, 32767]
    slots = [i * P + s for i in ids for s in range(P)][:600]
    k, v = _randn((600, Hk, 128), "bf16", 1), _randn((600, Hk, 128), "bf16", 2)
    kv4.append(None, None, _i32(slots), None, None, k, v, cache, P)
    k_out, v_out = torch.empty_like(k), torch.empty_like(v)
    kv4.read(_i32(slots), cache, P, k_out, v_out)
    small = cache[ids].contiguous()
    moved = [i * P + s for i in range(5) for s in range(P)][:600]
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    kv4.read(_i32(moved), small, P, k2, v2)
    assert torch.equal(k_out, k2) and torch.equal(v_out, v2) and (k_out - k).abs().max() < 0.5
    q = _randn((1, 32, 128), "bf16", 3)
    ws = fi.Workspace(_config(), device=DEV)
    info = fi.plan(ws, [0, 1], [0, 5], ids, [600 - 4 * P], 32, Hk, 128, P, 0, pages)
    o, o2, lse, lse2 = torch.empty_like(q), torch.empty_like(q), *torch.empty((2, 1, 32), device=DEV)
    kv4.run(ws, info, q, cache, _i32(ids), o, lse, 0.1)
    kv4.run(ws, info, q, small, _i32(range(5)), o2, lse2, 0.1)
    assert fi.device_status(ws) == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
