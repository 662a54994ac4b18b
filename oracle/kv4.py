"""The 4-bit cache in numpy (the oracle of include/fi_kv4.h): its quantiser in
single fp32 operations, to the bit, its layout byte by byte, and attention over
the values it holds in fp64."""
from __future__ import annotations

import math

import numpy as np

D, BLOCK = 128, 32
F = np.float32


def quantise(x):
    """Codes [.., 128] and words [..] of fp32 rows x [.., 128]."""
    x = np.asarray(x, F)
    with np.errstate(all="ignore"):
        lo = np.minimum(np.fmin.reduce(x, -1, initial=F(0)), F(0)).astype(F)
        hi = np.maximum(np.fmax.reduce(x, -1, initial=F(0)), F(0)).astype(F)
        near = ((hi - lo) * F(1 / 15)).astype(np.float16)
        bits = np.minimum((near.view(np.uint16).astype(np.int64) + 15) // 16 * 16, 0x6C00)
        s = bits.astype(np.uint16).view(np.float16).astype(F)
        inv = np.where(s > 0, F(1) / np.where(s > 0, s, F(1)), F(0)).astype(F)
        z = np.clip(np.rint(-lo * inv), 0, 15)
        t = np.rint((x * inv[..., None]).astype(F))
        n = np.clip(np.where(np.isnan(t), -15, t) + z[..., None], 0, 15)
    return n.astype(np.uint8), (bits + z.astype(np.int64)).astype(np.uint16)


def values(codes, words):
    """What codes and words stand for, fp64."""
    w = np.asarray(words, np.uint16)
    s = (w & 0xFFF0).astype(np.uint16).view(np.float16).astype(np.float64)
    return (np.asarray(codes, np.float64) - (w & 15)[..., None]) * s[..., None]


def page_bytes(page_size):
    b = min(page_size, BLOCK)
    return page_size // b * (-(-132 * b // 16) * 16)


def places(page_size, slot):
    """Byte offsets in a page of slot's k row, v row, k word, v word."""
    b = min(page_size, BLOCK)
    base = slot // b * (-(-132 * b // 16) * 16)
    i = slot % b
    return base + 64 * i, base + 64 * (b + i), base + 128 * b + 2 * i, base + 130 * b + 2 * i


def put(cache, page_size, slot, head, k_row, v_row):
    """Quantise fp32 rows k_row, v_row into cache (uint8 [pages, heads, bytes]) at a slot of the pool."""
    page = cache[slot // page_size, head]
    at = places(page_size, slot % page_size)
    for row, r, w in ((k_row, at[0], at[2]), (v_row, at[1], at[3])):
        n, word = quantise(row)
        page[r:r + 64] = n[0::2] + 16 * n[1::2]
        page[w], page[w + 1] = int(word) % 256, int(word) // 256


def get(cache, page_size, slot, head):
    """fp64 (k, v) rows held at a slot of the pool."""
    page = cache[slot // page_size, head]
    at = places(page_size, slot % page_size)
    out = []
    for r, w in ((at[0], at[2]), (at[1], at[3])):
        n = np.empty(D, np.uint8)
        n[0::2], n[1::2] = page[r:r + 64] % 16, page[r:r + 64] // 16
        out.append(values(n, np.uint16(int(page[w]) + 256 * int(page[w + 1]))))
    return out


def all_values(cache, page_size):
    """fp64 k and v [pages, page_size, heads, 128] of a whole cache."""
    pages, heads, _ = cache.shape
    out = []
    b = min(page_size, BLOCK)
    blocks = cache.reshape(pages, heads, page_size // b, -1)
    for which in (0, 1):
        rows = blocks[..., 64 * b * which:64 * b * (which + 1)].reshape(pages, heads, page_size, 64)
        at = 128 * b + 2 * b * which
        words = np.ascontiguousarray(blocks[..., at:at + 2 * b]).view("<u2").reshape(pages, heads, page_size)
        n = np.stack([rows % 16, rows // 16], -1).reshape(pages, heads, page_size, D)
        with np.errstate(all="ignore"):
            out.append(values(n, words).transpose(0, 2, 1, 3))
    return out


def norm_exact_order(x, w, eps):
    """The append's norm in fp32, its sum in its order."""
    x = np.asarray(x, F)
    y = (x * x).astype(F)
    y = (y[..., :64] + y[..., 64:]).reshape(*x.shape[:-1], 8, 8)
    for d in (4, 2, 1):
        y = y[..., :d] + y[..., d:]
    y = y[..., 0]
    for d in (4, 2, 1):
        y = y[..., :d] + y[..., d:]
    f = F(1) / np.sqrt(y * F(1 / 128) + F(eps))
    return ((x * f).astype(F) * np.asarray(w, F)).astype(F)


def attention(qo_indptr, kv_indptr, kv_indices, last_page_len, page_size, causal, scale, q, k, v, window=-1, sink=0,
              num_pages=None):
    """o [tokens, Hq, 128], lse [tokens, Hq] and sum_j p_j |v_j|, fp64; k, v [pages, P, Hkv, 128] as all_values gives
    them.  Page ids outside [0, num_pages) read as zeros."""
    T, Hq, _ = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    o, size = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    num_pages = k.shape[0] if num_pages is None else num_pages
    for b in range(len(qo_indptr) - 1):
        ids = np.asarray(kv_indices[kv_indptr[b]:kv_indptr[b + 1]], np.int64)
        n = (len(ids) - 1) * page_size + int(last_page_len[b]) if len(ids) else 0
        good = (ids >= 0) & (ids < num_pages)
        there = np.repeat(good, page_size)[:n, None, None]
        safe = np.where(good, ids, 0)
        kb, vb = (np.where(there, x[safe].reshape(-1, Hkv, D)[:n], 0) for x in (k, v))
        lq = int(qo_indptr[b + 1] - qo_indptr[b])
        if lq == 0 or n == 0:
            continue
        pos = np.arange(lq)[:, None] + (n - lq)
        key = np.arange(n)[None]
        see = key <= pos if causal else key < n + 0 * pos
        if window >= 0:
            see = see & ((key >= pos - window) | (key < sink))
        rows = slice(int(qo_indptr[b]), int(qo_indptr[b + 1]))
        used = see.any(0)
        for h in range(Hkv):
            kh, vh = kb[:, h][used], vb[:, h][used]
            m = see[:, used]
            for a in range(h * G, h * G + G):
                s = np.where(m, scale * (q[rows, a] @ kh.T), -np.inf)
                top = s.max(-1, initial=-np.inf)
                e = np.exp(s - np.where(np.isinf(top), 0, top)[:, None])
                l = e.sum(-1)
                ok = l > 0
                p = np.where(ok[:, None], e / np.where(ok, l, 1)[:, None], 0)
                o[rows, a], size[rows, a] = p @ vh, p @ np.abs(vh)
                lse[rows, a] = np.where(ok, top + np.log(np.where(ok, l, 1)), -np.inf)
    return o, lse, size


def row_faults(word, got, ref, size):
    """What is wrong with a held row (values got [128], its word) of the fp64 row ref, which the quantiser met to within
    `size`: names of the parts, none if it is as defined.

    s is the range / 15 to fp16 (2^-11) and up by at most 15 of 1024 steps.  z is -lo / s rounded, behind two fp32 roundings
    of up to 15 2^-24 each (below 2e-6).  A code is at most half a step off, or, kept within 0 .. 15 at the ends of the range
    (15 s (1 + 2^-11) at most), 15 2^-11 < 2^-7 more."""
    s, z = float(np.uint16(word & 0xFFF0).view(np.float16)), word & 15
    lo, hi = min(ref.min(), 0.0), max(ref.max(), 0.0)
    exact = (hi - lo) / 15
    bad = []
    if not exact * (1 - 2.0**-11) - size <= s <= exact * (1 + 2.0**-11 + 15 / 1024) + size:
        bad.append("scale")
    if abs(z - min(-lo / s, 15)) > 0.5 + size / s + 2e-6:
        bad.append("zero point")
    if (np.abs(got - ref) > s * (0.5 + 2.0**-7) + 3 * size).any():
        bad.append("values")
    return bad
