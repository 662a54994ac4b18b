"""Differential attention in numpy fp64 (the oracle of include/fi_diff.h).

Per query row of head h with halves q = [q1 | q2], k = [k1 | k2] (64 dims
each) and values of 128 dims: S_i = softmax(scale q_i k_i^T) V over the
visible keys, y = S_1 - lambda_h S_2, then out_scale * y or, with a norm
weight w, out_scale * y / sqrt(mean(y^2) + eps) * w.  Query token t of a
request with Lq queries and Lkv keys sits at Lkv - Lq + t; causal rows see
keys at or before it; with a window W, keys at or after it minus W, and keys
before `sink`.  A row without a visible key gives o = 0 and lse = -inf.

slack() bounds the error of a kernel from its roundings alone.
"""
from __future__ import annotations

import numpy as np


def attention(qo_indptr, kv_indptr, kv_indices, last_page_len, page_size, causal, scale, q, k, v, lam, w=None,
              eps=1e-5, out_scale=1.0, window=-1, sink=0, mag=False):
    """q [tokens, Hq, 128], k, v [pages, P, Hkv, 128], lam [Hq], all fp64:
    (o [tokens, Hq, 128], lse [tokens, Hq, 2]); with mag also
    sum_i |c_i| softmax_i |V| of each row before norm and scale (c = 1, lambda)."""
    T, Hq, _ = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    y = np.zeros((T, Hq, 128))
    size = np.zeros((T, Hq, 128))
    lse = np.full((T, Hq, 2), -np.inf)
    for b in range(len(qo_indptr) - 1):
        ids = np.asarray(kv_indices[kv_indptr[b]:kv_indptr[b + 1]], dtype=np.int64)
        n = (len(ids) - 1) * page_size + int(last_page_len[b]) if len(ids) else 0
        kb = k[ids].reshape(-1, Hkv, 128)[:n]
        vb = v[ids].reshape(-1, Hkv, 128)[:n]
        lq = int(qo_indptr[b + 1] - qo_indptr[b])
        key = np.arange(n)
        for t in range(lq):
            pos = n - lq + t
            see = key <= pos if causal else np.ones(n, bool)
            if window >= 0:
                see = see & ((key >= pos - window) | (key < sink))
            if not see.any():
                continue
            row = int(qo_indptr[b]) + t
            for h in range(Hq):
                kh, vh = kb[see, h // G], vb[see, h // G]
                for i, c in ((0, 1.0), (1, -lam[h])):
                    s = scale * (kh[:, 64 * i:64 * i + 64] @ q[row, h, 64 * i:64 * i + 64])
                    m = s.max()
                    e = np.exp(s - m)
                    p = e / e.sum()
                    lse[row, h, i] = m + np.log(e.sum())
                    y[row, h] += c * (p @ vh)
                    size[row, h] += abs(c) * (p @ np.abs(vh))
    o = y.copy()
    if w is not None:
        o = o / np.sqrt((o * o).mean(-1, keepdims=True) + eps) * w
    o = o * out_scale
    return (o, lse, y, size) if mag else (o, lse)


def slack(o, y, size, weight_eps, out_eps, w=None, eps=1e-5, out_scale=1.0):
    """Element-wise bound on |kernel - o|.  weight_eps: relative error of a
    softmax weight (so |dy| <= weight_eps * size); the norm turns dy into at
    most f |w| (|dy| + |y| rms(dy) / r), with r its root and f = out_scale / r;
    out_eps: half a step of the output type."""
    dy = weight_eps * size
    if w is None:
        err = abs(out_scale) * dy
    else:
        r = np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        err = abs(out_scale) * np.abs(w) / r * (dy + np.abs(y) * np.sqrt((dy * dy).mean(-1, keepdims=True)) / r)
    return err * (1 + out_eps) + out_eps * np.abs(o)
