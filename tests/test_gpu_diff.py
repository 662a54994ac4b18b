"""Differential attention on the GPU against the fp64 oracle.

Tolerances come from roundings alone (oracle.diff.slack).  A logit is 64
products summed in fp32: with |q|, |k| <= 5 and scale 1/8 its error is below
64 * 2^-24 * 64 * 25 / 8 = 7.6e-4 in the worst order and some 1e-5 in earnest;
exponent, weights and sums add less than 1e-5.  WEIGHT covers these with 1e-4.
On the tensor cores w_1 - lambda w_2 is rounded to the input type, by at most
eps / 2 (eps is allowed); a split unit's chunk has weights of two terms."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import serving_attention_gb300 as fi
import workloads
from oracle import diff as oracle_diff
from serving_attention_gb300 import differential

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
WEIGHT = 1e-4
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _config(**kw):
    return fi.default_plan_config(0, differential=1, max_items=1 << 15, max_merge_units=1 << 13,
                                  max_partial_rows=1 << 17, **kw)


def _batch(seed, qo, kv, hq, hkv, page, dtype, causal=0, poison=True):
    b = workloads.make_batch("diff", dtype, qo, kv, hq, hkv, page, causal, seed, DEV)
    if poison:  # slots past the end of a request: anything, NaN included
        for i in range(len(kv)):
            if kv[i] % page:
                last = int(b.kv_indices[b.kv_indptr[i + 1] - 1])
                b.k[last, kv[i] % page:] = float("nan")
                b.v[last, kv[i] % page:] = float("nan")
    g = torch.Generator(device=DEV).manual_seed(seed)
    lam = 1.2 * torch.rand(hq, generator=g, device=DEV) - 0.2
    w = 1 + 0.2 * torch.randn(128, generator=g, device=DEV)
    return b, lam, w


def _run(b, lam, w, cfg, out_scale=1.0, stream=None, ws=None, lse=True, eps=1e-5):
    ws = ws or fi.Workspace(cfg, device=DEV)
    info = fi.plan(ws, b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, b.num_qo_heads, b.num_kv_heads, 128,
                   b.page_size, b.causal, b.num_pages, stream=stream)
    kvi = torch.as_tensor(b.kv_indices if b.kv_indices.size else np.zeros(1, np.int32), device=DEV)
    o = torch.full_like(b.q, float("nan"))
    l = torch.full((*b.q.shape[:2], 2), float("nan"), device=DEV) if lse else None
    differential.run(ws, info, b.q, b.k, b.v, kvi, lam, o, l, b.sm_scale, norm_weight=w, norm_eps=eps,
                     out_scale=out_scale, stream=stream)
    return o, l, info, ws, kvi


def _check(b, lam, w, o, lse, out_scale=1.0, window=-1, sink=0, rounded=False):
    f = lambda t: np.nan_to_num(t.double().cpu().numpy(), nan=0.0)  # noqa: E731
    wd = None if w is None else w.double().cpu().numpy()
    ro, rl, y, size = oracle_diff.attention(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, b.page_size,
                                            b.causal, b.sm_scale, f(b.q), f(b.k), f(b.v), f(lam), wd, 1e-5, out_scale,
                                            window, sink, mag=True)
    n = b.total_qo
    half = torch.finfo(o.dtype).eps / 2
    tol = oracle_diff.slack(ro, y, size, WEIGHT + (2 * half if rounded else 0), half, wd, 1e-5, out_scale)
    og, lg = o[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
    ro, rl, tol = ro[:n], rl[:n], tol[:n]
    assert np.isfinite(og).all()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lg), empty)
    assert (og[empty.all(-1)] == 0).all()
    assert (np.abs(og - ro) <= tol + 1e-7).all(), float((np.abs(og - ro) - tol).max())
    assert np.abs(lg[~empty] - rl[~empty]).max(initial=0) <= 1e-3
    # rows behind the last sequence stay as they were
    assert torch.isnan(o[n:]).all() and torch.isnan(lse[n:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hkv,group", [(2, 1), (1, 4), (2, 8), (1, 16), (2, 5)])
@pytest.mark.parametrize("page", [1, 4, 16, 128])
def test_decode(dtype, hkv, group, page):
    kv = [1, 16, 17, 127, 128, 129, 300, 0, 1001]
    b, lam, w = _batch(10 + page + group, [1] * len(kv), kv, hkv * group, hkv, page, dtype)
    cfg = _config()
    o, lse, info, ws, _ = _run(b, lam, w if group != 4 else None, cfg, 0.3)
    assert fi.device_status(ws) == 0
    _check(b, lam, w if group != 4 else None, o, lse, 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_split_decode(dtype):
    """Chunks of 64 keys: every request is merged from many partial states."""
    kv = [2000, 64, 65, 1, 777]
    b, lam, w = _batch(3, [1] * 5, kv, 8, 2, 16, dtype)
    o, lse, info, ws, _ = _run(b, lam, w, _config(decode_min_chunk=64, split_factor=8))
    assert info.num_merge_units > 0 and fi.device_status(ws) == 0
    _check(b, lam, w, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page,hkv,group", [(16, 2, 4), (8, 1, 8), (64, 1, 1), (1, 2, 2), (16, 1, 3), (128, 1, 16)])
@pytest.mark.parametrize("causal", [0, 1])
def test_prefill(dtype, page, hkv, group, causal):
    qo, kv = [1, 2, 33, 70, 130, 9], [5, 2, 300, 70, 257, 140]
    b, lam, w = _batch(20 + page + group, qo, kv, hkv * group, hkv, page, dtype, causal)
    o, lse, info, ws, _ = _run(b, lam, w, _config(), 0.5)
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, 0.5, rounded=True)


def test_rows_without_keys():
    """More queries than keys under the causal mask, and requests without keys."""
    b, lam, w = _batch(5, [40, 3, 1, 20], [10, 0, 0, 1], 8, 2, 16, "bf16", causal=1)
    o, lse, info, ws, _ = _run(b, lam, w, _config())
    _check(b, lam, w, o, lse, rounded=True)


def test_rows_without_keys_and_no_eps():
    """The norm of a zero row with eps 0 is zero, not 0 / 0."""
    b, lam, w = _batch(5, [40, 3, 1, 20], [10, 0, 0, 1], 8, 2, 16, "bf16", causal=1)
    o, lse, *_ = _run(b, lam, w, _config(), eps=0.0)
    empty = torch.isneginf(lse[:b.total_qo]).all(-1)
    assert empty.any() and (o[:b.total_qo][empty] == 0).all() and torch.isfinite(o[:b.total_qo]).all()


@pytest.mark.parametrize("lam_value", [0.0, 1.0, -1.5, 40.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_lambdas(lam_value, dtype):
    b, lam, w = _batch(6, [1, 70, 130], [500, 300, 2000], 8, 2, 16, dtype, causal=1)
    lam = torch.full_like(lam, lam_value)
    for kw in ({}, dict(prefill_min_chunk=128, decode_min_chunk=64, split_factor=16)):
        o, lse, info, ws, _ = _run(b, lam, None, _config(**kw), 0.5)
        assert fi.device_status(ws) == 0
        _check(b, lam, None, o, lse, 0.5, rounded=True)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 0), (100, 4), (37, 300), (5000, 2)])
def test_window_and_sink(window, sink, split):
    kw = dict(decode_min_chunk=64, prefill_min_chunk=128, split_factor=16) if split else {}
    b, lam, w = _batch(7, [1, 60, 200, 3], [700, 400, 900, 150], 8, 2, 16, "bf16", causal=1)
    o, lse, info, ws, _ = _run(b, lam, w, _config(window_left=window, sink_tokens=sink, **kw))
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, window=window, sink=sink, rounded=True)


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 20, 3])
def test_widest_windows_of_queries_before_the_keys(window, page):
    """More queries than keys without the causal mask: the first ones lie before key 0, and
    their distance to the window's lowest key passes an int."""
    b, lam, w = _batch(23, [40, 3, 2], [10, 1, 100], 8, 2, page, "bf16")
    o, lse, info, ws, _ = _run(b, lam, w, _config(window_left=window))
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, window=window, rounded=True)


@pytest.mark.parametrize("page", [4, 16])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("window,sink", [(2**31 - 1, 0), (2**31 - 1, 4), (2**31 - 100, 300), (2**30, 2**31 - 1)])
def test_widest_windows_over_several_tiles(window, sink, causal, page):
    """The window's lowest key lies so far before a tile that their distance passes an int."""
    b, lam, w = _batch(25, [40, 1, 130], [300, 255, 129], 8, 2, page, "fp16", causal)
    o, lse, info, ws, _ = _run(b, lam, w, _config(window_left=window, sink_tokens=sink))
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, window=window, sink=sink, rounded=True)


@pytest.mark.parametrize("page", [4, 16, 128])
@pytest.mark.parametrize("window,sink", [(100, 1), (255, 128), (300, 130), (640, 300)])
def test_sinks_before_a_window(window, sink, page):
    """A sink's tiles in the item of its window (pages of 8 and more), up to sinks of several tiles."""
    b, lam, w = _batch(16, [40, 200, 9], [1500, 900, 450], 8, 2, page, "bf16", causal=1)
    o, lse, info, ws, _ = _run(b, lam, w, _config(window_left=window, sink_tokens=sink, num_ctas=4))
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, window=window, sink=sink, rounded=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_split_prefill(dtype):
    b, lam, w = _batch(8, [50, 129, 1], [1500, 700, 900], 8, 2, 16, dtype, causal=1)
    o, lse, info, ws, _ = _run(b, lam, w, _config(prefill_min_chunk=128, decode_min_chunk=64, split_factor=16))
    assert info.num_merge_units > 2 and fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, rounded=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [4, 16])
def test_a_chunk_that_one_map_leaves(page, dtype):
    """Map 1 looks at the first chunk, map 2 at the fourth; in the first, map 2's
    largest weight is that of a key with large values, which counts for nothing
    in the whole (e^-30).  A chunk's weights are two terms, 2^-16 of a weight at
    most, which WEIGHT covers: no rounding of one term."""
    b, lam, w = _batch(22, [40, 1], [700, 640], 8, 2, page, dtype, causal=1, poison=False)
    b.q.zero_()
    b.k.zero_()
    b.v.mul_(0.01)
    b.q[..., 0] = 8
    b.q[..., 64] = 8
    b.sm_scale = 0.125  # a logit is the key's one dim
    for i in range(2):
        ids = torch.as_tensor(b.kv_indices[b.kv_indptr[i]:b.kv_indptr[i + 1]], device=DEV).long()
        at = lambda key: (ids[key // page], key % page)  # noqa: E731
        for key in range(128):
            b.k[at(key)][:, 0] = 20
            b.k[at(384 + key)][:, 64] = 40
        b.k[at(5)][:, 0] = -20
        b.k[at(5)][:, 64] = 10
        b.v[at(5)] *= 8000
    o, lse, info, ws, _ = _run(b, lam, None, _config(prefill_min_chunk=128, decode_min_chunk=64, split_factor=16))
    assert info.num_merge_units > 2 and fi.device_status(ws) == 0
    _check(b, lam, None, o, lse)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["up", "down", "spike"])
def test_steep_logits(order, dtype, split):
    """Logits that leave the first tile's far behind, in opposite orders in the
    two maps.  Queries and keys have one dim each map, of few bits, so a logit
    is exact; its factor log2(e) in fp32 is off by 2^-25, at most 1e-5 over 250."""
    b, lam, w = _batch(17, [1, 40, 140], [900, 600, 1000], 8, 2, 16, dtype, causal=1, poison=False)
    n = 1000
    ramp = (torch.arange(n, device=DEV) // 4).float()
    if order == "down":
        ramp = 249 - ramp
    if order == "spike":
        ramp = torch.where(torch.arange(n, device=DEV) % 331 == 330, 200.0, 0.0)
    b.q.zero_()
    b.k.zero_()
    b.q[..., 0] = 8
    b.q[..., 64] = 8
    for i in range(3):
        ids = torch.as_tensor(b.kv_indices[b.kv_indptr[i]:b.kv_indptr[i + 1]], device=DEV).long()
        for p in range(len(ids)):
            part = ramp[16 * p:16 * p + 16]
            for h in range(2):
                b.k[ids[p], :len(part), h, 0] = part.to(b.k.dtype)
                b.k[ids[p], :len(part), h, 64] = (250 - part).to(b.k.dtype)
    b.sm_scale = 0.125
    kw = dict(prefill_min_chunk=128, decode_min_chunk=64, split_factor=16) if split else {}
    o, lse, info, ws, _ = _run(b, lam, w, _config(**kw))
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, rounded=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ctas,kw", [(1, {}), (3, {}), (2, dict(prefill_min_chunk=128, split_factor=64)),
                                     (3, dict(window_left=300, sink_tokens=4)), (5, dict(split_factor=4))])
def test_few_ctas(ctas, kw, dtype):
    """Many items a CTA: whole and split ones, ends of requests, empty requests, decode items behind them."""
    b, lam, w = _batch(18, [130, 1, 33, 70, 1, 200, 20], [700, 600, 33, 301, 0, 520, 0], 8, 2, 16, dtype, causal=1)
    o, lse, info, ws, _ = _run(b, lam, w, _config(num_ctas=ctas, **kw))
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, window=kw.get("window_left", -1), sink=kw.get("sink_tokens", 0), rounded=True)


@pytest.mark.parametrize("page", [4, 8, 64])
@pytest.mark.parametrize("ctas", [1, 3])
def test_runs_of_short_prompts(ctas, page):
    """Many items of one tile in a row, where nothing but their own barriers holds the K and V loaders together."""
    kv = [int(x) for x in np.random.default_rng(ctas + page).integers(9, 129, size=40)]
    b, lam, w = _batch(21, kv, kv, 4, 1, page, "bf16", causal=1)
    o, lse, info, ws, _ = _run(b, lam, w, _config(num_ctas=ctas))
    assert info.num_items >= 40 and fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, rounded=True)


@pytest.mark.parametrize("page", [1, 2, 4])
@pytest.mark.parametrize("ctas,kw", [(2, {}), (3, dict(prefill_min_chunk=128, split_factor=64)),
                                     (2, dict(window_left=200, sink_tokens=5))])
def test_prefill_on_small_pages(ctas, kw, page):
    """Tiles copied row by row: many items a CTA, split ones, a sink's tile, decode items behind them."""
    b, lam, w = _batch(19, [130, 1, 33, 70, 1, 200, 20], [700, 600, 33, 301, 0, 520, 7], 8, 2, page, "fp16", causal=1)
    o, lse, info, ws, _ = _run(b, lam, w, _config(num_ctas=ctas, **kw))
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, window=kw.get("window_left", -1), sink=kw.get("sink_tokens", 0), rounded=True)


@pytest.mark.parametrize("page", [1, 4])
@pytest.mark.parametrize("ctas", [1, 4])
def test_few_rows_beside_prompts_on_small_pages(ctas, page):
    """Requests of 17 to 32 packed rows, the longest of all, in a CTA with prompts and decodes."""
    b, lam, w = _batch(24, [8, 100, 1, 5, 130, 7], [1500, 300, 900, 1100, 200, 700], 8, 2, page, "bf16", causal=1)
    o, lse, info, ws, _ = _run(b, lam, w, _config(num_ctas=ctas))
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, rounded=True)


def test_strides_and_padding_rows():
    """q and o inside wider rows, caches with a padding head, more buffer rows
    than the plan's, no lse."""
    b, lam, w = _batch(9, [1, 20, 1], [200, 90, 33], 8, 2, 16, "bf16", causal=1)
    n = b.total_qo
    wide = torch.full((n + 5, 10, 256), float("nan"), dtype=b.q.dtype, device=DEV)
    q = wide[:, 1:9, 64:192]
    q[:n] = b.q[:n]
    kc = torch.full((b.num_pages, 16, 3, 128), float("nan"), dtype=b.q.dtype, device=DEV)
    vc = torch.full((b.num_pages, 2, 16, 128), float("nan"), dtype=b.q.dtype, device=DEV).transpose(1, 2)
    kc[:, :, 1:] = b.k
    vc[:] = b.v
    ow = torch.full((n + 5, 9, 160), float("nan"), dtype=b.q.dtype, device=DEV)
    o = ow[:, 1:, 16:144]
    ref, _, info, ws, kvi = _run(b, lam, w, _config())
    differential.run(ws, info, q, kc[:, :, 1:], vc, kvi, lam, o, None, b.sm_scale, norm_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(o[:n], ref[:n])
    ow[:n, 1:, 16:144] = float("nan")
    assert torch.isnan(ow).all()


def test_graph_replays_other_plans_and_streams():
    """One captured graph serves plans of other lengths; a side stream gives the same bits."""
    cfg = _config()
    b, lam, w = _batch(11, [1] * 6, [900, 5, 130, 64, 2000, 1], 8, 2, 16, "bf16")
    c, _, _ = _batch(12, [1] * 6, [3, 800, 1, 128, 40, 1500], 8, 2, 16, "bf16")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o1, l1, info, ws, kvi = _run(b, lam, w, cfg, stream=side)
    side.synchronize()
    _check(b, lam, w, o1, l1)
    n = max(b.kv_indices.size, c.kv_indices.size)
    table = torch.zeros(n, dtype=torch.int32, device=DEV)
    q = torch.empty_like(b.q)
    pages = max(b.num_pages, c.num_pages)
    k, v = (torch.zeros((pages, 16, 2, 128), dtype=b.q.dtype, device=DEV) for _ in range(2))
    o, lse = torch.empty_like(b.q), torch.empty_like(l1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        differential.run(ws, info, q, k, v, table, lam, o, lse, b.sm_scale, norm_weight=w)
    for x in (b, c, b):
        fi.plan(ws, x.qo_indptr, x.kv_indptr, x.kv_indices, x.last_page_len, 8, 2, 128, 16, 0, x.num_pages)
        table[:x.kv_indices.size] = torch.as_tensor(x.kv_indices, device=DEV)
        q.copy_(x.q)
        k[:x.num_pages] = x.k
        v[:x.num_pages] = x.v
        g.replay()
        torch.cuda.synchronize()
        assert fi.device_status(ws) == 0
        _check(x, lam, w, o, lse)


def test_plans_without_rows_write_nothing():
    """No requests, and requests without queries, in buffers of a padded size."""
    b, lam, w = _batch(26, [1, 2], [40, 50], 8, 2, 16, "bf16")
    ws = fi.Workspace(_config(), device=DEV)
    kvi = torch.zeros(9, dtype=torch.int32, device=DEV)
    for qo, kvp, last in (([0], [0], []), ([0, 0, 0], [0, 3, 7], [4, 5])):
        info = fi.plan(ws, np.array(qo), np.array(kvp), [], np.array(last, dtype=np.int32), 8, 2, 128, 16, 0)
        o = torch.full_like(b.q, float("nan"))
        differential.run(ws, info, b.q, b.k, b.v, kvi, lam, o, None, b.sm_scale)
        assert fi.device_status(ws) == 0 and torch.isnan(o).all()


def test_more_ctas_than_sms():
    b, lam, w = _batch(27, [1, 300, 40, 1], [3000, 800, 900, 70], 16, 4, 16, "bf16", causal=1)
    o, lse, info, ws, _ = _run(b, lam, w, _config(num_ctas=400, decode_min_chunk=64, prefill_min_chunk=128))
    assert fi.device_status(ws) == 0
    _check(b, lam, w, o, lse, rounded=True)


def test_two_streams_at_once():
    """Calls on two streams, each with its workspace, give what they give alone."""
    calls = [_batch(28, [1, 300, 40], [3000, 800, 900], 16, 4, 16, "bf16", causal=1),
             _batch(29, [200, 1, 33], [500, 2000, 33], 8, 2, 4, "fp16", causal=1)]
    alone = [_run(*c, _config()) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for (b, lam, w), (o, _, info, ws, kvi), s in zip(calls, alone, streams):
            with torch.cuda.stream(s):
                x = torch.empty_like(o)
                differential.run(ws, info, b.q, b.k, b.v, kvi, lam, x, None, b.sm_scale, norm_weight=w, stream=s)
                got.append((x[:b.total_qo], o[:b.total_qo]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got) and all(fi.device_status(a[3]) == 0 for a in alone)


def test_repeats_give_the_same_bits():
    b, lam, w = _batch(13, [1, 100, 1, 1], [3000, 500, 70, 4000], 16, 4, 16, "bf16", causal=1)
    first = _run(b, lam, w, _config())
    for _ in range(3):
        o, lse, *_ = _run(b, lam, w, _config(), ws=first[3])
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_plans_of_the_other_kind_are_refused_on_the_device():
    b, lam, w = _batch(14, [1, 1], [40, 50], 8, 2, 16, "bf16")
    o, lse, info, ws, kvi = _run(b, lam, w, _config())
    plain = fi.default_plan_config(0, max_items=1 << 15, max_merge_units=1 << 13, max_partial_rows=1 << 17)
    ws.cfg = plain
    other = fi.plan(ws, b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 8, 2, 128, 16, 0, b.num_pages)
    with pytest.raises(fi.FIError):
        differential.run(ws, other, b.q, b.k, b.v, kvi, lam, o, lse, b.sm_scale)
    o.fill_(float("nan"))
    differential.run(ws, info, b.q, b.k, b.v, kvi, lam, o, lse, b.sm_scale)
    torch.cuda.synchronize()
    assert fi.device_status(ws) == 6 and torch.isnan(o).all()
    ws.cfg = _config()
    fi.plan(ws, b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 8, 2, 128, 16, 0, b.num_pages)
    stale = fi.PlanInfo.from_buffer_copy(other)
    plain_lse = torch.empty(b.q.shape[:2], device=DEV)
    fi.run(ws, stale, b.q, b.k, b.v, kvi, o, plain_lse, b.sm_scale)
    torch.cuda.synchronize()
    assert fi.device_status(ws) == 6 and torch.isnan(o).all()


def test_a_windowed_plan_is_refused_by_a_launch_without_a_window():
    b, lam, w = _batch(14, [200, 1], [400, 50], 8, 2, 16, "bf16", causal=1)
    o, lse, info, ws, kvi = _run(b, lam, w, _config())
    ws.cfg = _config(window_left=20, sink_tokens=2)
    fi.plan(ws, b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 8, 2, 128, 16, 1, b.num_pages)
    o.fill_(float("nan"))
    differential.run(ws, info, b.q, b.k, b.v, kvi, lam, o, lse, b.sm_scale)
    torch.cuda.synchronize()
    assert fi.device_status(ws) == 6 and torch.isnan(o).all()


def test_bad_page_ids_read_as_zeros():
    """An id outside the cache is not followed: its keys and values are zeros."""
    b, lam, w = _batch(15, [1, 30], [40, 64], 8, 2, 16, "bf16", poison=False)
    o, lse, info, ws, kvi = _run(b, lam, None, _config())
    for bad in (b.num_pages, -1, 2**31 - 1):
        broken = kvi.clone()
        broken[1] = bad
        k, v = b.k.clone(), b.v.clone()
        k[int(b.kv_indices[1])] = 0
        v[int(b.kv_indices[1])] = 0
        ref, got = torch.empty_like(o), torch.empty_like(o)
        differential.run(ws, info, b.q, k, v, kvi, lam, ref, None, b.sm_scale)
        differential.run(ws, info, b.q, b.k, b.v, broken, lam, got, None, b.sm_scale)
        torch.cuda.synchronize()
        assert torch.equal(ref, got)
