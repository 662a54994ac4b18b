"""Sliding window, attention sink and logits soft-cap: CUDA path (through the C
ABI) against the fp64 oracle, same bar as the plain path (O max-abs <= 8e-3,
LSE abs <= 1e-3, blind rows exactly (0, -inf))."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import serving_attention_gb300 as fi
import workloads
from helpers import LSE_TOL, O_TOL, compare, gpu_run, oracle_problem

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _variant_cfg(window=-1, sink=0, cap=0.0, **kw):
    return fi.default_plan_config(0, window_left=window, sink_tokens=sink, logits_soft_cap=cap, **kw)


def _full(b, window=-1, sink=0, cap=0.0, **kw):
    o, lse, info, ws = gpu_run(b, cfg=_variant_cfg(window, sink, cap, **kw))
    torch.cuda.synchronize()
    assert fi.device_status(ws) == 0
    o_ref, l_ref = oracle.attention(oracle_problem(b, window, sink, cap))
    n = b.total_qo
    err_o, err_l = compare(o[:n], lse[:n], o_ref, l_ref)
    assert err_o <= O_TOL and err_l <= LSE_TOL, (err_o, err_l)
    return info


@pytest.mark.parametrize("seed,page,group,causal,qo_max,window,sink,cap", [
    (301, 16, 4, 0, 1, 100, 0, 0.0),     # decode, window only
    (302, 16, 4, 0, 1, 100, 4, 0.0),     # decode, window + sink
    (303, 4, 2, 1, 3, 37, 2, 0.0),       # small pages, causal, several tokens per 16-row tile
    (304, 16, 8, 0, 1, -1, 0, 3.0),      # decode, soft-cap only
    (305, 16, 4, 1, 2, 64, 3, 10.0),     # all three
    (306, 1, 4, 1, 9, 20, 1, 0.0),       # page 1 (CUDA-core prefill path), window + sink
    (307, 32, 4, 1, 40, 300, 16, 5.0),   # prefill-class rows on the tensor cores (q scaled 2.5x: still clear)
    (308, 16, 1, 0, 1, 0, 0, 0.0),       # zero window: each query sees its own position only
])
def test_variants_small_full(seed, page, group, causal, qo_max, window, sink, cap):
    hkv = 2
    b = workloads.random_batch(seed, batch=6, qo_max=qo_max, kv_max=1500, num_qo_heads=hkv * group,
                               num_kv_heads=hkv, page_size=page, causal=causal, device=DEV, kv_min=1)
    if cap > 0:
        b.q.mul_(2.5)  # logits large enough for the cap to bend them
    _full(b, window, sink, cap, num_ctas=9, decode_min_chunk=64, prefill_min_chunk=128, split_factor=3)


@pytest.mark.parametrize("qo,kv,window,sink,cap", [
    ([100], [900], 200, 0, 0.0),         # 400 rows: two items, window edge inside tiles
    ([100], [900], 200, 8, 0.0),         # ... with sink keys in the first tile
    ([64, 33], [1000, 40], 130, 5, 3.0),
    ([40], [300], -1, 0, 2.0),           # strong cap, no window
])
def test_variants_tensor_core_tiles(qo, kv, window, sink, cap):
    """N(0,1) queries: logits up to about +-4, which caps of 2-3 bend strongly.
    (Scaled-up queries make the softmax peaked enough for the 16-bit rounding
    of P in the P V MMA to reach the O bar on its own, variant or not.)"""
    b = workloads.make_batch("tcv", "bf16", qo, kv, 8, 2, 16, 1, 400 + kv[0] + max(window, 0), DEV,
                             pool_pages=sum((k + 15) // 16 for k in kv) + 2)
    info = _full(b, window, sink, cap)
    assert info.num_prefill_items > 0


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 20, 3])
def test_widest_windows_of_queries_before_the_keys(window, page):
    """More queries than keys without the causal mask: the first ones lie before key 0, and
    their distance to the window's lowest key passes an int."""
    b = workloads.make_batch("wide", "bf16", [40, 3, 2], [10, 1, 100], 8, 2, page, 0, 500, DEV)
    _full(b, window)


def test_windowed_long_decode_sampled():
    """Llama-3-8B-shaped decode with a 4096-token window and 4 sink tokens."""
    b = workloads.llama8b_decode(device=DEV, batch=16)
    cfg = _variant_cfg(4096, 4)
    o, lse, info, ws = gpu_run(b, cfg=cfg)
    torch.cuda.synchronize()
    assert fi.device_status(ws) == 0
    rows = np.arange(b.total_qo, dtype=np.int64)
    heads = np.array([0, 7, 21, 31])
    rr, hh = np.repeat(rows, len(heads)), np.tile(heads, len(rows))
    o_ref, l_ref = oracle.attention_select(oracle_problem(b, 4096, 4), rr, hh)
    err_o, err_l = compare(o[torch.as_tensor(rr), torch.as_tensor(hh)], lse[torch.as_tensor(rr), torch.as_tensor(hh)],
                           o_ref, l_ref)
    assert err_o <= O_TOL and err_l <= LSE_TOL, (err_o, err_l)


def test_windowed_ragged_prefill_sampled():
    b = workloads.ragged_prefill(device=DEV, batch=4)
    o, lse, info, ws = gpu_run(b, cfg=_variant_cfg(1024, 16, 50.0))
    torch.cuda.synchronize()
    assert fi.device_status(ws) == 0
    rows = []
    for r in range(b.batch):
        q0, q1 = int(b.qo_indptr[r]), int(b.qo_indptr[r + 1])
        rows += [q0, q0 + 1, (q0 + q1) // 2, q1 - 1]
    rows = np.array(rows, np.int64)
    heads = np.array([0, 5, 30])
    rr, hh = np.repeat(rows, len(heads)), np.tile(heads, len(rows))
    o_ref, l_ref = oracle.attention_select(oracle_problem(b, 1024, 16, 50.0), rr, hh)
    err_o, err_l = compare(o[torch.as_tensor(rr), torch.as_tensor(hh)], lse[torch.as_tensor(rr), torch.as_tensor(hh)],
                           o_ref, l_ref)
    assert err_o <= O_TOL and err_l <= LSE_TOL, (err_o, err_l)


def test_soft_cap_extreme_logits():
    """Soft-cap on logits far past the cap (keys scaled by 1e4, |y| well above
    the exponential's range of 126) and exactly zero: the capped logits sit
    at +-cap, and O and LSE still meet the bar against the oracle."""
    b = workloads.make_batch("capx", "bf16", [64, 3], [300, 40], 8, 2, 16, 1, 733, DEV,
                             pool_pages=(300 + 15) // 16 + (40 + 15) // 16 + 2)
    b.k.mul_(1.0e4)
    b.k[:, 3].zero_()  # slot 3 of every page: logit exactly 0
    cfg = fi.default_plan_config(0, logits_soft_cap=30.0)
    o, lse, info, ws = gpu_run(b, cfg=cfg)
    torch.cuda.synchronize()
    assert fi.device_status(ws) == 0 and info.num_prefill_items > 0
    o_ref, l_ref = oracle.attention(oracle_problem(b, -1, 0, 30.0))
    n = b.total_qo
    err_o, err_l = compare(o[:n], lse[:n], o_ref, l_ref)
    assert err_o <= O_TOL and err_l <= LSE_TOL, (err_o, err_l)


@pytest.mark.parametrize("dtype,cap,qscale", [("fp16", 30.0, 20.0), ("fp16", 50.0, 40.0), ("bf16", 5.0, 4.0),
                                              ("bf16", 2.0, 1.5)])
def test_soft_cap_logits_near_the_cap(dtype, cap, qscale):
    """Logits of the order of the cap itself (queries scaled so that s / cap
    spreads over about +-1), where the capped logit bends most and a relative
    error in tanh weighs most: tensor-core tiles against the oracle.  Caps of
    30 and 50 run in fp16: logits that large make rows so peaked that in bf16
    the 16-bit rounding of P and of the stored O alone reaches the flat bar
    (8.2e-3 measured at cap 30), as with the peaked-softmax cases."""
    b = workloads.make_batch("capn", dtype, [64, 40], [700, 300], 8, 2, 16, 1, 761 + int(cap), DEV,
                             pool_pages=(700 + 15) // 16 + (300 + 15) // 16 + 2)
    b.q.mul_(qscale)
    cfg = fi.default_plan_config(0, logits_soft_cap=cap)
    o, lse, info, ws = gpu_run(b, cfg=cfg)
    torch.cuda.synchronize()
    assert fi.device_status(ws) == 0 and info.num_prefill_items > 0
    o_ref, l_ref = oracle.attention(oracle_problem(b, -1, 0, cap))
    n = b.total_qo
    err_o, err_l = compare(o[:n], lse[:n], o_ref, l_ref)
    assert err_o <= O_TOL and err_l <= LSE_TOL, (err_o, err_l)
