"""Differential attention without a GPU: the oracle against torch's attention
in fp64 and closed forms, the plan against its re-derivation byte for byte, and
the calls that are refused before any CUDA work."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import serving_attention_gb300 as fi
import workloads
from oracle import diff as oracle_diff
from oracle import plan_ref
from serving_attention_gb300 import differential


def _problem(seed, qo, kv, hq, hkv, page):
    rng = np.random.default_rng(seed)
    kvp, last = workloads._pages_for(np.asarray(kv), page)
    pool = int(kvp[-1]) + 3
    qop = np.concatenate([[0], np.cumsum(qo)])
    q = rng.standard_normal((int(qop[-1]), hq, 128))
    k, v = rng.standard_normal((2, pool, page, hkv, 128))
    return qop, kvp, rng.permutation(pool)[:int(kvp[-1])], last, q, k, v, rng.uniform(-0.5, 1.5, hq), \
        rng.standard_normal(128)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("page,hq,hkv", [(1, 4, 1), (4, 6, 3), (16, 2, 2)])
def test_oracle_is_the_difference_of_two_attentions(causal, page, hq, hkv):
    qo, kv = [3, 1, 7], [11, 5, 7]
    qop, kvp, ids, last, q, k, v, lam, w = _problem(page, qo, kv, hq, hkv, page)
    o, lse = oracle_diff.attention(qop, kvp, ids, last, page, causal, 0.2, q, k, v, lam, w, 1e-3, 0.7)
    t = lambda x: torch.as_tensor(x)  # noqa: E731
    for b in range(3):
        kb = t(k[ids[kvp[b]:kvp[b + 1]]].reshape(-1, hkv, 128)[:kv[b]]).repeat_interleave(hq // hkv, 1).transpose(0, 1)
        vb = t(v[ids[kvp[b]:kvp[b + 1]]].reshape(-1, hkv, 128)[:kv[b]]).repeat_interleave(hq // hkv, 1).transpose(0, 1)
        qb = t(q[qop[b]:qop[b + 1]]).transpose(0, 1)
        mask = torch.ones(qo[b], kv[b], dtype=torch.bool).tril(kv[b] - qo[b]) if causal else None
        maps = [torch.nn.functional.scaled_dot_product_attention(qb[..., d], kb[..., d], vb, attn_mask=mask, scale=0.2)
                for d in (slice(0, 64), slice(64, 128))]
        y = maps[0] - t(lam)[:, None, None] * maps[1]
        y = 0.7 * y / (y.square().mean(-1, keepdim=True) + 1e-3).sqrt() * t(w)
        assert np.abs(y.transpose(0, 1).numpy() - o[qop[b]:qop[b + 1]]).max() < 1e-11
        for i in range(2):
            s = 0.2 * qb[..., 64 * i:64 * i + 64] @ kb[..., 64 * i:64 * i + 64].transpose(1, 2)
            s = s if mask is None else s.masked_fill(~mask, -np.inf)
            assert np.abs(torch.logsumexp(s, -1).T.numpy() - lse[qop[b]:qop[b + 1], :, i]).max() < 1e-12


def test_oracle_closed_forms():
    qop, kvp, ids, last, q, k, v, lam, w = _problem(1, [1], [1], 2, 1, 4)
    o, lse = oracle_diff.attention(qop, kvp, ids, last, 4, 0, 0.2, q, k, v, lam)  # one key: (1 - lambda) v
    assert np.abs(o[0] - (1 - lam)[:, None] * v[ids[0], 0, 0]).max() < 1e-14
    k[..., 64:] = k[..., :64]  # equal maps: (1 - lambda) of one attention, nothing at lambda 1
    q[..., 64:] = q[..., :64]
    o, _ = oracle_diff.attention(qop, kvp, ids, last, 4, 0, 0.2, q, k, v, np.ones(2))
    assert np.abs(o).max() < 1e-14
    o, lse = oracle_diff.attention([0, 2], [0, 0], ids, [1], 4, 1, 0.2, np.ones((2, 2, 128)), k, v, lam)
    assert (o == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("seed", range(24))
def test_plan_matches_reference(seed):
    rng = np.random.default_rng(seed)
    batch, page = int(rng.integers(1, 40)), int(rng.choice([1, 4, 16, 128]))
    hkv, group, causal = int(rng.choice([1, 2, 8])), int(rng.choice([1, 2, 4, 5, 8, 16])), int(rng.integers(0, 2))
    qo = rng.choice([1, 1, 1, 2, 4, 5, 17, 40, 130, 300], size=batch)
    kv = rng.integers(0, 3000, size=batch) * (rng.random(batch) > 0.1)
    kvp, last = workloads._pages_for(kv, page)
    qop = np.concatenate([[0], np.cumsum(qo)]).astype(np.int32)
    window = int(rng.choice([-1, -1, 0, 100, 900]))
    cfg = fi.make_plan_config(int(rng.choice([1, 7, 152])), differential=1, split_factor=int(rng.integers(1, 6)),
                              decode_min_chunk=64, prefill_min_chunk=int(rng.choice([128, 1024])), window_left=window,
                              sink_tokens=int(rng.choice([0, 4])))
    args = (qop, kvp, np.arange(int(kvp[-1])), last, hkv * group, hkv, 128, page, causal, int(kvp[-1]) + 1)
    st, ws, info = fi.plan_host(cfg, *args)
    st_ref, ws_ref, info_ref = plan_ref.make_plan(cfg.as_dict(), *args)
    assert st == st_ref == 0 and np.array_equal(ws, ws_ref)
    got = info.as_dict()
    assert all(got[k] == v for k, v in info_ref.items())
    assert info.variant & 8 and info.num_late_merge_units == info.num_merge_units
    # chunks of a merge unit own disjoint partial rows, two per packed row
    spans = []
    for i in range(info.num_items):
        f = ws[int(ws[7]) + 16 * i: int(ws[7]) + 16 * i + 16]
        assert f[3] - f[2] <= 128 and f[12] == 0
        if f[6] >= 0:
            spans.append((f[6], f[6] + 2 * (f[3] - f[2])))
    spans.sort()
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])) and all(s[1] <= info.num_partial_rows for s in spans)


@pytest.mark.parametrize("page", [1, 4, 8])
def test_requests_of_few_rows_come_behind_prompts(page):
    """On pages below 8 tokens requests of 17 to 32 packed rows take the 16-row path, which a CTA does not leave
    again: they come behind its larger ones, however long, and before those of up to 16 rows."""
    qo, kv = [8, 100, 1, 5, 300, 7, 64], [9000, 300, 5000, 8000, 400, 6000, 64]
    kvp, last = workloads._pages_for(np.asarray(kv), page)
    cfg = fi.make_plan_config(3, differential=1)
    args = (np.concatenate([[0], np.cumsum(qo)]), kvp, np.arange(int(kvp[-1])), last, 8, 2, 128, page, 1,
            int(kvp[-1]) + 1)
    st, ws, info = fi.plan_host(cfg, *args)
    assert st == 0 and np.array_equal(ws, plan_ref.make_plan(cfg.as_dict(), *args)[1])
    for c in range(3):
        items = ws[ws[7] + 16 * ws[32 + c]:ws[7] + 16 * ws[33 + c]].reshape(-1, 16)
        kinds = [0 if r > (32 if page < 8 else 16) else 1 if r > 16 else 2 for r in items[:, 9] * 4]
        assert kinds == sorted(kinds)


@pytest.mark.parametrize("field,value,status", [("differential", 2, 1), ("differential", -1, 1),
                                                ("logits_soft_cap", 30.0, 2), ("rope_max_positions", 4096, 2)])
def test_plan_refusals(field, value, status):
    cfg = fi.make_plan_config(8, **{"differential": 1, field: value})
    args = (np.array([0, 1]), np.array([0, 1]), np.array([0]), np.array([3]), 8, 2, 128, 16, 0)
    assert fi.plan_host(cfg, *args)[0] == status
    assert plan_ref.make_plan(cfg.as_dict(), *args, 0)[0] == status


@pytest.mark.parametrize("keys,status", [(2**31 - 1, 2), (2**31 - 256, 2), (2**31 - 257, 0)])
def test_plan_refuses_requests_whose_tiles_pass_an_int32(keys, status):
    cfg = fi.make_plan_config(8, differential=1)
    args = (np.array([0, 1]), np.array([0, -(-keys // 128)]), np.array([0]), np.array([(keys - 1) % 128 + 1]), 8, 2,
            128, 128, 0)
    assert fi.plan_host(cfg, *args)[0] == status
    assert plan_ref.make_plan(cfg.as_dict(), *args, 0)[0] == status


def test_cascade_refuses_differential():
    cfg = fi.make_plan_config(8, differential=1)
    one = (np.array([0, 1]), np.array([0, 1]), np.array([0]), np.array([3]))
    assert fi.plan_cascade_host(cfg, *one, 16, *one, 8, 2, 128, 16, 0)[0] == 2


def _run(**kw):
    """The status of a call whose pointers are fake: every case returns before any CUDA call."""
    info = fi.PlanInfo(num_ctas=1, head_dim=128, page_size=16, num_qo_heads=8, num_kv_heads=2, variant=8)
    a = dict(info=ctypes.addressof(info), q=16, qt=1024, qh=128, n=4, k=32, k0=4096, k1=256, k2=128, v=64, v0=4096,
             v1=256, v2=128, pages=10, idx=48, lam=80, w=96, o=112, ot=1024, oh=128, lse=128, dt=fi.BF16, iws=144,
             fws=160, sm=0.1, eps=1e-5, scale=1.0, reserved=0.0)
    for name, value in kw.items():
        if name in a:
            a[name] = value
        else:
            setattr(info, name, value)
    lib = differential.load()
    return lib.fi_batch_paged_attention_run_differential(differential._ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(info=0), 1), (dict(q=0), 1), (dict(o=0), 1), (dict(lam=0), 1), (dict(iws=0), 1), (dict(k=0), 1),
    (dict(v=0), 1), (dict(idx=0), 1), (dict(pages=0), 1), (dict(pages=1 << 31), 1), (dict(n=0), 1),
    (dict(sm=float("nan")), 1), (dict(sm=0.0), 1), (dict(sm=-0.125), 1), (dict(sm=1e-40), 1), (dict(sm=3e38), 1),
    (dict(scale=float("inf")), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(dt=fi.FP32), 2), (dict(q=18), 4), (dict(o=120), 4), (dict(lam=82), 4), (dict(lse=130), 4),
    (dict(qt=1020), 4), (dict(oh=0), 4), (dict(k1=250), 4), (dict(v2=-128), 4),
    (dict(variant=0), 1), (dict(variant=4), 1), (dict(num_ctas=0), 1), (dict(head_dim=64), 2),
    (dict(page_size=24), 2), (dict(num_kv_heads=3), 2), (dict(fws=0, num_partial_rows=4), 1)])
def test_run_refusals(kw, status):
    assert _run(**kw) == status


@pytest.mark.parametrize("heads", [0, -2])
def test_run_refuses_a_plan_without_heads(heads):
    assert _run(num_qo_heads=heads, page_size=4) == 2


def test_run_refuses_no_arguments():
    assert differential.load().fi_batch_paged_attention_run_differential(None, None) == 1


def test_ordinary_run_refuses_a_differential_plan():
    info = fi.PlanInfo(num_ctas=1, head_dim=128, page_size=16, num_qo_heads=8, num_kv_heads=2, variant=8)
    ks = (ctypes.c_int64 * 3)(4096, 256, 128)
    assert fi.load().fi_batch_paged_attention_run(ctypes.byref(info), 16, 1024, 128, 4, 32, ks, 64, ks, 10, 48, 80,
                                                  1024, 128, None, fi.BF16, 0.1, 96, 112, None) == 1


def test_binding_refuses_cpu_tensors():
    class Ws:
        int_ws, float_ws = torch.zeros(4, dtype=torch.int32), torch.zeros(4)

    info = fi.PlanInfo(num_ctas=1, head_dim=128, page_size=16, num_qo_heads=2, num_kv_heads=1, variant=8)
    q = torch.zeros(1, 2, 128, dtype=torch.float16)
    c = torch.zeros(1, 16, 1, 128, dtype=torch.float16)
    idx, lam = torch.zeros(1, dtype=torch.int32), torch.zeros(2)
    with pytest.raises(TypeError):
        differential.run(Ws(), info, q, c, c, idx, lam, q, None, 0.1)
    with pytest.raises(TypeError):
        differential.run(Ws(), info, q, c.bfloat16(), c, idx, lam, q, None, 0.1)
    with pytest.raises(TypeError):
        differential.run(Ws(), info, q, c, c, idx.long(), lam, q, None, 0.1)
    with pytest.raises(TypeError):
        differential.run(Ws(), info, q, c, c, idx, lam.half(), q, None, 0.1)
    with pytest.raises(ValueError):
        differential.run(Ws(), info, q[:, :1], c, c, idx, lam, q, None, 0.1)
    with pytest.raises(ValueError):
        differential.run(Ws(), info, q, c[:, :8], c, idx, lam, q, None, 0.1)
    with pytest.raises(ValueError):
        differential.run(Ws(), info, q, c, c, idx, torch.zeros(3), q, None, 0.1)
    with pytest.raises(ValueError):
        differential.run(Ws(), info, q, c, c, idx, lam, q, torch.zeros(1, 2), 0.1)
    with pytest.raises(ValueError):
        differential.run(Ws(), info, q, c, c, idx, lam, q, None, 0.1, norm_weight=torch.ones(64))


def test_every_entry_is_declared():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "fi_diff.h")).read()
    assert set(re.findall(r"^fi_status\s+(fi_\w+)\s*\(", text, re.M)) == set(differential.EXPORTS)
