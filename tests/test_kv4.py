"""The 4-bit cache on the CPU: the oracle's format and quantiser, plans, and every refusal."""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import serving_attention_gb300 as fi
import workloads
from oracle import kv4 as oracle_kv4
from oracle import plan_ref
from serving_attention_gb300 import kv4, step

F = np.float32


# ------------------------------------------------------------------ format

@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128])
def test_layout(page):
    """No two rows or words of a page share a byte; a cache of values reads back slot by slot."""
    assert kv4.page_bytes(page) == oracle_kv4.page_bytes(page) and kv4.page_bytes(page) % 16 == 0
    taken = np.zeros(kv4.page_bytes(page), int)
    for slot in range(page):
        k, v, kw, vw = oracle_kv4.places(page, slot)
        for at, n in ((k, 64), (v, 64), (kw, 2), (vw, 2)):
            taken[at:at + n] += 1
    assert taken.max() == 1 and taken.sum() == 132 * page
    rng = np.random.default_rng(page)
    cache = np.zeros((3, 2, kv4.page_bytes(page)), np.uint8)
    for slot in range(3 * page):
        for h in range(2):
            oracle_kv4.put(cache, page, slot, h, rng.standard_normal(128), rng.standard_normal(128))
    ka, va = oracle_kv4.all_values(cache, page)
    for slot in range(3 * page):
        for h in range(2):
            k, v = oracle_kv4.get(cache, page, slot, h)
            assert np.array_equal(ka[slot // page, slot % page, h], k)
            assert np.array_equal(va[slot // page, slot % page, h], v)


@pytest.mark.parametrize("page", [0, -1, 3, 24, 256])
def test_page_bytes_refusals(page):
    assert kv4.load().fi_kv4_page_bytes(page) == 0
    with pytest.raises(ValueError):
        kv4.page_bytes(page)


def test_quantiser():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((4000, 128)) * np.exp(rng.uniform(-12, 8, (4000, 1)))).astype(F)
    x[:40] = np.abs(x[:40])
    x[40:80] = -np.abs(x[40:80])
    n, w = oracle_kv4.quantise(x)
    s = (w & 0xFFF0).astype(np.uint16).view(np.float16).astype(np.float64)
    got = oracle_kv4.values(n, w)
    lo, hi = np.minimum(x.min(-1), 0), np.maximum(x.max(-1), 0)
    exact = (hi.astype(np.float64) - lo) / 15
    big = exact >= 2.0**-14
    # s: rounded to fp16 (off by 2^-11 of it, below 2^-14 by half a subnormal's step of 2^-24: 2^-25), then up by at
    # most 15 of its 1024 steps
    assert (s >= exact * (1 - 2.0**-11) * (1 - 1e-6) - 2.0**-25).all() and (s[big] <= exact[big] * (1 + 2.0**-11 + 15 / 1024)).all()
    # a value is at most half a step off, and those at the ends by what z's rounding shifts them
    assert (np.abs(got - x) <= s[:, None] * (1.0 + 2.0**-6) + 1e-12).all()
    inner = (x > (lo + s)[:, None]) & (x < (hi - s)[:, None])
    assert (np.abs(got - x)[inner] <= (np.broadcast_to(s[:, None], x.shape) * 0.5 * (1 + 1e-5))[inner]).all()
    assert np.array_equal(got.astype(np.float16).astype(np.float64), got)  # every value is an fp16
    assert np.array_equal(oracle_kv4.values(*oracle_kv4.quantise(np.zeros((1, 128)))), np.zeros((1, 128)))


def test_quantiser_ends():
    """Infinities and values beyond 15 * 4096 saturate; a NaN is code 0 and does not touch the others."""
    x = np.linspace(-1, 1, 128).astype(F)
    y = x.copy()
    y[5] = np.nan
    n, w = oracle_kv4.quantise(y[None])
    n0, w0 = oracle_kv4.quantise(x[None])
    assert w == w0 and n[0, 5] == 0 and np.array_equal(np.delete(n[0], 5), np.delete(n0[0], 5))
    for big in (np.inf, 1e30, 70000.0):
        y[5] = big
        v = oracle_kv4.values(*oracle_kv4.quantise(y[None]))[0]
        assert np.isfinite(v).all() and abs(v[5]) <= 15 * 4096 and v[5] >= 50000
    y[5] = -np.inf
    v = oracle_kv4.values(*oracle_kv4.quantise(y[None]))[0]
    assert v[5] == -15 * 4096


def test_oracle_attention_is_attention():
    rng = np.random.default_rng(3)
    P, Hkv, G, n = 8, 2, 3, 29
    pages = -(-n // P)
    k, v = rng.standard_normal((2, pages + 1, P, Hkv, 128))
    q = rng.standard_normal((4, Hkv * G, 128))
    ids = rng.permutation(pages + 1)[:pages]
    o, lse, _ = oracle_kv4.attention([0, 4], [0, pages], ids, [n - (pages - 1) * P], P, 1, 0.1, q, k, v)
    kf = torch.tensor(k[ids].reshape(-1, Hkv, 128)[:n]).repeat_interleave(G, 1)
    vf = torch.tensor(v[ids].reshape(-1, Hkv, 128)[:n]).repeat_interleave(G, 1)
    mask = torch.ones(4, n, dtype=torch.bool).tril(n - 4)
    ref = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q).transpose(0, 1), kf.transpose(0, 1),
                                                           vf.transpose(0, 1), attn_mask=mask, scale=0.1)
    assert np.abs(o - ref.transpose(0, 1).numpy()).max() < 1e-12
    x = torch.einsum("thd,nhd->htn", torch.tensor(q), kf) * 0.1
    assert np.abs(lse - torch.logsumexp(x.masked_fill(~mask, -np.inf), -1).T.numpy()).max() < 1e-12


# ------------------------------------------------------------------- plans

@pytest.mark.parametrize("seed", range(24))
def test_plan_matches_reference(seed):
    rng = np.random.default_rng(seed)
    batch, page = int(rng.integers(1, 40)), int(rng.choice([1, 4, 16, 128]))
    hkv, group, causal = int(rng.choice([1, 2, 8])), int(rng.choice([1, 2, 4, 5, 8, 16])), int(rng.integers(0, 2))
    qo = rng.choice([1, 1, 1, 2, 4, 5, 17, 40, 130, 300], size=batch)
    kv = rng.integers(0, 3000, size=batch) * (rng.random(batch) > 0.1)
    kvp, last = workloads._pages_for(kv, page)
    qop = np.concatenate([[0], np.cumsum(qo)]).astype(np.int32)
    cfg = fi.make_plan_config(int(rng.choice([1, 7, 152])), kv_bits=4, split_factor=int(rng.integers(1, 6)),
                              decode_min_chunk=64, prefill_min_chunk=int(rng.choice([128, 1024])),
                              window_left=int(rng.choice([-1, -1, 0, 100, 900])), sink_tokens=int(rng.choice([0, 4])),
                              decode_cost_weight=int(rng.choice([1, 8, 9])))
    args = (qop, kvp, np.arange(int(kvp[-1])), last, hkv * group, hkv, 128, page, causal, int(kvp[-1]) + 1)
    st, ws, info = fi.plan_host(cfg, *args)
    st_ref, ws_ref, info_ref = plan_ref.make_plan(cfg.as_dict(), *args)
    assert st == st_ref == 0 and np.array_equal(ws, ws_ref)
    got = info.as_dict()
    assert all(got[k] == v for k, v in info_ref.items())
    assert info.variant & 16 and ws[0] == plan_ref.MAGIC_KV4
    assert all(ws[int(ws[7]) + 16 * i + 12] == 0 for i in range(info.num_items))  # no multi-head units


def _items(ws, info):
    at = int(ws[7])
    return [tuple(int(x) for x in ws[at + 16 * i:at + 16 * i + 6]) for i in range(info.num_items)]


@pytest.mark.parametrize("qo,kv,hq,hkv,kw,ctas,most", [
    ([1, 1], [99991, 131072], 64, 8, {}, 152, 152),                    # 160 items by the shares alone: one wave
    ([1, 1, 1], [5000, 70000, 64], 8, 2, {}, 7, None),                 # one wave would leave 70000 keys to one CTA
    ([400], [9000], 32, 8, {}, 152, 152),                              # prefill class
    ([200, 60], [4000, 2500], 16, 4, {"window_left": 1023, "sink_tokens": 4}, 152, 152),
    ([1] * 40, [3000] * 40, 8, 4, {}, 152, None),                      # more units than CTAs
    ([1, 1], [99991, 131072], 64, 8, {"split_factor": 2}, 152, None),
])
def test_plan_splits_evenly_and_in_one_wave(qo, kv, hq, hkv, kw, ctas, most):
    page = 16
    pages = [-(-n // page) for n in kv]
    args = (np.cumsum([0] + qo).astype(np.int32), np.cumsum([0] + pages).astype(np.int32), [],
            np.array([n - (p - 1) * page for n, p in zip(kv, pages)], np.int32), hq, hkv, 128, page, 1)
    cfg = fi.make_plan_config(ctas, kv_bits=4, **kw)
    st, ws, info = fi.plan_host(cfg, *args)
    st_ref, ws_ref, _ = plan_ref.make_plan(cfg.as_dict(), *args, 0)
    assert st == st_ref == 0 and np.array_equal(ws[:len(ws_ref)], ws_ref)
    if most:
        assert info.num_items <= most
    units = {}
    for b, hk, r0, r1, k0, k1 in _items(ws, info):
        units.setdefault((b, hk, r0), []).append((k0, k1))
    granule = 64 if max(q * hq // hkv for q in qo) <= 16 else 128
    for at in units.values():
        runs = [[p] for p in sorted(at)[:1]]
        for p in sorted(at)[1:]:  # a range's pieces follow one another
            if runs[-1][-1][1] == p[0]:
                runs[-1].append(p)
            else:
                runs.append([p])
        for run in runs:
            steps = {b - a for a, b in run[:-1]}
            assert len(steps) <= 1
            if steps:  # equal but for the granule, which the last piece makes up for
                n, step = len(run), steps.pop()
                assert step - (run[-1][1] - run[-1][0]) < n * granule


@pytest.mark.parametrize("field,value,status", [("kv_bits", 3, 1), ("kv_bits", -4, 1), ("kv_bits", 8, 1),
                                                ("logits_soft_cap", 30.0, 2), ("rope_max_positions", 4096, 2),
                                                ("differential", 1, 2)])
def test_plan_refusals(field, value, status):
    cfg = fi.make_plan_config(8, **{"kv_bits": 4, field: value})
    args = (np.array([0, 1]), np.array([0, 1]), np.array([0]), np.array([3]), 8, 2, 128, 16, 0)
    assert fi.plan_host(cfg, *args)[0] == status
    assert plan_ref.make_plan(cfg.as_dict(), *args, 0)[0] == status


@pytest.mark.parametrize("keys,status", [(2**31 - 1, 2), (2**31 - 256, 2), (2**31 - 257, 0)])
def test_plan_refuses_requests_whose_tiles_pass_an_int32(keys, status):
    cfg = fi.make_plan_config(8, kv_bits=4)
    args = (np.array([0, 1]), np.array([0, -(-keys // 128)]), np.array([0]), np.array([(keys - 1) % 128 + 1]), 8, 2,
            128, 128, 0)
    assert fi.plan_host(cfg, *args)[0] == status
    assert plan_ref.make_plan(cfg.as_dict(), *args, 0)[0] == status


def test_cascade_refuses_four_bits():
    cfg = fi.make_plan_config(8, kv_bits=4)
    one = (np.array([0, 1]), np.array([0, 1]), np.array([0]), np.array([3]))
    assert fi.plan_cascade_host(cfg, *one, 16, *one, 8, 2, 128, 16, 0)[0] == 2


def test_sixteen_bits_is_the_ordinary_plan():
    args = (np.array([0, 1]), np.array([0, 1]), np.array([0]), np.array([3]), 8, 2, 128, 16, 0)
    a, b = (fi.plan_host(fi.make_plan_config(8, kv_bits=bits), *args) for bits in (0, 16))
    assert a[0] == b[0] == 0 and np.array_equal(a[1], b[1])


# ---------------------------------------------------------------- refusals

def _run(**kw):
    """The status of a call whose pointers are fake: every case returns before any CUDA call."""
    info = fi.PlanInfo(num_ctas=1, head_dim=128, page_size=16, num_qo_heads=8, num_kv_heads=2, variant=16)
    a = dict(info=ctypes.addressof(info), q=16, qt=1024, qh=128, n=4, cache=32, cp=4224, ch=2112, pages=10, idx=48,
             o=112, ot=1024, oh=128, lse=128, dt=fi.BF16, iws=144, fws=160, sm=0.1, reserved=0.0)
    for name, value in kw.items():
        if name in a:
            a[name] = value
        else:
            setattr(info, name, value)
    return kv4.load().fi_batch_paged_attention_run_kv4(kv4._RUN_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(info=0), 1), (dict(q=0), 1), (dict(o=0), 1), (dict(iws=0), 1), (dict(cache=0), 1), (dict(idx=0), 1),
    (dict(pages=0), 1), (dict(pages=1 << 31), 1), (dict(n=0), 1), (dict(n=1 << 31), 1), (dict(sm=float("nan")), 1),
    (dict(sm=0.0), 1), (dict(sm=-0.125), 1), (dict(sm=1e-40), 1), (dict(sm=3e38), 1), (dict(dt=fi.FP32), 2),
    (dict(q=18), 4), (dict(o=120), 4), (dict(lse=130), 4), (dict(cache=40), 4), (dict(qt=1020), 4), (dict(oh=0), 4),
    (dict(cp=4216), 4), (dict(ch=8), 4), (dict(cp=-4224), 1), (dict(variant=0), 1), (dict(variant=8), 1),
    (dict(num_ctas=0), 1), (dict(head_dim=64), 2), (dict(page_size=24), 2), (dict(num_kv_heads=3), 2),
    (dict(num_qo_heads=0), 2), (dict(num_qo_heads=34), 2), (dict(fws=0, num_partial_rows=4), 1)])
def test_run_refusals(kw, status):
    assert _run(**kw) == status


def test_other_runs_refuse_the_plan():
    info = fi.PlanInfo(num_ctas=1, head_dim=128, page_size=16, num_qo_heads=8, num_kv_heads=2, variant=16)
    ks = (ctypes.c_int64 * 3)(4096, 256, 128)
    assert fi.load().fi_batch_paged_attention_run(ctypes.byref(info), 16, 1024, 128, 4, 32, ks, 64, ks, 10, 48, 80,
                                                  1024, 128, None, fi.BF16, 0.1, 96, 112, None) == 1
    from serving_attention_gb300 import differential
    args = [ctypes.addressof(info), 16, 1024, 128, 4, 32, 4096, 256, 128, 64, 4096, 256, 128, 10, 48, 80, 96, 112,
            1024, 128, 128, fi.BF16, 144, 160, 0.1, 1e-5, 1.0, 0.0]
    assert differential.load().fi_batch_paged_attention_run_differential(differential._ARGS.pack(*args), None) == 1


_ROT = step.rotary_setup(128)


def _append(**kw):
    a = dict(rot=ctypes.addressof(_ROT), pos=16, slots=32, n=4, q=48, qt=1024, qh=128, qo=1 << 20, qot=1024, qoh=128,
             hq=8, k=64, kt=256, kh=128, v=80, vt=256, vh=128, hk=2, qw=96, qws=0, kw=112, kws=0, cache=128, cp=4224,
             ch=2112, page=16, pages=10, dt=fi.BF16, eps=1e-6)
    a.update(kw)
    return kv4.load().fi_kv4_append(kv4._APPEND_ARGS.pack(*a.values()), None)


_ROT64 = step.rotary_setup(64)


@pytest.mark.parametrize("kw,status", [
    (dict(pos=0), 1), (dict(slots=0), 1), (dict(q=0), 1), (dict(qo=0), 1), (dict(k=0), 1), (dict(v=0), 1),
    (dict(cache=0), 1), (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(hq=-1), 1), (dict(hk=0), 1), (dict(hk=-2), 1),
    (dict(pages=0), 1), (dict(pages=1 << 31), 1), (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1),
    (dict(eps=1e300), 1), (dict(rot=ctypes.addressof(_ROT64)), 2), (dict(dt=fi.FP32), 2), (dict(page=24), 2),
    (dict(page=256), 2), (dict(page=0), 2), (dict(hq=70000), 2), (dict(pos=18), 4), (dict(slots=34), 4),
    (dict(q=52), 4), (dict(kt=252), 4), (dict(vh=-128), 4), (dict(cache=136), 4), (dict(cp=4220), 4), (dict(ch=2104), 4),
    (dict(ch=2096), 1), (dict(cp=2112), 1), (dict(cp=-4224), 1), (dict(qw=100), 4), (dict(qws=64), 1), (dict(kws=-128), 1),
    (dict(kws=130), 4), (dict(qoh=64), 1), (dict(q=48, qo=48 + 256), 1)])
def test_append_refusals(kw, status):
    assert _append(**kw) == status


def test_append_without_tokens_needs_no_pointers():
    assert _append(n=0, pos=0, slots=0, q=0, qo=0, k=0, v=0, cache=0, qw=0, kw=0) == 0
    assert kv4.load().fi_kv4_append(None, None) == kv4.load().fi_kv4_read(None, None) == 1
    assert kv4.load().fi_batch_paged_attention_run_kv4(None, None) == 1


def _read(**kw):
    a = dict(slots=32, n=4, k=64, kt=256, kh=128, v=1 << 20, vt=256, vh=128, hk=2, cache=128, cp=4224, ch=2112,
             page=16, pages=10, dt=fi.BF16)
    a.update(kw)
    return kv4.load().fi_kv4_read(kv4._READ_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(slots=0), 1), (dict(cache=0), 1), (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(hk=0), 1), (dict(pages=0), 1),
    (dict(dt=fi.FP32), 2), (dict(page=3), 2), (dict(slots=33), 4), (dict(k=72), 4), (dict(vt=100), 4),
    (dict(cache=129), 4), (dict(cp=2112), 1), (dict(kt=128), 1), (dict(vt=0), 1), (dict(n=0, slots=0, cache=0), 0),
    (dict(k=0, v=0, slots=0), 0)])
def test_read_refusals(kw, status):
    assert _read(**kw) == status


def test_bindings_refuse_wrong_tensors():
    class Ws:
        int_ws, float_ws = torch.zeros(4, dtype=torch.int32), torch.zeros(4)

    info = fi.PlanInfo(num_ctas=1, head_dim=128, page_size=16, num_qo_heads=2, num_kv_heads=1, variant=16)
    q, idx = torch.zeros(3, 2, 128).half(), torch.zeros(3, dtype=torch.int32)
    k, c = q[:, :1], kv4.empty_cache(2, 16, 1, "cpu")
    run = lambda *a: kv4.run(Ws(), info, *a, 0.1)  # noqa: E731
    with pytest.raises(TypeError):  # not on a GPU
        run(q, c, idx, q.clone(), None)
    with pytest.raises(TypeError):
        run(q, c, idx.long(), q.clone(), None)
    with pytest.raises(TypeError):
        run(q, c.view(torch.int8), idx, q.clone(), None)
    with pytest.raises(TypeError):
        run(q, c, idx, q.float(), None)
    with pytest.raises(ValueError):
        run(q[:, :1], c, idx, q[:, :1], None)
    with pytest.raises(ValueError):
        run(q, c[..., :16], idx, q.clone(), None)
    with pytest.raises(ValueError):
        run(q, c, idx, q.clone(), torch.zeros(3))
    append = lambda *a, **kw: kv4.append(*a, 16, **kw)  # noqa: E731
    with pytest.raises(TypeError):
        append(_ROT, idx, idx, q, q.clone(), k, k, c)
    with pytest.raises(TypeError):
        append(_ROT, idx, idx, q, q.clone(), k, k.float(), c)
    with pytest.raises(TypeError):
        append(_ROT, idx, idx, q, q.clone(), k, k, c, q_weight=torch.ones(128).half())
    with pytest.raises(ValueError):
        append(_ROT64, idx, idx, q, q.clone(), k, k, c)
    with pytest.raises(ValueError):
        append(_ROT, None, idx, q, q.clone(), k, k, c)
    with pytest.raises(ValueError):
        append(_ROT, idx[:2], idx, q, q.clone(), k, k, c)
    with pytest.raises(ValueError):
        append(_ROT, idx, idx, q, None, k, k, c)
    with pytest.raises(ValueError):
        append(_ROT, idx, idx, q, q.clone(), k, k[..., :64], c)
    with pytest.raises(ValueError):
        append(_ROT, idx, idx, q, q.clone(), q, q, c)  # heads of the cache
    with pytest.raises(ValueError):
        append(_ROT, idx, idx, q, q.clone(), k, k, c, k_weight=torch.ones(2, 128))
    with pytest.raises(TypeError):
        kv4.read(idx, c, 16, k, k.clone())
    with pytest.raises(ValueError):
        kv4.read(idx, c, 16, None, None)
    with pytest.raises(ValueError):
        kv4.read(idx[:2], c, 16, k, None)


def test_every_entry_is_declared():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "fi_kv4.h")).read()
    assert set(re.findall(r"^(?:fi_status|size_t)\s+(fi_\w+)\s*\(", text, re.M)) == set(kv4.EXPORTS)
