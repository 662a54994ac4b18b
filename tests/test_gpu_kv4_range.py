"""Attention over the 4-bit cache where weights and values span many powers of two.

Tolerances, with S = sum_j p_j |v_j|, P = sum_j p_j max_d |v_jd| (a quantised row holds a value of 7 s or more, for its
range is at least 14 s: 15 sum_j p_j s_j <= 15 / 7 P) and n keys:

* a weight (decode: p_j s_j; prompts: p_j) is rounded to fp16 once, in a unit that keeps the row's largest so far at 2^11
  or more: off by at most 2^-11 of itself, or, below 2^-14, by 2^-25 of the unit, 2^-36 of the largest: n 2^-36 15 / 7 P
  (decode), n 2^-36 max |v| (prompts);
* fp32 logits, exponentials and sums are off by less than 1e-4 of S;
* decode sums weights times codes and weights times zero points apart, 16 keys a product.  A product keeps its addends, up
  to 16 and what is summed so far, down to 2^-25 of the largest's power of two, an operand below 2^-14 counting as that
  (so measured on a GB300).  Codes come in as n 2^-21 at the least: an addend loses at most 2^-14 2^-25 w, which is 2^-18
  of a code's unit, or 2^-22 of a zero point's (n 2^-17); for all products (min(n, 16) + 1) (2^-18 + 2^-22) sum_j p_j s_j
  = (min(n, 16) + 1) 17 / 16 2^-18 / 7 P at most.  Beside the sum so far, at most 15 sum_j p_j s_j, each of the at most
  2 ceil(n / 128) products of a warp loses 17 2^-25 of it, twice (codes and zero points): 17 2^-24 15 / 7 P.

|o - ref| <= (2^-11 + 1e-4) S + half a step of the output + n 2^-36 max |v| (prompts)
or + (n 2^-36 15 / 7 + (min(n, 16) + 1) 17 / 16 2^-18 / 7 + 2 ceil(n / 128) 17 2^-24 15 / 7) P (decode)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_attention_gb300 as fi
from oracle import kv4 as oracle_kv4
from serving_attention_gb300 import kv4
from test_gpu_kv4 import DEV, DT, Batch, _config, _f64, _gen, _i32, _randn

pytestmark = pytest.mark.gpu
SPLIT = dict(prefill_min_chunk=128, decode_min_chunk=64, split_factor=8)


def _filled(b, kv, k, v):
    """The batch with rows k, v [sum kv, Hkv, 128] in its cache, request by request."""
    slots = [int(b.ids[b.kvp[r] + j // b.page]) * b.page + j % b.page for r, n in enumerate(kv) for j in range(n)]
    kv4.append(None, None, _i32(slots), None, None, k, v, b.cache, b.page)
    return b


def _check(b, cfg, window=-1, sink=0):
    o, lse, info, ws = b.run(cfg)
    assert fi.device_status(ws) == 0
    t = int(b.qo[-1])
    k, v = (np.nan_to_num(x, posinf=0, neginf=0) for x in oracle_kv4.all_values(b.cache.cpu().numpy(), b.page))
    ref = lambda x: oracle_kv4.attention(b.qo, b.kvp, b.ids, b.last, b.page, b.causal, b.scale, _f64(b.q), k, x,  # noqa: E731
                                         window, sink, b.pool)
    ro, rl, size = (x[:t] for x in ref(v))
    most = ref(np.broadcast_to(np.abs(v).max(-1, keepdims=True), v.shape))[2][:t]
    og, lg = _f64(o[:t]), _f64(lse[:t])
    assert np.isfinite(og).all()
    lens = (np.diff(b.kvp) - 1) * b.page + b.last
    rows = np.diff(b.qo) * (b.hq // b.hkv)
    n, decode = (np.repeat(x, np.diff(b.qo))[:, None, None] for x in (lens, rows <= 16))
    half = torch.finfo(o.dtype).eps / 2
    sums = (np.minimum(n, 16) + 1) * 17 / 16 * 2.0**-18 / 7 + 2 * np.ceil(n / 128) * 17 * 2.0**-24 * 15 / 7
    held = np.abs(v[b.ids]).max()
    tol = (2.0**-11 + 1e-4) * size + np.where(decode, (n * 2.0**-36 * 15 / 7 + sums) * most, n * 2.0**-36 * held)
    tol = tol * (1 + half) + half * np.abs(ro) + torch.finfo(o.dtype).smallest_normal * 2 * half
    worst = float((np.abs(og - ro) / tol).max())
    assert worst <= 1, f"{worst:.2f} times the tolerance"
    seen = ~np.isneginf(rl)
    assert np.array_equal(~np.isneginf(lg), seen) and np.abs(lg[seen] - rl[seen]).max(initial=0) <= 2e-4


# ------------------------------------------------------ values held as zero

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ratio", [2.0**8, 2.0**10, 2.0**13])
@pytest.mark.parametrize("page", [1, 16])
def test_dims_that_a_large_value_row_holds_as_zero(dtype, ratio, page):
    """One key with eight dims of up to `ratio` times the ordinary and the others 0, beside some of ordinary values."""
    kv, hkv = [16, 12, 16, 14, 9, 16], 2
    b = Batch(90, [1] * len(kv), kv, 4 * hkv, hkv, page, dtype, 0)
    n = sum(kv)
    v = torch.randn(n, hkv, 128, generator=_gen(91), device=DEV)
    for at in np.cumsum([0] + kv[:-1]):
        v[at, :, 3::16] *= ratio
        v[at].masked_fill_((torch.arange(128, device=DEV) % 16 != 3), 0)
    _check(_filled(b, kv, 0.5 * _randn((n, hkv, 128), dtype, 92), v.to(DT[dtype])), _config())


# ------------------------------------------------ value scales far apart (decode)

@pytest.mark.parametrize("dtype,std,large", [("fp16", 1.0, 61440.0), ("bf16", 2.0**-5, 61440.0), ("bf16", 2.0**-12, 61440.0),
                                             ("bf16", 2.0**-12, 1.0), ("fp16", 2.0**-3, 4096.0)])
@pytest.mark.parametrize("qo,page,split", [(1, 16, False), (4, 16, False), (1, 1, False), (4, 64, True)])
def test_a_large_value_of_no_weight(dtype, std, large, qo, page, split):
    """Logits of deviation 3 and one key some 60 below them, whose values are up to 2^28 times the others'."""
    n, hkv, g = 4096, 2, 4
    for at in (5, n // 2, n - 3):
        b = Batch(100 + at, [qo], [n], hkv * g, hkv, page, dtype, 0)
        base = _randn((hkv, 128), "fp16", 7).float()
        b.q.copy_((base.repeat_interleave(g, 0) + 0.05 * torch.randn(b.q.shape, generator=_gen(8), device=DEV)).to(b.q.dtype))
        k = 3 * torch.randn(n, hkv, 128, generator=_gen(9), device=DEV)
        k[at] = -60 / (b.scale * base.square().sum(-1, keepdim=True)) * base
        v = std * torch.randn(n, hkv, 128, generator=_gen(10), device=DEV)
        v[at] = large * torch.where(torch.arange(128, device=DEV) % 2 == 0, 1.0, -1.0) * 0.5
        _check(_filled(b, [n], k.to(DT[dtype]), v.to(DT[dtype])), _config(**(SPLIT if split else {})))


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("window,sink", [(-1, 0), (700, 5)])
@pytest.mark.parametrize("first,last", [(-10, 8), (8, -10)])
def test_values_that_grow_along_a_request(first, last, window, sink, split):
    """Every stage of a warp brings values of another size, so its unit moves under what it holds."""
    kv, hkv, g = [3000, 900, 64], 2, 4
    b = Batch(120, [4, 1, 2], kv, hkv * g, hkv, 16, "bf16", 1)
    k = torch.cat([_randn((n, hkv, 128), "bf16", 121 + n) for n in kv])
    v = torch.cat([torch.randn(n, hkv, 128, generator=_gen(n), device=DEV) *
                   torch.exp2(torch.linspace(first, last, n, device=DEV))[:, None, None] for n in kv]).to(torch.bfloat16)
    _check(_filled(b, kv, k, v), _config(window_left=window, sink_tokens=sink, **(SPLIT if split else {})), window, sink)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("qo,split", [(1, False), (4, True), (40, False)])
@pytest.mark.parametrize("logits", [(-30, 30), (30, -30), (-3, 3)])
@pytest.mark.parametrize("sizes", [(-9, 9), (9, -9)])
def test_logits_and_values_that_grow_along_a_request(dtype, qo, split, logits, sizes):
    """Maximum and unit move together or against each other, in nearly every stage."""
    n, hkv, g = 2000, 2, 4
    b = Batch(125, [qo], [n], hkv * g, hkv, 16, dtype, 0)
    base = _randn((hkv, 128), "fp16", 126).float()
    b.q.copy_((base.repeat_interleave(g, 0) + 0.05 * torch.randn(b.q.shape, generator=_gen(127), device=DEV)).to(b.q.dtype))
    k = torch.linspace(*logits, n, device=DEV)[:, None, None] / (b.scale * base.square().sum(-1, keepdim=True)) * base
    v = torch.randn(n, hkv, 128, generator=_gen(128), device=DEV) * torch.exp2(torch.linspace(*sizes, n, device=DEV))[:, None, None]
    _check(_filled(b, [n], k.to(DT[dtype]), v.to(DT[dtype])), _config(**(SPLIT if split else {})))


@pytest.mark.parametrize("split", [False, True])
def test_large_values_that_some_rows_do_not_see(split):
    """One query head a key head and 16 tokens, keys of equal weight: one of the last has values of 2^24 times the
    others', which are all alike, and is hidden from all rows but the last five of a pass."""
    kv, hkv = [1200, 40], 4
    b = Batch(130, [16, 16], kv, hkv, hkv, 16, "fp16", 1)
    v = (2.0**-9 * (1 + torch.arange(hkv, device=DEV)[:, None] * 0.3) *
         (1 + torch.rand(128, generator=_gen(131), device=DEV))).expand(sum(kv), hkv, 128).half().clone()
    for end in (1200, 1240):
        v[end - 5] = (v[end - 5].float() * 2.0**24).clamp(max=61440.0).half()
    k = torch.zeros_like(v)
    _check(_filled(b, kv, k, v), _config(**(SPLIT if split else {})))


# ------------------------------------------- a few keys far above a flat tail

@pytest.mark.parametrize("qo", [1, 4, 40])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nats", [6, 12, 13.9, 15, 16, 16.5])
def test_keys_far_below_others_without_values(qo, dtype, nats):
    """Every 64th key is `nats` above all others and has no values: the output is that of the others."""
    n, hkv, g = 3000, 2, 4
    b = Batch(140, [qo], [n], hkv * g, hkv, 16, dtype, 0)
    base = torch.where(torch.rand(hkv, 128, generator=_gen(3), device=DEV) < 0.5, -1.0, 1.0)
    b.q.copy_(base.repeat_interleave(g, 0).expand(b.q.shape))
    k, v = torch.zeros(n, hkv, 128, device=DEV), 2048 * (1 + torch.rand(n, hkv, 128, generator=_gen(4), device=DEV))
    k[5::64], v[5::64] = nats / (b.scale * 128) * base, 0
    _check(_filled(b, [n], k.to(DT[dtype]), v.to(DT[dtype])), _config())


# --------------------------------------------------- small factors of the logits

@pytest.mark.parametrize("qo", [4, 40])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [1e-9, 1e-12, 1e-20, 2.0**-124])
def test_small_scales_and_rows_of_zeros(qo, dtype, scale):
    """A row's factor, the scale times its power of two, stays above 0: what a mask hides stays hidden."""
    b = Batch(150, [qo, 2], [300, 40], 8, 2, 16, dtype, 1, scale=scale)
    b.q[::2] = 0
    b.q[1::4] *= 2.0**-20
    if dtype == "bf16":
        b.q[3::4] *= 2.0**-110
    _check(b, _config())
