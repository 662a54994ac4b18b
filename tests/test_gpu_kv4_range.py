"""Attention over the 4-bit cache where weights and values span many powers of two.

Tolerances, with S = sum_j p_j |v_j|, P = sum_j p_j max_d |v_jd| (a quantised row holds a value of 7 s or more, for its
range is at least 14 s: 15 sum_j p_j s_j <= 15 / 7 P) and n keys:

* the weights' one rounding to fp16 is off by at most 2^-11 of each, fp32 logits, exponentials and sums by 1e-4 of S;
* decode sums weights times codes and weights times zero points apart, 16 keys a product.  A product keeps its addends, up
  to 16 and what is summed so far, down to 2^-25 of the largest's power of two, an operand below 2^-14 counting as that
  (so measured on a GB300).  Codes come in as n 2^-21 at the least: an addend loses at most 2^-14 2^-25 w, which is 2^-18
  of a code's unit, or 2^-22 of a zero point's (n 2^-17); for all products (min(n, 16) + 1) (2^-18 + 2^-22) sum_j p_j s_j
  = (min(n, 16) + 1) 17 / 16 2^-18 / 7 P at most.  Beside the sum so far, at most 15 sum_j p_j s_j, each of the at most
  2 ceil(n / 128) products of a warp loses 17 2^-25 of it, twice (codes and zero points): 17 2^-24 15 / 7 P.

|o - ref| <= (2^-11 + 1e-4) S + half a step of the output,
for decode + ((min(n, 16) + 1) 17 / 16 2^-18 / 7 + 2 ceil(n / 128) 17 2^-24 15 / 7) P."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_attention_gb300 as fi
from oracle import kv4 as oracle_kv4
from serving_attention_gb300 import kv4
from test_gpu_kv4 import DEV, DT, Batch, _config, _f64, _gen, _i32, _randn

pytestmark = pytest.mark.gpu


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
    tol = (2.0**-11 + 1e-4) * size + np.where(decode, sums, 0) * most
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
