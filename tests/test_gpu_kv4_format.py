"""The append's words on the GPU: every one of them, and those of rotated rows against the fp64 row."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv4 as oracle_kv4
from oracle import step as oracle_step
from serving_attention_gb300 import kv4, step
from test_gpu_kv4 import DEV, DT, _f64, _gen, _i32, _randn
from test_kv4_format import all_words

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [1, 64])
def test_every_word(page):
    """Rows of the values that a word holds: the append gives the word and the codes back, read the values."""
    words, _, rows = all_words()
    x = torch.from_numpy(rows[:, None]).half().to(DEV)  # exact
    n = len(words)
    pages = -(-n // page)
    cache, slots = kv4.empty_cache(pages, page, 1, DEV), _i32(range(n))
    kv4.append(None, None, slots, None, None, x, x.flip(0), cache, page)
    k, v = torch.empty_like(x), torch.empty_like(x)
    kv4.read(slots, cache, page, k, v)
    assert torch.equal(k, x) and torch.equal(v, x.flip(0))
    k, v = (torch.empty_like(x, dtype=torch.bfloat16) for _ in range(2))
    kv4.read(slots, cache, page, k, v)
    assert torch.equal(k, x.bfloat16()) and torch.equal(v, x.flip(0).bfloat16())
    raw = cache.cpu().numpy()
    for i in range(n):
        at = oracle_kv4.places(page, i % page)[2:]
        got = [int(raw[i // page, 0, a]) + 256 * int(raw[i // page, 0, a + 1]) for a in at]
        assert got == [words[i], words[n - 1 - i]]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (16, True), (80, False)])
@pytest.mark.parametrize("norm", [False, True])
def test_rotated_rows(dtype, rot, interleaved, norm):
    """Scale, zero point and every value of a rotated row."""
    T, H, Hk, P, pages = 53, 2, 3, 16, 5
    r = step.rotary_setup(128, rot, interleaved, 500000.0, "yarn", 8.0, 8192)
    f, amp = oracle_step.rates(rot, 500000.0, "yarn", 8.0, 8192, 1.0, 32.0)
    pos = [0, 1, 131071, 1000003, 2**31 - 1, -5] + list(range(500, 500 + T - 6))
    qkv = _randn((T, H + 2 * Hk, 128), dtype, 70 + rot)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    k[::5] = k[::5].abs()  # rows of one sign, as far as the rotation leaves it
    w = 1 + 0.2 * torch.randn(128, generator=_gen(5), device=DEV) if norm else None
    cache = kv4.empty_cache(pages, P, Hk, DEV)
    slots = np.random.default_rng(rot).permutation(pages * P)[:T]
    kv4.append(r, _i32(pos), _i32(slots), q, torch.empty_like(q), k, v, cache, P, q_weight=w, k_weight=w)
    x = _f64(k)
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * _f64(w)
    ref = oracle_step.rotate(x, pos, f, amp, rot, interleaved)
    # an angle's fp32 rounding (up to pi 2^-24 = 2e-7), cosf and sinf (2 ulp), the norm's factor (2^-23) and the products'
    # roundings: below 1e-6 of a pair, whose values are below 4.5 in two dims
    size = 2 * amp * 4.5 * 1e-6
    raw = cache.cpu().numpy()
    for t in range(T):
        page, at = raw[slots[t] // P], oracle_kv4.places(P, int(slots[t]) % P)[2]
        for h in range(Hk):
            word = int(page[h, at]) + 256 * int(page[h, at + 1])
            got = oracle_kv4.get(raw, P, int(slots[t]), h)[0]
            assert oracle_kv4.row_faults(word, got, ref[t, h], size) == []


@pytest.mark.parametrize("rows", [1, 40])
def test_read_into_one_buffer(rows):
    """k and v rows side by side, heads inside or outside: apart, if one buffer."""
    page, heads = 16, 3
    cache = kv4.empty_cache(3, page, heads, DEV)
    x, y = _randn((3 * page, heads, 128), "bf16", 1), _randn((3 * page, heads, 128), "bf16", 2)
    kv4.append(None, None, _i32(range(3 * page)), None, None, x, y, cache, page)
    slots = _i32(range(5, 5 + rows))
    k, v = (torch.empty((rows, heads, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kv4.read(slots, cache, page, k, v)
    for shape, cut in (((rows, heads, 2, 128), lambda b, i: b[:, :, i]), ((rows, 2, heads, 128), lambda b, i: b[:, i]),
                       ((2, rows, heads, 128), lambda b, i: b[i])):
        buf = torch.full(shape, 9.0, dtype=torch.bfloat16, device=DEV)
        kv4.read(slots, cache, page, cut(buf, 0), cut(buf, 1))
        assert torch.equal(cut(buf, 0), k) and torch.equal(cut(buf, 1), v)
    with pytest.raises(RuntimeError):
        kv4.read(slots, cache, page, k, k)
