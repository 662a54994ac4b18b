"""Every word of the 4-bit format, what the check of quantised rows finds, and outputs that a read refuses (CPU)."""
from __future__ import annotations

import math

import numpy as np
import pytest

import serving_attention_gb300 as fi
from oracle import kv4 as oracle_kv4
from oracle.kv4 import row_faults
from serving_attention_gb300 import kv4


def all_words():
    """Words [N] of every scale above 0 with every zero point, and rows [N, 128] of the values that they hold: every code,
    the ends among them.  A row's values give its word back."""
    bits = np.arange(16, 0x6C01, 16)
    words = (bits[:, None] + np.arange(16)).reshape(-1).astype(np.uint16)
    rng = np.random.default_rng(1)
    codes = np.concatenate([np.arange(16), rng.integers(0, 16, 112)])
    return words, np.broadcast_to(codes, (len(words), 128)), oracle_kv4.values(codes, words)


def test_every_word_is_what_the_format_says():
    words, codes, rows = all_words()
    for i in range(0, len(words), 16):
        b = int(words[i]) & 0xFFF0
        s = math.ldexp(b & 0x3FF, -24) if b < 0x400 else math.ldexp(1024 + (b & 0x3FF), (b >> 10) - 25)
        assert s <= 4096
        for z in range(16):
            assert np.array_equal(rows[i + z], (codes[i + z] - float(z)) * s)
    assert rows.min() == -15 * 4096 and rows.max() == 15 * 4096
    assert np.array_equal(rows.astype(np.float16).astype(np.float64), rows)  # every value is an fp16
    assert (oracle_kv4.values(codes[:16], np.arange(16, dtype=np.uint16)) == 0).all()  # a scale of 0


def test_the_quantiser_gives_every_word_back():
    words, codes, rows = all_words()
    n, w = oracle_kv4.quantise(rows)
    assert np.array_equal(w, words) and np.array_equal(n, codes)


def test_scales_are_rounded_up():
    """A range a little above a word's takes the next one: past exponents' ends, not past 4096; 1 + 2^-9 of a normal scale is
    at least one fp16 step more."""
    words, _, rows = all_words()
    words, rows = words[::16], rows[::16]
    normal = words >= 0x400
    _, w = oracle_kv4.quantise(rows[normal] * (1 + 2.0**-9))
    assert np.array_equal(w & 0xFFF0, np.minimum(words[normal].astype(int) + 16, 0x6C00))


@pytest.mark.parametrize("seed", range(4))
def test_row_faults(seed):
    """Rows as quantised are as defined; a zero point of 0 or one off, a value off and a scale twice
    as large are not."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((50, 128)) * np.exp(rng.uniform(-4, 4, (50, 1)))
    n, w = oracle_kv4.quantise(x)
    got, sizes = oracle_kv4.values(n, w), 1e-6 * np.abs(x).max(-1)

    def coded(row, word):  # the row's codes beside another word, as clipped to 0 .. 15
        s = float(np.uint16(word & 0xFFF0).view(np.float16))
        return oracle_kv4.values(np.clip(np.rint(row / s) + (word & 15), 0, 15), np.uint16(word))

    for i in range(50):
        word, size = int(w[i]), sizes[i]
        assert row_faults(word, got[i], x[i], size) == []
        for other in (word & 0xFFF0, word + 1, word - 1):
            assert 0 < other & 15 < 15 or other == word & 0xFFF0
            assert "zero point" in row_faults(other, coded(x[i], other), x[i], size)
        assert "values" in row_faults(word & 0xFFF0, coded(x[i], word & 0xFFF0), x[i], size)
        assert row_faults(word, np.where(np.arange(128) == 7, got[i] + 1.01 * got[i].std(), got[i]), x[i], size) == ["values"]
        double = word + 0x400
        assert row_faults(double, coded(x[i], double), x[i], size)[0] == "scale"


@pytest.mark.parametrize("kw", [dict(v=64), dict(v=64 + 16), dict(v=64 + 256), dict(v=64 + 512 + 32), dict(v=64 - 512 * 3),
                                dict(v=64, vt=512, vh=128), dict(v=64 + 128, kt=256, kh=256, vt=256, vh=256, hk=1),
                                dict(v=64 + 16, n=1)])
def test_read_refuses_outputs_that_meet(kw):
    """Before any launch: the pointers are fake."""
    a = dict(slots=32, n=4, k=64, kt=256, kh=128, v=1 << 20, vt=256, vh=128, hk=2, cache=128, cp=4224, ch=2112, page=16,
             pages=10, dt=fi.BF16)
    a.update(kw)
    assert kv4.load().fi_kv4_read(kv4._READ_ARGS.pack(*a.values()), None) == 1
