"""Refusals of the append with head norms (CPU)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import serving_attention_gb300 as fi
from serving_attention_gb300 import step

_ROT = step.rotary_setup(128)


def _norm_append(**kw):
    a = dict(rot=ctypes.addressof(_ROT), pos=16, slots=32, n=4, q=48, qt=1024, qh=128, qo=1 << 20, qot=1024, qoh=128,
             hq=8, k=64, kt=256, kh=128, v=80, vt=256, vh=128, v_dim=128, hk=2, kc=96, k0=4096, k1=256, k2=128, vc=112,
             v0=4096, v1=256, v2=128, page=16, pages=10, dt=fi.BF16, qw=96, qws=0, kw=112, kws=0, eps=1e-6)
    a.update(kw)
    return step.load().fi_norm_rotary_append(step._NORM_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), 1), (dict(pos=0), 1), (dict(k=0), 1), (dict(kc=0), 1), (dict(hk=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("inf")), 1), (dict(qw=98), 4), (dict(qws=2), 1), (dict(kws=126), 1), (dict(kws=131), 4),
    (dict(kws=-4), 1), (dict(dt=fi.FP32), 2), (dict(page=3), 2), (dict(v_dim=1024), 2), (dict(k0=8), 1),
    (dict(qoh=64), 1), (dict(kt=4), 4)])
def test_norm_append_refusals(kw, status):
    assert _norm_append(**kw) == status


def test_norm_append_without_tokens_needs_no_pointers():
    assert _norm_append(n=0, pos=0, slots=0, q=0, qo=0, k=0, v=0, kc=0, vc=0, qw=0, kw=0) == 0
    assert step.load().fi_norm_rotary_append(None, None) == 1


def test_binding_refuses_wrong_weights():
    q, idx = torch.zeros(3, 2, 128).half(), torch.zeros(3, dtype=torch.int32)
    k, cache = q[:, :1], torch.zeros(2, 16, 1, 128).half()
    with pytest.raises(TypeError):
        step.norm_append(_ROT, idx, idx, q, q.clone(), None, k, torch.ones(128).double(), k, cache, cache)
    with pytest.raises(ValueError):
        step.norm_append(_ROT, idx, idx, q, q.clone(), torch.ones(64), k, None, k, cache, cache)
    with pytest.raises(ValueError):
        step.norm_append(_ROT, idx, idx, q, q.clone(), torch.ones(3, 128), k, None, k, cache, cache)
    with pytest.raises(TypeError):  # not on a GPU
        step.norm_append(_ROT, idx, idx, q, q.clone(), torch.ones(2, 128), k, None, k, cache, cache)
