"""The append with head norms on the GPU against the fp64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import step as oracle_step
from serving_attention_gb300 import step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=_gen(seed), device=DEV).to(DT[dtype])


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,rot,v_dim", [(128, 128, 128), (64, 64, 64), (80, 32, 80), (256, 256, 256), (96, 16, 96),
                                           (256, 16, 0), (16, 16, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weights", ["both", "per_head", "q", "none"])
def test_norm_append(dtype, dim, rot, v_dim, interleaved, weights):
    T, H, Hk, P, pages = 29, 6, 3, 8, 6
    r = step.rotary_setup(dim, rot, interleaved, 500000.0, "yarn", 8.0, 8192)
    f, amp = oracle_step.rates(rot, 500000.0, "yarn", 8.0, 8192, 1.0, 32.0)
    pos = [0, 1, 131071, 1000003, 2**31 - 1, -5] + list(range(100, 100 + T - 6))
    slots = np.random.default_rng(dim).permutation(pages * P)[:T]
    slots[3], slots[8] = -1, pages * P
    wide = _randn((T, H + Hk, dim + 8), dtype, dim + rot)
    wide[4] *= 0.001
    wide[5] = 0
    q, k = wide[:, :H, :dim], wide[:, H:, 8:]
    v = _randn((T, Hk, v_dim), dtype, 9) if v_dim else None
    shape = {"per_head": (H + Hk, dim)}.get(weights, (dim,))
    w = 1 + 0.2 * torch.randn(shape, generator=_gen(4), device=DEV)
    qw = None if weights == "none" else w[:H] if weights == "per_head" else w
    kw = w[H:] if weights == "per_head" else w if weights == "both" else None
    k_cache = torch.full((pages, P, Hk + 1, dim), 7.0, dtype=DT[dtype], device=DEV)
    v_cache = torch.full((pages, P, Hk, v_dim), 7.0, dtype=DT[dtype], device=DEV) if v_dim else None
    q_out = torch.empty_like(q)
    step.norm_append(r, _i32(pos), _i32(slots), q, q_out, qw, k, kw, v, k_cache[:, :, :Hk], v_cache, eps=1e-5)
    half, tiny = torch.finfo(DT[dtype]).eps / 2, torch.finfo(DT[dtype]).smallest_normal * torch.finfo(DT[dtype]).eps

    def check(got, x, weight, rows):
        x = _f64(x)
        if weight is not None:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5) * _f64(weight)
        ref = oracle_step.rotate(x, pos, f, amp, rot, interleaved)
        # the rotation's 1e-6 of a pair (see test_gpu_step) and the norm's factor: a sum of at most 256 squares, its
        # root and two products, 1e-6 of the value again at most (in most orders a tenth of that)
        tol = 2e-6 * amp * 2 * np.abs(x).max(-1, keepdims=True) + half * np.abs(ref) * (1 + 1e-6) + tiny
        assert (np.abs(_f64(got) - ref)[rows] <= tol[rows]).all()

    check(q_out, q, qw, np.arange(T))
    ok = (slots >= 0) & (slots < pages * P)
    at = np.where(ok, slots, 0)
    check(k_cache[:, :, :Hk].flatten(0, 1)[torch.as_tensor(at, device=DEV)], k, kw, np.flatnonzero(ok))
    if v_dim:
        assert torch.equal(v_cache.flatten(0, 1)[torch.as_tensor(slots[ok], device=DEV)],
                           v[torch.as_tensor(np.flatnonzero(ok), device=DEV)])
    untouched = np.setdiff1d(np.arange(pages * P), slots)
    assert (k_cache.flatten(0, 1)[torch.as_tensor(untouched, device=DEV)] == 7).all() and (k_cache[:, :, Hk] == 7).all()


def test_norm_append_without_weights_is_append():
    r = step.rotary_setup(128, theta=1e6)
    qkv = _randn((600, 16, 128), "bf16", 3)
    q, k, v = qkv[:, :8], qkv[:, 8:12], qkv[:, 12:]
    pos = torch.arange(600, device=DEV).int()
    got = []
    for norm in (False, True):
        q_out, kc, vc = torch.empty_like(q), *torch.zeros((2, 40, 16, 4, 128), dtype=torch.bfloat16, device=DEV)
        if norm:
            step.norm_append(r, pos, pos, q, q_out, None, k, None, v, kc, vc)
        else:
            step.append(r, pos, pos, q, q_out, k, v, kc, vc)
        got.append((q_out, kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("dim,v_dim", [(128, 128), (80, 80), (64, 128), (256, 256)])
def test_norm_append_in_place_captured_and_in_parts(dim, v_dim):
    """One call of many tokens, in place and replayed from a graph, does what small calls do, to the bit; v is copied
    whatever its bits."""
    T, H, Hk, P = 5001, 5, 3, 16
    r = step.rotary_setup(dim, theta=1e6)
    q, k, v = _randn((T, H, dim), "bf16", 1), _randn((T, Hk, dim), "bf16", 2), _randn((T, Hk, v_dim), "bf16", 3)
    v.view(torch.int16).copy_(torch.randint(-2**15, 2**15, v.shape, generator=_gen(4), device=DEV).short())
    w = [1 + 0.2 * torch.randn((n, dim), generator=_gen(5), device=DEV) for n in (H, Hk)]
    pos = torch.arange(T, device=DEV).int()
    slots = torch.randperm(-(-T // P) * P, generator=_gen(6), device=DEV)[:T].int()
    small = [torch.empty_like(q), *(torch.zeros((-(-T // P), P, Hk, d), dtype=q.dtype, device=DEV) for d in (dim, v_dim))]
    for a in range(0, T, 61):
        b = min(T, a + 61)
        step.norm_append(r, pos[a:b], slots[a:b], q[a:b], small[0][a:b], w[0], k[a:b], w[1], v[a:b], *small[1:])
    turned, caches = q.clone(), [torch.zeros_like(x) for x in small[1:]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.norm_append(r, pos, slots, turned, turned, w[0], k, w[1], v, *caches)
    for _ in range(2):
        turned.copy_(q)
        graph.replay()
    for x, y in zip((turned, *caches), small):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
