"""The step operators on the GPU against their fp64 oracle.

Rotary tolerance: the angle is exact to 2^-32 of a turn and sincospi to 2^-22
relative of its result or better; product sums in fp32 add 2 * 2^-24; so 1e-6
times amplitude * (|a| + |b|), and half a step of the output type."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import serving_attention_gb300 as fi
from oracle import diff as oracle_diff
from oracle import step as oracle_step
from serving_attention_gb300 import differential, step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=_gen(seed), device=DEV).to(DT[dtype])


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _near(got, ref, x, dtype, amp):
    half = torch.finfo(DT[dtype]).eps / 2
    tiny = torch.finfo(DT[dtype]).smallest_normal * half * 2  # half a subnormal step
    tol = 1e-6 * amp * 2 * np.abs(x).max() + half * np.abs(ref) * (1 + 1e-6) + tiny
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 64), (80, 32), (256, 256), (96, 16), (128, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_rotate(dtype, dim, rot, interleaved, scaling):
    T = 37
    r = step.rotary_setup(dim, rot, interleaved, 500000.0, scaling, 8.0 if scaling == "yarn" else 1.0, 8192)
    f, amp = oracle_step.rates(rot, 500000.0, scaling, 8.0, 8192, 1.0, 32.0)
    pos = [0, 1, 2, 131071, 1000003, 2**31 - 1, -5] + list(range(100, 100 + T - 7))
    wide = _randn((T, 9, dim + 8), dtype, dim + rot)  # rows inside wider ones
    q, k = wide[:, :6, :dim], wide[:, 6:, 8:]
    q_out, k_out = torch.empty_like(q), torch.full((T, 5, dim), 7.0, dtype=DT[dtype], device=DEV)
    step.rotate(r, _i32(pos), q, q_out, k, k_out[:, 1:4])
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    for got, x in ((q_out, q), (k_out[:, 1:4], k)):
        x = f64(x)
        ref = oracle_step.rotate(x, pos, f, amp, rot, interleaved)
        # fp64 angles of the last positions are off by 2^31 * 2^-53 relative: far below the bound
        _near(got, ref, x, dtype, amp)
        assert np.array_equal(f64(got)[..., rot:], x[..., rot:])
    assert (k_out[:, 0] == 7).all() and (k_out[:, 4] == 7).all()
    step.rotate(r, _i32(pos), q, q)  # in place, q alone
    assert torch.equal(q, q_out)


def test_rotate_beside_its_input():
    """Outputs in the memory of their inputs, rows apart: columns behind or before the input's, rows behind all
    of them, heads between the input's, one token or head with any stride; heads the outer dimension."""
    r = step.rotary_setup(64)
    T, H = 9, 3
    pos = torch.arange(T, device=DEV).int()
    wide, tall = _randn((T, 2 * H, 64), "bf16", 1), _randn((2 * T, H, 64), "bf16", 2)
    outer = _randn((2 * H, T, 64), "bf16", 3).transpose(0, 1)
    one = _randn((1, 4, 72), "bf16", 4)[:, :, :64]
    for x, y in ((wide[:, :H], wide[:, H:]), (wide[:, H:], wide[:, :H]), (tall[:T], tall[T:]), (tall[T:], tall[:T]),
                 (wide[:, ::2], wide[:, 1::2]), (wide[:, 1::2], wide[:, ::2]), (outer[:, :H], outer[:, H:]),
                 (outer[:, 1::2], outer[:, ::2]), (wide[:, 1:2], wide[:, 5:6]), (wide[3:4], wide[2:3])):
        want, p = torch.empty_like(x), pos[:x.shape[0]]
        step.rotate(r, p, x, want)
        step.rotate(r, p, x, y)
        assert torch.equal(y, want)
    want = torch.empty((1, 4, 64), dtype=torch.bfloat16, device=DEV)
    step.rotate(r, pos[:1], one, want)
    step.rotate(r, pos[:1], one, one.as_strided(one.shape, (8, 72, 1)))  # in place; one token has no token stride
    assert torch.equal(one, want)
    for x, y in ((wide[:, :H], wide[:, 1:1 + H]), (tall[:T], tall[2:2 + T]), (tall[5:5 + T], tall[:T])):
        with pytest.raises(fi.FIError):
            step.rotate(r, pos, x, y)


@pytest.mark.parametrize("tokens", [1, 63, 700, 9001])
def test_rotate_token_counts(tokens):
    r = step.rotary_setup(128)
    q = _randn((tokens, 4, 128), "bf16", tokens)
    pos = torch.randint(0, 100000, (tokens,), generator=_gen(1), device=DEV).int()
    out = torch.empty_like(q)
    step.rotate(r, pos, q, out)
    f, _ = oracle_step.rates(128, 10000.0)
    at = [0, tokens // 2, tokens - 1]
    x = q[at].double().cpu().numpy()
    _near(out[at], oracle_step.rotate(x, pos[at].tolist(), f, 1.0, 128, False), x, "bf16", 1.0)
    # every token on its own gives the same bits
    one = torch.empty_like(q[:1])
    for t in at:
        step.rotate(r, pos[t:t + 1].contiguous(), q[t:t + 1], one)
        assert torch.equal(one[0], out[t])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hk,dim,v_dim,page", [(8, 2, 128, 128, 16), (16, 1, 64, 512, 64), (3, 3, 80, 80, 1),
                                                  (0, 4, 96, 0, 8)])
def test_append(dtype, hq, hk, dim, v_dim, page):
    T, pages = 45, 60
    r = step.rotary_setup(dim, 32, True)
    q, k = _randn((T, hq, dim), dtype, 1) if hq else None, _randn((T, hk, dim), dtype, 2)
    v = _randn((T, hk, v_dim), dtype, 3) if v_dim else None
    kc = _randn((pages, page, hk + 1, dim), dtype, 4)[:, :, 1:]  # a padding head
    vc = _randn((pages, hk, page, v_dim), dtype, 5).transpose(1, 2) if v_dim else None
    k0, v0 = kc.clone(), vc.clone() if v_dim else None
    slots = torch.randperm(pages * page, generator=_gen(6), device=DEV)[:T].int()
    skip = {3: -1, 20: pages * page, 44: 2**31 - 1, 7: -2**31}
    for t, s in skip.items():
        slots[t] = s
    pos = torch.arange(T, device=DEV).int() * 997
    q_out = torch.empty_like(q) if hq else None
    step.append(r, pos, slots, q, q_out, k, v, kc, vc)
    f, amp = oracle_step.rates(32, 10000.0)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    if hq:
        _near(q_out, oracle_step.rotate(f64(q), pos.tolist(), f, amp, 32, True), f64(q), dtype, amp)
    ref = oracle_step.rotate(f64(k), pos.tolist(), f, amp, 32, True)
    written = torch.zeros(pages, page, dtype=torch.bool, device=DEV)
    for t in range(T):
        if t in skip:
            continue
        s = int(slots[t])
        at = (s // page, s % page)
        written[at] = True
        _near(kc[at], ref[t], f64(k), dtype, amp)
        if v_dim:
            assert torch.equal(vc[at], v[t])
    assert torch.equal(kc[~written], k0[~written])
    if v_dim:
        assert torch.equal(vc[~written], v0[~written])


def test_append_far_into_a_large_cache():
    """Element offsets past 2^31."""
    pages = 70000
    kc = torch.empty((pages, 128, 2, 128), dtype=torch.bfloat16, device=DEV)  # 4.6 GB: offsets to 2.3e9
    r = step.rotary_setup(128)
    k = _randn((2, 2, 128), "bf16", 1)
    slots = _i32([pages * 128 - 1, 66000 * 128 + 5])
    kc[-1, -1] = 0
    step.append(r, _i32([0, 0]), slots, None, None, k, None, kc, None)
    assert torch.equal(kc[-1, -1], k[0]) and torch.equal(kc[66000, 5], k[1])


def _lengths(seed, batch, kv_max, chunk):
    rng = np.random.default_rng(seed)
    kv = rng.integers(0, kv_max, size=batch)
    kv[rng.random(batch) < 0.1] = 0
    q = np.minimum(kv, np.where(rng.random(batch) < 0.3, rng.integers(0, chunk, size=batch), 1))
    return q.tolist(), kv.tolist()


def _table_case(seed, batch, kv_max, chunk, page):
    q, kv = _lengths(seed, batch, kv_max, chunk)
    rng = np.random.default_rng(seed + 1)
    width = max(1, -(-kv_max // page))
    ids = rng.permutation(batch * width + 9000)
    return q, kv, ids[:batch * width].reshape(batch, width).tolist(), ids[batch * width:].tolist()


@pytest.mark.parametrize("batch,kv_max,chunk", [(1, 5, 2), (3, 40, 9), (64, 3000, 2), (511, 200, 4), (513, 333, 30),
                                                (4097, 100, 3), (8192, 20, 2)])
@pytest.mark.parametrize("page", [1, 16, 128])
def test_tables(batch, kv_max, chunk, page):
    q, kv, table, free = _table_case(batch + page, batch, kv_max, chunk, page)
    head, tokens, pages = 13, sum(q) + 5, sum(-(-x // page) for x in kv) + 3
    ref = oracle_step.tables(q, kv, table, page, free, head, pages, tokens)
    wide = torch.full((batch, len(table[0]) + 4), -7, dtype=torch.int32, device=DEV)
    bt = wide[:, :len(table[0])]
    bt.copy_(_i32(table))
    t = step.StepTables(batch, pages, tokens, DEV)
    h = _i32([head])
    for _ in range(2):  # the same call again gives the same
        step.build_tables(t, _i32(q), _i32(kv), bt, page, _i32(free), h)
        assert t.counts.tolist() == ref["counts"] and int(h) == head
        for name in ("qo_indptr", "kv_indptr", "last_page_len", "positions", "slots"):
            assert getattr(t, name).tolist() == ref[name], name
        n = len(ref["kv_indices"])
        assert t.kv_indices[:n].tolist() == ref["kv_indices"] and (t.kv_indices[n:] == -1).all()
        assert bt.tolist() == ref["table"] and (wide[:, len(table[0]):] == -7).all()


@pytest.mark.parametrize("what", ["query over keys", "negative", "too long", "pages", "tokens", "free", "head"])
def test_tables_refuse_on_the_device(what):
    q, kv, page, head, free = [1, 4, 1], [33, 4, 16], 16, 2, list(range(100, 106))
    pages, tokens, status = 5, 6, 3
    if what == "query over keys":
        q[1], status = 5, 1
    elif what == "negative":
        q[2], status = -1, 1
    elif what == "too long":
        kv[0], status = 5 * 16 + 1, 1
    elif what == "pages":
        pages = 4
    elif what == "tokens":
        tokens = 5
    elif what == "free":
        free = free[:3]
    else:
        head = -1
    table = [[1, 2, 3, 4, 5], [6, 7, 8, 9, 10], [11, 12, 13, 14, 15]]
    assert oracle_step.tables(q, kv, table, page, free, head, pages, tokens) == status
    t = step.StepTables(3, pages, tokens, DEV)
    before = [x.clone() for x in (t.qo_indptr, t.kv_indptr, t.last_page_len, t.kv_indices, t.positions, t.slots)]
    bt = _i32(table)
    step.build_tables(t, _i32(q), _i32(kv), bt, page, _i32(free), _i32([head]))
    assert int(t.counts[4]) == status and int(t.counts[3]) == head
    assert bt.tolist() == table
    for a, b in zip(before, (t.qo_indptr, t.kv_indptr, t.last_page_len, t.kv_indices, t.positions, t.slots)):
        assert torch.equal(a, b)


def test_tables_of_batches_around_the_shared_memory_opt_in():
    """Lengths that fill the 48 KB of a launch without an opt-in but for the kernel's static arrays (3624 to
    3640 requests).  In a process of its own: a larger batch before would opt in for all."""
    code = ("import torch\nfrom serving_attention_gb300 import step\n"
            "for n in range(3560, 3660, 4):\n"
            "    t, one = step.StepTables(n, n, n), torch.ones(n, dtype=torch.int32, device='cuda')\n"
            "    ids = torch.arange(n, device='cuda').int()\n"
            "    step.build_tables(t, one, 2 * one, ids[:, None], 16)\n"
            "    assert t.counts.tolist() == [n, n, 0, 0, 0, 0, 0, 0] and t.slots.equal(16 * ids + 1)\n")
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr


@pytest.mark.parametrize("what", ["free", "tokens", "lengths"])
def test_refused_tables_append_nothing(what):
    """A step whose tables are refused behind one that was not: the append of the same captured
    step leaves the cache, which holds the earlier step's keys at its slots, as it is."""
    t = step.StepTables(3, 9, 600, DEV)
    bt, free, head = _i32([[b] + 39 * [-1] for b in (1, 2, 3)]), _i32([4, 5]), _i32([0])
    ql, kl = _i32([1, 2, 3]), _i32([10, 11, 12])
    k = _randn((600, 2, 64), "bf16", 1)
    kc, vc = (torch.zeros((8, 16, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    r = step.rotary_setup(64)

    def device_step():
        step.build_tables(t, ql, kl, bt, 16, free, head)
        step.append(r, t.positions, t.slots, None, None, k, k, kc, vc)

    device_step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        device_step()
    assert int(t.counts[4]) == 0 and int((t.slots >= 0).sum()) == 6
    before = [x.clone() for x in (kc, vc, bt, t.qo_indptr, t.kv_indptr, t.last_page_len, t.kv_indices)]
    k.copy_(_randn((600, 2, 64), "bf16", 2))
    if what == "free":
        kl.copy_(_i32([17, 18, 19]))  # three pages of two
    elif what == "tokens":
        ql.copy_(_i32([1, 2, 598]))
        kl.copy_(_i32([10, 11, 600]))
    else:
        kl.copy_(_i32([10, 1, 12]))
    graph.replay()
    assert int(t.counts[4]) != 0 and int(t.counts[3]) == 0
    assert (t.slots == -1).all() and (t.positions == 0).all()
    for a, b in zip(before, (kc, vc, bt, t.qo_indptr, t.kv_indptr, t.last_page_len, t.kv_indices)):
        assert torch.equal(a, b)


def test_tables_without_a_free_list():
    t = step.StepTables(2, 4, 2, DEV)
    step.build_tables(t, _i32([1, 1]), _i32([18, 5]), _i32([[3, 4], [5, 6]]), 16)
    assert t.counts.tolist() == [2, 3, 0, 0, 0, 0, 0, 0] and t.slots.tolist() == [4 * 16 + 1, 5 * 16 + 4]
    step.build_tables(t, _i32([1, 1]), _i32([17, 5]), _i32([[3, 4], [5, 6]]), 16)  # needs a page
    assert int(t.counts[4]) == 3


def test_steps_of_a_batch_captured_and_replayed():
    """Tables, rotary append and differential attention as one step, the device
    part captured once and replayed over growing requests, padded to a fixed
    number of tokens; against the oracle of the whole sequence at each step."""
    P, Hq, Hk, B, cap_tok, width = 16, 8, 2, 3, 40, 12
    lens, steps = [30, 0, 15], [[1, 20, 5], [1, 1, 1], [16, 1, 0], [1, 1, 17]]
    pages = 64
    rng = np.random.default_rng(3)
    perm = rng.permutation(pages)
    table = np.full((B, width), -1)
    free, used = [], 0
    for b, n in enumerate(lens):
        k = -(-n // P)
        table[b, :k] = perm[used:used + k]
        used += k
    free = perm[used:]
    bt, free_t = _i32(table.tolist()), _i32(free.tolist())
    kc, vc = (torch.zeros((pages, P, Hk, 128), dtype=torch.float16, device=DEV) for _ in range(2))
    r = step.rotary_setup(64, theta=10000.0)  # each 64-dim half is rotated on its own
    f, _ = oracle_step.rates(64, 10000.0)
    lam = _i32([1]).float() * torch.linspace(0.1, 0.8, Hq, device=DEV)
    cfg = fi.default_plan_config(0, differential=1, max_items=1 << 12, max_merge_units=1 << 10,
                                 max_partial_rows=1 << 14, decode_min_chunk=64, prefill_min_chunk=128)
    ws = fi.Workspace(cfg, device=DEV)
    tabs = step.StepTables(B, 64, cap_tok, DEV)
    head = _i32([0])
    qkv = torch.zeros((cap_tok, (Hq + 2 * Hk) * 128), dtype=torch.float16, device=DEV)
    q, k, v = (x.unflatten(1, (-1, 128)) for x in qkv.split([Hq * 128, Hk * 128, Hk * 128], 1))
    q_rot, o = torch.zeros((cap_tok, Hq, 128), dtype=torch.float16, device=DEV), torch.zeros(
        (cap_tok, Hq, 128), dtype=torch.float16, device=DEV)
    lse = torch.zeros((cap_tok, Hq, 2), device=DEV)
    ql, kl = _i32([0] * B), _i32([0] * B)
    seq = [(np.zeros((0, Hk, 128)), np.zeros((0, Hk, 128))) for _ in range(B)]
    half = lambda t: t.unflatten(2, (2, 64)).flatten(1, 2)  # noqa: E731

    def device_step(info):
        step.build_tables(tabs, ql, kl, bt, P, free_t, head)
        step.append(r, tabs.positions, tabs.slots, half(q), q_rot.view(cap_tok, 2 * Hq, 64), half(k), half(v),
                    kc.view(pages, P, 2 * Hk, 64), vc.view(pages, P, 2 * Hk, 64))
        differential.run(ws, info, q_rot, kc, vc, tabs.kv_indices, lam, o, lse, 0.125)

    graph, info = None, None
    for n, qs in enumerate(steps):
        kvs = [a + b for a, b in zip(lens, qs)]
        if n == 0:  # keys of the earlier part of each request
            for b in range(B):
                old = rng.standard_normal((lens[b], Hk, 128))
                kk, vv = torch.tensor(old).half(), torch.tensor(rng.standard_normal((lens[b], Hk, 128))).half()
                for j in range(lens[b]):
                    kc[int(table[b, j // P]), j % P] = kk[j].to(DEV)
                    vc[int(table[b, j // P]), j % P] = vv[j].to(DEV)
                seq[b] = (kk.double().numpy(), vv.double().numpy())
        total = sum(qs)
        qkv.copy_(torch.tensor(rng.standard_normal(qkv.shape)))
        ql.copy_(_i32(qs))
        kl.copy_(_i32(kvs))
        kvp = np.concatenate([[0], np.cumsum([-(-x // P) for x in kvs])])
        qop = np.concatenate([[0], np.cumsum(qs)])
        last = [x - (-(-x // P) - 1) * P if x else 1 for x in kvs]
        info_n = fi.plan(ws, qop, kvp, [], last, Hq, Hk, 128, P, 1)
        if graph is None:
            info = info_n
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                device_step(info)
        graph.replay()
        torch.cuda.synchronize()
        assert fi.device_status(ws) == 0 and int(tabs.counts[4]) == 0
        assert tabs.kv_indptr.tolist() == kvp.tolist() and tabs.qo_indptr.tolist() == qop.tolist()
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        ids, dense_k, dense_v = [], np.zeros((int(kvp[-1]), P, Hk, 128)), np.zeros((int(kvp[-1]), P, Hk, 128))
        rq = np.zeros((total, Hq, 128))
        for b in range(B):
            sl = slice(int(qop[b]), int(qop[b + 1]))
            pos = list(range(lens[b], kvs[b]))
            # the rotated rows enter attention in fp16
            rk = oracle_step.rotate(f64(half(k))[sl], pos, f, 1.0, 64, False).reshape(-1, Hk, 128)
            rq[sl] = f64(q_rot)[sl]
            want = oracle_step.rotate(f64(half(q))[sl], pos, f, 1.0, 64, False).reshape(-1, Hq, 128)
            assert np.abs(rq[sl] - want).max(initial=0) <= 2.0 ** -11 * 6 + 1e-5  # |x| < 6: half a step
            rk16 = torch.tensor(rk).half().double().numpy()
            seq[b] = (np.concatenate([seq[b][0], rk16]), np.concatenate([seq[b][1], f64(v)[sl]]))
            for j in range(kvs[b]):
                dense_k[int(kvp[b]) + j // P, j % P] = seq[b][0][j]
                dense_v[int(kvp[b]) + j // P, j % P] = seq[b][1][j]
        ro, rl, y, size = oracle_diff.attention(qop, kvp, np.arange(int(kvp[-1])), last, P, 1, 0.125, rq, dense_k,
                                                dense_v, f64(lam), mag=True)
        # fp16: weights within 2^-10 (rounded weight and sum), and a key off by one fp16
        # step where its fp64 rotation falls between two (|q| sqrt(64) 2^-11 * 6 / 8 of a logit)
        tol = oracle_diff.slack(ro, y, size, 2.0 ** -10 + 2e-2, 2.0 ** -11) + 1e-7
        assert (np.abs(f64(o)[:total] - ro) <= tol).all()
        assert np.abs(f64(lse)[:total] - rl).max() <= 2e-2
        head.copy_(tabs.counts[3:4])
        lens = kvs


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [1, 16])
def test_a_step_against_the_cache_that_it_wrote(page, dtype):
    """The same three calls, attention against the oracle over the rotated queries and the cache as they
    are, so that its own roundings are all there is: 1e-4 of a weight for the exponentials and sums (as in the
    tests of the attention alone), one rounding of a weight, half a step of the output."""
    Hq, Hk, qs, kvs = 8, 2, [1, 40, 1, 9], [300, 200, 33, 9]
    pages = [-(-x // page) for x in kvs]
    n, pool = sum(qs), sum(pages) + 5
    ids = np.random.default_rng(page).permutation(pool).astype(np.int32)
    table = np.full((4, max(pages)), -1, np.int32)
    for b in range(4):
        had = -(-(kvs[b] - qs[b]) // page)
        table[b, :had], ids = ids[:had], ids[had:]
    t = step.StepTables(4, sum(pages), n + 3, DEV)
    step.build_tables(t, _i32(qs), _i32(kvs), _i32(table.tolist()), page, _i32(ids.tolist()), _i32([0]))
    q, k, v = (_randn((n + 3, h, 128), dtype, i) for i, h in enumerate((Hq, Hk, Hk)))
    kc, vc = _randn((pool, page, Hk, 128), dtype, 3), _randn((pool, page, Hk, 128), dtype, 4)
    half = lambda x: x.unflatten(2, (2, 64)).flatten(1, 2)  # noqa: E731
    step.append(step.rotary_setup(64), t.positions, t.slots, half(q), half(q), half(k), half(v),
                kc.view(pool, page, 2 * Hk, 64), vc.view(pool, page, 2 * Hk, 64))
    lam, w = torch.rand(Hq, generator=_gen(5), device=DEV), 1 + 0.2 * torch.randn(128, generator=_gen(6), device=DEV)
    ws = fi.Workspace(fi.default_plan_config(0, differential=1, max_items=1 << 12, max_merge_units=1 << 10,
                                             max_partial_rows=1 << 14), device=DEV)
    qop, kvp = np.cumsum([0] + qs), np.cumsum([0] + pages)
    last = [x - (p - 1) * page for x, p in zip(kvs, pages)]
    info = fi.plan(ws, qop, kvp, [], last, Hq, Hk, 128, page, 1)
    o, lse = torch.empty_like(q), torch.empty((n + 3, Hq, 2), device=DEV)
    differential.run(ws, info, q, kc, vc, t.kv_indices, lam, o, lse, 0.125, norm_weight=w)
    assert fi.device_status(ws) == 0 and int(t.counts[4]) == 0
    f64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    ro, rl, y, size = oracle_diff.attention(qop, kvp, t.kv_indices.cpu().numpy(), last, page, 1, 0.125, f64(q)[:n],
                                            f64(kc), f64(vc), f64(lam), f64(w), 1e-5, 1.0, mag=True)
    eps = torch.finfo(DT[dtype]).eps / 2
    tol = oracle_diff.slack(ro, y, size, 1e-4 + eps, eps, f64(w)) + 1e-7
    assert (np.abs(f64(o)[:n] - ro) <= tol).all() and np.abs(f64(lse)[:n] - rl).max() <= 1e-3
