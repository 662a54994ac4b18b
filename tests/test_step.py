"""The step operators without a GPU: rotary rates against their definitions,
and the calls that are refused before any CUDA work."""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import serving_attention_gb300 as fi
from oracle import step as oracle_step
from serving_attention_gb300 import step

TURN = 2.0 ** 64


@pytest.mark.parametrize("rot_dim", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("theta", [10000.0, 500000.0])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("by_parts", 8.0),
                                            ("yarn", 16.0), ("yarn", 1.0)])
def test_rates(rot_dim, theta, scaling, factor):
    rot = step.rotary_setup(256, rot_dim, theta=theta, scaling=scaling, factor=factor, original_positions=4096)
    high = 32.0 if scaling == "yarn" else 4.0
    f, amp = oracle_step.rates(rot_dim, theta, scaling, factor, 4096, 1.0, high)
    got = np.array([float(rot.turns[i]) for i in range(rot_dim // 2)])
    want = f / (2 * np.pi) * TURN
    # pow and log in fp64 (a few steps of 2^-53), and rounding to a whole 2^-64 of a
    # turn: 0.5 of some 4e7, 1e-8 turns a position, for the slowest pairs
    assert (np.abs(got - want) <= 0.5 + 1e-12 * want).all()
    assert abs(rot.amplitude - amp) < 1e-6 and all(rot.turns[i] == 0 for i in range(rot_dim // 2, 128))


def test_closed_forms():
    rot = step.rotary_setup(64)
    assert abs(rot.turns[0] / TURN - 1 / (2 * np.pi)) < 1e-16
    plain = [step.rotary_setup(64, scaling=s, factor=1.0, original_positions=4096).turns[:32]
             for s in ("linear", "ntk", "by_parts", "yarn")]
    # a factor of 1 changes nothing (the ramp adds one rounding)
    assert all(abs(a - b) <= b * 2.0 ** -50 for p in plain for a, b in zip(p, rot.turns[:32]))
    assert step.rotary_setup(64, scaling="yarn", factor=8.0, original_positions=4096, amplitude=2.0).amplitude == 2.0


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=264), 2), (dict(head_dim=60), 2), (dict(head_dim=8), 2), (dict(rot_dim=24), 2),
    (dict(rot_dim=144), 2), (dict(rot_dim=0), 2), (dict(theta=1.0), 1), (dict(theta=float("nan")), 1),
    (dict(theta=float("inf")), 1), (dict(factor=0.5), 1), (dict(factor=float("inf")), 1), (dict(amplitude=-1.0), 1),
    (dict(amplitude=float("inf")), 1), (dict(scaling="yarn"), 1), (dict(scaling="by_parts"), 1),
    (dict(scaling="yarn", original_positions=64, low_turns=0.0), 1),
    (dict(scaling="by_parts", original_positions=64, low_turns=4.0), 1)])
def test_setup_refusals(kw, status):
    with pytest.raises(fi.FIError) as e:
        step.rotary_setup(**{"head_dim": 128, **kw})
    assert e.value.status == status


def test_setup_refuses_unknown_scaling():
    with pytest.raises(ValueError):
        step.rotary_setup(128, scaling="dynamic")
    cfg = step.RotaryConfig(128, 128, 0, 9, 1e4, 1.0, 0, 1.0, 4.0, 0.0)
    assert step.load().fi_rotary_setup(ctypes.byref(cfg), ctypes.byref(step.Rotary())) == 1
    cfg = step.RotaryConfig(128, 128, 2, 0, 1e4, 1.0, 0, 1.0, 4.0, 0.0)
    assert step.load().fi_rotary_setup(ctypes.byref(cfg), ctypes.byref(step.Rotary())) == 1


# The pointers are fake: every case returns before any CUDA call.
def _apply(**kw):
    rot = step.rotary_setup(128)
    a = dict(rot=ctypes.addressof(rot), pos=16, n=4, q=32, qt=1024, qh=128, qo=48, qot=1024, qoh=128, hq=8, k=64, kt=256,
             kh=128, ko=80, kot=256, koh=128, hk=2, dt=fi.BF16)
    a.update(kw)
    return step.load().fi_rotary_apply(step._APPLY_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), 1), (dict(pos=0), 1), (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(q=0), 1), (dict(qo=0), 1),
    (dict(k=0), 1), (dict(hq=-1), 1), (dict(dt=fi.FP32), 2), (dict(q=34), 4), (dict(qo=40), 4), (dict(k=72), 4),
    (dict(qt=1020), 4), (dict(koh=-128), 4), (dict(pos=18), 4), (dict(n=0), 0), (dict(hq=0, hk=0), 0)])
def test_apply_refusals(kw, status):
    assert _apply(**kw) == status


def _append(**kw):
    rot = step.rotary_setup(128)
    a = dict(rot=ctypes.addressof(rot), pos=16, slots=16, n=4, q=32, qt=1024, qh=128, qo=48, qot=1024, qoh=128, hq=8,
             k=64, kt=256, kh=128, v=96, vt=256, vh=128, vd=128, hk=2, kc=112, k0=4096, k1=256, k2=128, vc=128,
             v0=4096, v1=256, v2=128, page=16, pages=9, dt=fi.FP16)
    a.update(kw)
    return step.load().fi_rotary_append(step._APPEND_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(slots=0), 1), (dict(kc=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(vc=0), 1), (dict(hk=0), 1),
    (dict(pages=0), 1), (dict(pages=1 << 31), 1), (dict(vd=520), 2), (dict(vd=12), 2), (dict(page=24), 2),
    (dict(page=256), 2), (dict(dt=fi.FP32), 2), (dict(kc=120), 4), (dict(vc=136), 4), (dict(slots=18), 4),
    (dict(v1=250), 4), (dict(k0=-8), 4), (dict(n=0), 0)])
def test_append_refusals(kw, status):
    assert _append(**kw) == status


@pytest.mark.parametrize("kw", [dict(qot=0), dict(qoh=0), dict(kot=0), dict(koh=0), dict(qo=32, qot=2048),
                                dict(ko=64, koh=256)])
def test_apply_refuses_outputs_that_overlap(kw):
    assert _apply(**kw) == 1


@pytest.mark.parametrize("kw", [dict(qot=0), dict(qoh=0), dict(k0=0), dict(k1=0), dict(k2=0), dict(v0=0), dict(v1=0),
                                dict(v2=0), dict(qo=32, qot=2048)])
def test_append_refuses_outputs_that_overlap(kw):
    assert _append(**kw) == 1


@pytest.mark.parametrize("kw", [dict(qoh=8), dict(qoh=120), dict(qot=1016), dict(qot=128), dict(kot=128, koh=128),
                                dict(qot=128, qoh=504), dict(qot=1 << 62), dict(qo=32 + 2048, qot=1024),
                                dict(qo=32 + 256), dict(q=32 + 6144, qo=32), dict(q=32 + 6144 + 1792, qo=32),
                                dict(ko=64 + 768), dict(qt=128, qh=512, qot=128, qoh=512, qo=32 + 2 * (3 * 512 + 384))])
def test_apply_refuses_rows_that_meet(kw):
    """Rows of 128 that overlap their neighbours; an output some tokens or heads from its input, at its strides."""
    assert _apply(**kw) == 1


@pytest.mark.parametrize("kw", [dict(k2=64), dict(k1=128), dict(k1=248), dict(k0=2048), dict(v2=64), dict(v0=4088),
                                dict(k0=128, k1=1152, k2=128), dict(v0=1 << 61), dict(qo=32 + 256), dict(qoh=64)])
def test_append_refuses_rows_that_meet(kw):
    assert _append(**kw) == 1


def test_no_tokens_need_no_pointers():
    """The rows of an empty tensor have no address."""
    none = dict(n=0, pos=0, q=0, qo=0, k=0)
    assert _apply(**none, ko=0) == 0 and _append(**none, slots=0, v=0) == 0


def _tables(**kw):
    a = dict(q=16, kv=32, batch=4, page=16, table=48, stride=8, width=8, free=64, num_free=9, head=80, qp=96, kp=112,
             last=128, idx=144, max_pages=9, pos=160, slots=176, max_tokens=9, counts=192)
    a.update(kw)
    return step.load().fi_build_step_tables(step._TABLE_ARGS.pack(*a.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), 1), (dict(table=0), 1), (dict(counts=0), 1), (dict(batch=0), 1), (dict(width=0), 1),
    (dict(stride=7), 1), (dict(free=0), 1), (dict(head=0), 1), (dict(num_free=-1), 1), (dict(idx=0), 1),
    (dict(slots=0), 1), (dict(max_tokens=-1), 1), (dict(max_pages=1 << 31), 1), (dict(head=200), 1),
    (dict(batch=8193), 2), (dict(page=12), 2), (dict(page=256), 2), (dict(pos=162), 4)])
def test_tables_refusals(kw, status):
    assert _tables(**kw) == status


def test_calls_refuse_no_arguments():
    lib = step.load()
    assert lib.fi_rotary_apply(None, None) == lib.fi_rotary_append(None, None) == 1
    assert lib.fi_build_step_tables(None, None) == 1


def test_bindings_refuse_wrong_tensors():
    rot = step.rotary_setup(64)
    q, pos, slots = torch.zeros(3, 2, 64).half(), torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    cache = torch.zeros(2, 16, 2, 64).half()
    with pytest.raises(TypeError):  # not on a GPU
        step.rotate(rot, pos, q, q)
    with pytest.raises(TypeError):
        step.append(rot, pos, slots, q, q, q, q, cache, cache)
    with pytest.raises(ValueError):
        step.rotate(rot, pos, None, None)
    with pytest.raises(ValueError):
        step.rotate(rot, pos, q, None)
    with pytest.raises(ValueError):
        step.rotate(rot, pos, q[..., :32], q[..., :32])
    with pytest.raises(TypeError):
        step.rotate(rot, pos.long(), q, q)
    with pytest.raises(TypeError):
        step.rotate(rot, pos, q, q.float())
    with pytest.raises(TypeError):
        step.rotate(rot, pos, q.double(), q.double())
    with pytest.raises(ValueError):
        step.append(rot, pos, slots[:2], q, q, q, q, cache, cache)
    with pytest.raises(ValueError):
        step.append(rot, pos, slots, q, q, q, None, cache, cache)
    with pytest.raises(ValueError):
        step.append(rot, pos, slots, q, q, q[:, :1], q[:, :1], cache, cache)
    t = step.StepTables(2, 4, 4, "cpu")
    lens, table = torch.ones(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(TypeError):
        step.build_tables(t, lens, lens, table, 16)
    with pytest.raises(ValueError):
        step.build_tables(t, lens, lens[:1], table, 16)
    with pytest.raises(ValueError):
        step.build_tables(step.StepTables(1, 4, 4, "cpu"), lens, lens, table, 16)
    with pytest.raises(ValueError):
        step.build_tables(t, lens, lens, table, 16, lens, None)
    with pytest.raises(TypeError):
        step.build_tables(t, lens, lens, table.t(), 16)


def test_every_entry_is_declared():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "fi_step.h")).read()
    assert set(re.findall(r"^fi_status\s+(fi_\w+)\s*\(", text, re.M)) == set(step.EXPORTS)


def test_oracle_tables_by_hand():
    got = oracle_step.tables([2, 0, 3], [5, 0, 3], [[7, 9, -1], [-1, -1, -1], [-1, -1, -1]], 4, [20, 21, 22], 1, 9, 6)
    # 3 old keys are one page (7): the fifth key opens page 21, the third request page 22
    assert got["kv_indices"] == [7, 21, 22] and got["slots"] == [7 * 4 + 3, 21 * 4, 88, 89, 90, -1]
    assert got["positions"] == [3, 4, 0, 1, 2, 0] and got["last_page_len"] == [1, 0, 3]
    assert got["counts"] == [5, 3, 2, 3, 0, 0, 0, 0]
