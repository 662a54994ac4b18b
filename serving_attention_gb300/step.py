"""Python binding of the operators around an attention step (include/fi_step.h):
page tables and slot maps built on the GPU, and rotary positions with the
append to the paged cache.  Argument marshalling only; there is no fallback.

    tables = StepTables(max_batch=64, max_pages=1 << 17, max_tokens=64)
    build_tables(tables, qo_lens, kv_lens, block_table, 16, free_pages, free_head)
    rot = rotary_setup(128, theta=500000.0)
    append(rot, tables.positions, tables.slots, q, q_rot, k, v, k_cache, v_cache)
"""
from __future__ import annotations

import ctypes

import torch

from . import _DTYPE, _check, _stream_ptr, load as _load_lib
from .differential import _on_device

EXPORTS = ["fi_build_step_tables", "fi_rotary_setup", "fi_rotary_apply", "fi_rotary_append"]
SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3, "yarn": 4}
MAX_BATCH, COUNTS, MAX_PAIRS = 8192, 8, 128


class RotaryConfig(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_positions", ctypes.c_int32), ("low_turns", ctypes.c_float), ("high_turns", ctypes.c_float),
                ("amplitude", ctypes.c_float)]


class Rotary(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("amplitude", ctypes.c_float), ("reserved2", ctypes.c_float),
                ("turns", ctypes.c_uint64 * MAX_PAIRS)]


_bound = False
_Strides = ctypes.c_int64 * 3


def load() -> ctypes.CDLL:
    global _bound
    lib = _load_lib()
    if not _bound:
        vp, i32, i64, ci = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
        rotp = ctypes.POINTER(Rotary)
        rows = [vp, i64, i64, vp, i64, i64, i32]
        lib.fi_rotary_setup.argtypes = [ctypes.POINTER(RotaryConfig), rotp]
        lib.fi_rotary_apply.argtypes = [rotp, vp, i32, *rows, *rows, ci, vp]
        lib.fi_rotary_append.argtypes = [rotp, vp, vp, i32, *rows, vp, i64, i64, vp, i64, i64, i32, i32, vp, vp, vp,
                                         vp, i32, i32, ci, vp]
        lib.fi_build_step_tables.argtypes = [vp, vp, i32, i32, vp, i64, i32, vp, i32, vp, vp, vp, vp, vp, i32, vp, vp,
                                             i32, vp, vp]
        for name in EXPORTS:
            getattr(lib, name).restype = ci
        _bound = True
    return lib


# ------------------------------------------------------------------ rotary

def rotary_setup(head_dim: int, rot_dim: int | None = None, interleaved: bool = False, theta: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, original_positions: int = 0, low_turns: float = 1.0,
                 high_turns: float | None = None, amplitude: float = 0.0) -> Rotary:
    """The rates of a model's rotary positions (see fi_rotary_config).
    high_turns defaults to 4 for "by_parts" and 32 for "yarn"."""
    if scaling not in SCALINGS:
        raise ValueError(f"scaling is one of {sorted(SCALINGS)}")
    if high_turns is None:
        high_turns = 32.0 if scaling == "yarn" else 4.0
    cfg = RotaryConfig(head_dim, head_dim if rot_dim is None else rot_dim, int(interleaved), SCALINGS[scaling], theta,
                       factor, original_positions, low_turns, high_turns, amplitude)
    rot = Rotary()
    _check(load().fi_rotary_setup(ctypes.byref(cfg), ctypes.byref(rot)), "fi_rotary_setup")
    return rot


def _rows(t: torch.Tensor | None, tokens: int, dtype, device, dim: int, what: str):
    """Checks [tokens, heads, dim] rows; their heads (0 for None)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.device != device:
        raise TypeError(f"{what} must have the dtype and device of the other tensors")
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != dim or t.stride(2) != 1:
        raise ValueError(f"{what} is [tokens, heads, {dim}], the last dimension contiguous")
    return t.shape[1]


def _index(t: torch.Tensor, device, what: str) -> int:
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.device != device:
        raise TypeError(f"{what} must be a contiguous int32 vector on the tensors' device")
    return t.shape[0]


def _ptr(t: torch.Tensor | None):
    return (t.data_ptr(), t.stride(0), t.stride(1)) if t is not None else (None, 0, 0)


def rotate(rot: Rotary, positions: torch.Tensor, q: torch.Tensor | None, q_out: torch.Tensor | None,
           k: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Rotate q into q_out and k into k_out ([tokens, heads, head_dim]; an output may be its input)."""
    some = q if q is not None else k
    if some is None:
        raise ValueError("q or k is needed")
    dtype, device = some.dtype, some.device
    if dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype}")
    tokens = _index(positions, device, "positions")
    hq, hk = (_rows(t, tokens, dtype, device, rot.head_dim, n) for t, n in ((q, "q"), (k, "k")))
    if _rows(q_out, tokens, dtype, device, rot.head_dim, "q_out") != hq or \
            _rows(k_out, tokens, dtype, device, rot.head_dim, "k_out") != hk:
        raise ValueError("q_out and k_out have the shapes of q and k")
    with _on_device(device):
        st = load().fi_rotary_apply(ctypes.byref(rot), positions.data_ptr(), tokens, *_ptr(q), *_ptr(q_out), hq,
                                    *_ptr(k), *_ptr(k_out), hk, _DTYPE[dtype], _stream_ptr(stream))
    _check(st, "fi_rotary_apply")


def append(rot: Rotary, positions: torch.Tensor, slots: torch.Tensor, q: torch.Tensor | None,
           q_out: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor | None, k_cache: torch.Tensor,
           v_cache: torch.Tensor | None, stream=None):
    """Rotate q into q_out and k into k_cache, and copy v into v_cache, token t
    at slot slots[t] = page * page_size + slot (outside the cache: not written).
    Caches [pages, page_size, heads, dim]."""
    dtype, device = k.dtype, k.device
    if dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype}")
    tokens = _index(positions, device, "positions")
    if _index(slots, device, "slots") != tokens:
        raise ValueError("positions and slots have one entry per token")
    hq = _rows(q, tokens, dtype, device, rot.head_dim, "q")
    if _rows(q_out, tokens, dtype, device, rot.head_dim, "q_out") != hq:
        raise ValueError("q_out has the shape of q")
    hk = _rows(k, tokens, dtype, device, rot.head_dim, "k")
    v_dim = 0 if v is None else v.shape[2]
    if v is not None and _rows(v, tokens, dtype, device, v_dim, "v") != hk:
        raise ValueError("v has the heads of k")
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    for c, dim in ((k_cache, rot.head_dim), (v_cache, v_dim)):
        if c is None:
            continue
        if c.dtype != dtype or c.device != device:
            raise TypeError("the caches must have the dtype and device of the other tensors")
        if c.dim() != 4 or c.shape[:2] != k_cache.shape[:2] or c.shape[2] != hk or c.shape[3] != dim or c.stride(3) != 1:
            raise ValueError("the caches are [pages, page_size, heads, dim], the last dimension contiguous")
    with _on_device(device):
        st = load().fi_rotary_append(
            ctypes.byref(rot), positions.data_ptr(), slots.data_ptr(), tokens, *_ptr(q), *_ptr(q_out), hq, *_ptr(k),
            *_ptr(v), v_dim, hk, k_cache.data_ptr(), _Strides(*k_cache.stride()[:3]),
            v_cache.data_ptr() if v_cache is not None else None,
            _Strides(*v_cache.stride()[:3]) if v_cache is not None else None, k_cache.shape[1], k_cache.shape[0],
            _DTYPE[dtype], _stream_ptr(stream))
    _check(st, "fi_rotary_append")


# ------------------------------------------------------------------ tables

class StepTables:
    """The device arrays that build_tables fills (see fi_build_step_tables)."""

    def __init__(self, max_batch: int, max_pages: int, max_tokens: int, device="cuda"):
        def i32(n, fill=0):
            return torch.full((n,), fill, dtype=torch.int32, device=device)

        self.max_batch, self.max_pages, self.max_tokens = max_batch, max_pages, max_tokens
        self.qo_indptr, self.kv_indptr, self.last_page_len = i32(max_batch + 1), i32(max_batch + 1), i32(max_batch)
        self.kv_indices, self.positions, self.slots = i32(max_pages, -1), i32(max_tokens), i32(max_tokens, -1)
        self.counts = i32(COUNTS)  # {tokens, pages, pages taken, next free_head, status, 0, 0, 0}


def build_tables(tables: StepTables, qo_lens: torch.Tensor, kv_lens: torch.Tensor, block_table: torch.Tensor,
                 page_size: int, free_pages: torch.Tensor | None = None, free_head: torch.Tensor | None = None,
                 stream=None):
    """Give out the step's new pages and fill `tables`, on the GPU (no host read).
    block_table int32 [batch, width] (rows may be strided) is updated in place;
    free_head int32 [1] is not: the next step's is counts[3:4]."""
    device = qo_lens.device
    batch = _index(qo_lens, device, "qo_lens")
    if _index(kv_lens, device, "kv_lens") != batch:
        raise ValueError("qo_lens and kv_lens have one entry per request")
    if batch > tables.max_batch:
        raise ValueError("more requests than the tables hold")
    if tables.counts.device != device:
        raise TypeError("the tables must be on the lengths' device")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.device != device or \
            block_table.shape[0] < batch or block_table.stride(1) != 1:
        raise TypeError("block_table is an int32 [batch, width] tensor, rows contiguous")
    if (free_pages is None) != (free_head is None):
        raise ValueError("free_pages and free_head go together")
    num_free = 0 if free_pages is None else _index(free_pages, device, "free_pages")
    if free_head is not None and _index(free_head, device, "free_head") != 1:
        raise ValueError("free_head has one entry")
    t = tables
    with _on_device(device):
        st = load().fi_build_step_tables(
            qo_lens.data_ptr(), kv_lens.data_ptr(), batch, page_size, block_table.data_ptr(), block_table.stride(0),
            block_table.shape[1], free_pages.data_ptr() if num_free else None, num_free,
            free_head.data_ptr() if free_head is not None else None, t.qo_indptr.data_ptr(), t.kv_indptr.data_ptr(),
            t.last_page_len.data_ptr(), t.kv_indices.data_ptr() if t.max_pages else None, t.max_pages,
            t.positions.data_ptr() if t.max_tokens else None, t.slots.data_ptr() if t.max_tokens else None,
            t.max_tokens, t.counts.data_ptr(), _stream_ptr(stream))
    _check(st, "fi_build_step_tables")
