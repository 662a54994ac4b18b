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
import struct

import torch

from . import _DTYPE, _check, load as _load_lib
from .differential import _call

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


_apply = _append = _tables = None
_APPLY_ARGS = struct.Struct("=18q")   # fi_rotary_apply_args
_APPEND_ARGS = struct.Struct("=30q")  # fi_rotary_append_args
_TABLE_ARGS = struct.Struct("=19q")   # fi_step_tables_args


def load() -> ctypes.CDLL:
    global _apply, _append, _tables
    lib = _load_lib()
    if _tables is None:
        lib.fi_rotary_setup.argtypes = [ctypes.POINTER(RotaryConfig), ctypes.POINTER(Rotary)]
        for name in EXPORTS:
            fn = getattr(lib, name)
            fn.restype = ctypes.c_int
            if name != "fi_rotary_setup":
                fn.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
        _apply, _append, _tables = lib.fi_rotary_apply, lib.fi_rotary_append, lib.fi_build_step_tables
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


def _rows(x: torch.Tensor | None, y: torch.Tensor | None, tokens: int, dim: int, dtype, index: int, what: str):
    """Checks [tokens, heads, dim] rows x and their outputs y: (heads, their fi_rows)."""
    if x is None or y is None:
        if x is not y:
            raise ValueError(f"{what} and its output go together")
        return 0, 0, 0, 0, 0, 0, 0
    if x.dtype is not dtype or y.dtype is not dtype or x.get_device() != index or y.get_device() != index:
        raise TypeError(f"{what} and its output must have the dtype and device of the other tensors")
    shape = x.shape
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim or y.shape != shape:
        raise ValueError(f"{what} and its output are [tokens, heads, {dim}]")
    xt, xh, xd = x.stride()
    yt, yh, yd = y.stride()
    if xd != 1 or yd != 1:
        raise ValueError(f"the last dimension of {what} and its output must be contiguous")
    return shape[1], x.data_ptr(), xt, xh, y.data_ptr(), yt, yh


def _index(t: torch.Tensor, index: int, what: str) -> int:
    if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.get_device() != index:
        raise TypeError(f"{what} must be a contiguous int32 vector on the tensors' device")
    return t.shape[0]


def rotate(rot: Rotary, positions: torch.Tensor, q: torch.Tensor | None, q_out: torch.Tensor | None,
           k: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Rotate q into q_out and k into k_out ([tokens, heads, head_dim]; an output may be its input)."""
    if _apply is None:
        load()
    some = q if q is not None else k
    if some is None:
        raise ValueError("q or k is needed")
    dtype, index = some.dtype, some.get_device()
    code = _DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    tokens, dim = _index(positions, index, "positions"), rot.head_dim
    hq, *q_rows = _rows(q, q_out, tokens, dim, dtype, index, "q")
    hk, *k_rows = _rows(k, k_out, tokens, dim, dtype, index, "k")
    _call(_apply, _APPLY_ARGS.pack(ctypes.addressof(rot), positions.data_ptr(), tokens, *q_rows, hq, *k_rows, hk, code),
          index, stream, "fi_rotary_apply")


def append(rot: Rotary, positions: torch.Tensor, slots: torch.Tensor, q: torch.Tensor | None,
           q_out: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor | None, k_cache: torch.Tensor,
           v_cache: torch.Tensor | None, stream=None):
    """Rotate q into q_out and k into k_cache, and copy v into v_cache, token t
    at slot slots[t] = page * page_size + slot (outside the cache: not written).
    Caches [pages, page_size, heads, dim]."""
    if _append is None:
        load()
    dtype, index = k.dtype, k.get_device()
    code = _DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    tokens, dim = _index(positions, index, "positions"), rot.head_dim
    if _index(slots, index, "slots") != tokens:
        raise ValueError("positions and slots have one entry per token")
    hq, *q_rows = _rows(q, q_out, tokens, dim, dtype, index, "q")
    k_shape, cache = k.shape, k_cache.shape
    kt, kh, kd = k.stride()
    kcp, kcs, kch, kcd = k_cache.stride()
    if len(k_shape) != 3 or k_shape[0] != tokens or k_shape[2] != dim or kd != 1:
        raise ValueError(f"k is [tokens, heads, {dim}], the last dimension contiguous")
    hk = k_shape[1]
    if k_cache.dtype is not dtype or k_cache.get_device() != index:
        raise TypeError("the caches must have the dtype and device of the other tensors")
    pages, page_size = cache[0], cache[1]
    if cache[2] != hk or cache[3] != dim or kcd != 1:
        raise ValueError("k_cache is [pages, page_size, heads of k, head_dim], the last dimension contiguous")
    if v is None or v_cache is None:
        if v is not v_cache:
            raise ValueError("v and v_cache go together")
        v_dim = vt = vh = vcp = vcs = vch = v_ptr = vc_ptr = 0
    else:
        if v.dtype is not dtype or v_cache.dtype is not dtype or v.get_device() != index or \
                v_cache.get_device() != index:
            raise TypeError("v and v_cache must have the dtype and device of the other tensors")
        v_dim = v.shape[-1]
        vt, vh, vd = v.stride()
        vcp, vcs, vch, vcd = v_cache.stride()
        if v.shape != (tokens, hk, v_dim) or v_cache.shape != (pages, page_size, hk, v_dim) or vd != 1 or vcd != 1:
            raise ValueError("v is [tokens, heads of k, v_dim] and v_cache [pages, page_size, heads, v_dim], the last "
                             "dimension contiguous")
        v_ptr, vc_ptr = v.data_ptr(), v_cache.data_ptr()
    _call(_append, _APPEND_ARGS.pack(ctypes.addressof(rot), positions.data_ptr(), slots.data_ptr(), tokens, *q_rows, hq,
                                     k.data_ptr(), kt, kh, v_ptr, vt, vh, v_dim, hk, k_cache.data_ptr(), kcp, kcs, kch,
                                     vc_ptr, vcp, vcs, vch, page_size, pages, code),
          index, stream, "fi_rotary_append")


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
    if _tables is None:
        load()
    index = qo_lens.get_device()
    batch = _index(qo_lens, index, "qo_lens")
    if _index(kv_lens, index, "kv_lens") != batch:
        raise ValueError("qo_lens and kv_lens have one entry per request")
    t = tables
    if batch > t.max_batch:
        raise ValueError("more requests than the tables hold")
    rows, width = block_table.shape
    row_stride, one = block_table.stride()
    if block_table.dtype is not torch.int32 or block_table.get_device() != index or rows < batch or one != 1:
        raise TypeError("block_table is an int32 [batch, width] tensor on the lengths' device, rows contiguous")
    if t.counts.get_device() != index:
        raise TypeError("the tables must be on the lengths' device")
    num_free = pages_ptr = head_ptr = 0
    if free_pages is not None and free_head is not None:
        num_free, pages_ptr, head_ptr = _index(free_pages, index, "free_pages"), free_pages.data_ptr(), \
            free_head.data_ptr()
        if _index(free_head, index, "free_head") != 1:
            raise ValueError("free_head has one entry")
    elif free_pages is not free_head:
        raise ValueError("free_pages and free_head go together")
    _call(_tables, _TABLE_ARGS.pack(qo_lens.data_ptr(), kv_lens.data_ptr(), batch, page_size, block_table.data_ptr(),
                                    row_stride if rows > 1 else max(row_stride, width), width, pages_ptr, num_free,
                                    head_ptr, t.qo_indptr.data_ptr(), t.kv_indptr.data_ptr(),
                                    t.last_page_len.data_ptr(), t.kv_indices.data_ptr(), t.max_pages,
                                    t.positions.data_ptr(), t.slots.data_ptr(), t.max_tokens, t.counts.data_ptr()),
          index, stream, "fi_build_step_tables")
