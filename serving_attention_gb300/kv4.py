"""Python binding of the 4-bit paged cache (include/fi_kv4.h): the append that
norms, rotates and quantises, attention over it, and rows read back in 16 bits.
Argument marshalling only; there is no fallback.

    cache = empty_cache(num_pages, 16, num_kv_heads)
    append(rot, tables.positions, tables.slots, q, q_rot, k, v, cache, 16)
    cfg = default_plan_config(0, kv_bits=4)
    ws = Workspace(cfg)
    info = plan(ws, qo_indptr, kv_indptr, kv_indices, last_page_len, 32, 8, 128, 16, causal=1)
    run(ws, info, q_rot, cache, kv_indices_dev, o, lse, sm_scale)
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _DTYPE, PlanInfo, Workspace, load as _load_lib
from .differential import _call
from .step import Rotary, _index, _rows, _weight

EXPORTS = ["fi_kv4_page_bytes", "fi_kv4_append", "fi_kv4_read", "fi_batch_paged_attention_run_kv4"]
HEAD_DIM = 128

_append = _read = _run = None
_APPEND_ARGS = struct.Struct("=28qd")  # fi_kv4_append_args
_READ_ARGS = struct.Struct("=15q")     # fi_kv4_read_args
_RUN_ARGS = struct.Struct("=17q2f")    # fi_kv4_args


def load() -> ctypes.CDLL:
    global _append, _read, _run
    lib = _load_lib()
    if _run is None:
        lib.fi_kv4_page_bytes.argtypes, lib.fi_kv4_page_bytes.restype = [ctypes.c_int64], ctypes.c_size_t
        for name in EXPORTS[1:]:
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
        _append, _read, _run = lib.fi_kv4_append, lib.fi_kv4_read, lib.fi_batch_paged_attention_run_kv4
    return lib


def page_bytes(page_size: int) -> int:
    """Bytes of one page of one head."""
    n = load().fi_kv4_page_bytes(page_size)
    if n == 0:
        raise ValueError("page_size is a power of two in [1, 128]")
    return n


def empty_cache(num_pages: int, page_size: int, num_kv_heads: int, device="cuda") -> torch.Tensor:
    """A cache of zeros: uint8 [num_pages, num_kv_heads, page_bytes(page_size)]."""
    return torch.zeros((num_pages, num_kv_heads, page_bytes(page_size)), dtype=torch.uint8, device=device)


_page_bytes: dict[int, int] = {}


def _cache(cache: torch.Tensor, page_size: int, heads: int, index: int):
    """(pointer, page stride, head stride, pages) of a checked cache."""
    per_page = _page_bytes.get(page_size)
    if per_page is None:
        per_page = _page_bytes[page_size] = page_bytes(page_size)
    if cache.dtype is not torch.uint8 or cache.get_device() != index:
        raise TypeError("the cache must be uint8 on the tensors' device")
    if cache.dim() == 3:
        pages, n, size = cache.shape
        page_stride, head_stride, one = cache.stride()
        if n == heads and size == per_page and one == 1:
            return cache.data_ptr(), page_stride, head_stride, pages
    raise ValueError(f"the cache is [pages, {heads} heads, {per_page} bytes], the last dimension contiguous")


def append(rot: Rotary | None, positions: torch.Tensor | None, slots: torch.Tensor, q: torch.Tensor | None,
           q_out: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, page_size: int,
           q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6, stream=None):
    """Norm q and k (where weights are given), rotate them (rot None: not), write q into q_out, and quantise k and v
    into the cache, token t at slot slots[t] = page * page_size + slot (outside the cache: not written).
    Weights fp32 [128] or [heads, 128]."""
    if _append is None:
        load()
    dtype, index = k.dtype, k.get_device()
    code = _DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    tokens = _index(slots, index, "slots")
    rot_ptr = pos_ptr = 0
    if rot is not None:
        if rot.head_dim != HEAD_DIM:
            raise ValueError("the 4-bit cache has heads of 128 dims")
        if positions is None or _index(positions, index, "positions") != tokens:
            raise ValueError("positions and slots have one entry per token")
        rot_ptr, pos_ptr = ctypes.addressof(rot), positions.data_ptr()
    hq, *q_rows = _rows(q, q_out, tokens, HEAD_DIM, dtype, index, "q")
    if v.dtype is not dtype or v.get_device() != index:
        raise TypeError("k and v must share dtype and device")
    shape = k.shape
    if len(shape) != 3 or v.shape != shape:
        raise ValueError("k and v are [tokens, heads, 128], the last dimension contiguous")
    n, hk, dim = shape
    kt, kh, kd = k.stride()
    vt, vh, vd = v.stride()
    if n != tokens or dim != HEAD_DIM or kd != 1 or vd != 1:
        raise ValueError("k and v are [tokens, heads, 128], the last dimension contiguous")
    c_ptr, cp, ch, pages = _cache(cache, page_size, hk, index)
    qw = _weight(q_weight, hq, HEAD_DIM, index, "q_weight")
    kw = _weight(k_weight, hk, HEAD_DIM, index, "k_weight")
    _call(_append, _APPEND_ARGS.pack(rot_ptr, pos_ptr, slots.data_ptr(), tokens, *q_rows, hq, k.data_ptr(), kt, kh,
                                     v.data_ptr(), vt, vh, hk, *qw, *kw, c_ptr, cp, ch, page_size, pages, code, eps),
          index, stream, "fi_kv4_append")


def _out(out: torch.Tensor | None, dtype, index: int, shape):
    """(pointer, token stride, head stride) of an output of read."""
    if out is None:
        return 0, 0, 0
    if out.dtype is not dtype or out.get_device() != index:
        raise TypeError("the outputs must share dtype and device")
    if out.shape == shape:
        row, head, one = out.stride()
        if one == 1:
            return out.data_ptr(), row, head
    raise ValueError("the outputs are [slots, heads, 128], the last dimension contiguous")


def read(slots: torch.Tensor, cache: torch.Tensor, page_size: int, k_out: torch.Tensor | None,
         v_out: torch.Tensor | None, stream=None):
    """Write the values held at slots[i] into row i of k_out and v_out [rows, heads, 128] (None: not wanted; a slot
    outside the cache: zeros)."""
    if _read is None:
        load()
    some = k_out if k_out is not None else v_out
    if some is None:
        raise ValueError("k_out or v_out is needed")
    dtype, index, shape = some.dtype, some.get_device(), some.shape
    code = _DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    rows = _index(slots, index, "slots")
    if len(shape) != 3:
        raise ValueError("the outputs are [slots, heads, 128], the last dimension contiguous")
    n, heads, dim = shape
    kp, kt, kh = _out(k_out, dtype, index, shape)
    vp, vt, vh = _out(v_out, dtype, index, shape)
    if n != rows or dim != HEAD_DIM:
        raise ValueError("the outputs are [slots, heads, 128], the last dimension contiguous")
    c_ptr, cp, ch, pages = _cache(cache, page_size, heads, index)
    _call(_read, _READ_ARGS.pack(slots.data_ptr(), rows, kp, kt, kh, vp, vt, vh, heads, c_ptr, cp, ch, page_size, pages,
                                 code), index, stream, "fi_kv4_read")


def run(ws: Workspace, info: PlanInfo, q: torch.Tensor, cache: torch.Tensor, kv_indices_dev: torch.Tensor,
        o: torch.Tensor, lse: torch.Tensor | None, sm_scale: float, stream=None):
    """Enqueue attention over the 4-bit cache for the current plan of `ws`.

    q, o [tokens, Hq, 128]; cache uint8 [pages, Hkv, page_bytes]; lse fp32 [tokens, Hq] or None."""
    if _run is None:
        load()
    dtype, index = q.dtype, q.get_device()
    code = _DTYPE.get(dtype)
    if code is None or o.dtype is not dtype:
        raise TypeError("q and o must share one 16-bit dtype")
    if kv_indices_dev.dtype is not torch.int32 or not kv_indices_dev.is_contiguous():
        raise TypeError("kv_indices must be a contiguous int32 device tensor")
    if not (index == kv_indices_dev.get_device() == o.get_device() == ws.int_ws.get_device()):
        raise TypeError("all tensors must be on one device")
    hq = info.num_qo_heads
    shape = q.shape
    tokens = shape[0]
    qt, qh, qd = q.stride()
    ot, oh, od = o.stride()
    if shape != (tokens, hq, HEAD_DIM) or o.shape != shape or qd != 1 or od != 1:
        raise ValueError("q and o are [tokens, num_qo_heads, 128], the last dimension contiguous")
    c_ptr, cp, ch, pages = _cache(cache, info.page_size, info.num_kv_heads, index)
    lse_ptr = 0
    if lse is not None:
        if lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != index or \
                lse.shape != (tokens, hq):
            raise ValueError("lse is a contiguous fp32 [tokens, num_qo_heads] tensor")
        lse_ptr = lse.data_ptr()
    _call(_run, _RUN_ARGS.pack(ctypes.addressof(info), q.data_ptr(), qt, qh, tokens, c_ptr, cp, ch, pages,
                               kv_indices_dev.data_ptr(), o.data_ptr(), ot, oh, lse_ptr, code, ws.int_ws.data_ptr(),
                               ws.float_ws.data_ptr(), sm_scale, 0.0),
          index, stream, "fi_batch_paged_attention_run_kv4")
