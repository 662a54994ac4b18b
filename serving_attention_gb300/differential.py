"""Python binding of differential attention over the paged cache (include/fi_diff.h).

Argument marshalling only, like the package's other bindings; there is no
fallback.  The plan is the ordinary one, made with differential=1:

    cfg = default_plan_config(0, differential=1)
    ws = Workspace(cfg)
    info = plan(ws, qo_indptr, kv_indptr, kv_indices, last_page_len, 32, 8, 128, 16, causal=1)
    differential.run(ws, info, q, k_cache, v_cache, kv_indices_dev, lam, o, lse, sm_scale)

A decode step makes its calls within microseconds of each other, so the
arguments travel as one packed struct and every attribute of a tensor is asked
for once.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _DTYPE, PlanInfo, Workspace, _check, load as _load_lib

EXPORTS = ["fi_batch_paged_attention_run_differential"]

_run = None
_ARGS = struct.Struct("=24q4f")  # fi_differential_args


def load() -> ctypes.CDLL:
    global _run
    lib = _load_lib()
    if _run is None:
        fn = lib.fi_batch_paged_attention_run_differential
        fn.argtypes, fn.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
        _run = fn
    return lib


def _call(fn, args: bytes, index: int, stream, where: str):
    """Calls fn on device `index`, whichever is current, and its current stream if none is given."""
    if index < 0:
        raise TypeError("the tensors must be on a CUDA device")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _call(fn, args, index, stream, where)
    status = fn(args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    if status:
        _check(status, where)


def run(ws: Workspace, info: PlanInfo, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
        kv_indices_dev: torch.Tensor, lam: torch.Tensor, o: torch.Tensor, lse: torch.Tensor | None, sm_scale: float,
        norm_weight: torch.Tensor | None = None, norm_eps: float = 1e-5, out_scale: float = 1.0, stream=None):
    """Enqueue differential attention for the current plan of `ws`.

    q, o [tokens, Hq, 128]; caches [pages, page_size, Hkv, 128]; lam fp32 [Hq];
    lse fp32 [tokens, Hq, 2] or None; norm_weight fp32 [128] or None."""
    if _run is None:
        load()
    dtype, index = q.dtype, q.get_device()
    code = _DTYPE.get(dtype)
    if code is None or k_cache.dtype is not dtype or v_cache.dtype is not dtype or o.dtype is not dtype:
        raise TypeError("q, k, v and o must share one 16-bit dtype")
    if kv_indices_dev.dtype is not torch.int32 or not kv_indices_dev.is_contiguous():
        raise TypeError("kv_indices must be a contiguous int32 device tensor")
    if not (index == k_cache.get_device() == v_cache.get_device() == kv_indices_dev.get_device() == o.get_device() ==
            lam.get_device() == ws.int_ws.get_device()):
        raise TypeError("all tensors must be on one device")
    if lam.dtype is not torch.float32 or not lam.is_contiguous():
        raise TypeError("lam must be contiguous fp32")
    hq = info.num_qo_heads
    shape, cache = q.shape, k_cache.shape
    tokens = shape[0]
    qt, qh, qd = q.stride()
    ot, oh, od = o.stride()
    kp, ks, kh, kd = k_cache.stride()
    vp, vs, vh, vd = v_cache.stride()
    if shape != (tokens, hq, 128) or o.shape != shape or qd != 1 or od != 1:
        raise ValueError("q and o are [tokens, num_qo_heads, 128], the last dimension contiguous")
    if cache != (cache[0], info.page_size, info.num_kv_heads, 128) or v_cache.shape != cache or kd != 1 or vd != 1:
        raise ValueError("the caches are [pages, page_size, num_kv_heads, 128], the last dimension contiguous")
    if lam.numel() != hq:
        raise ValueError("lam has num_qo_heads entries")
    w = 0
    if norm_weight is not None:
        if norm_weight.dtype is not torch.float32 or not norm_weight.is_contiguous() or norm_weight.numel() != 128 or \
                norm_weight.get_device() != index:
            raise ValueError("norm_weight is 128 contiguous fp32 values on the tensors' device")
        w = norm_weight.data_ptr()
    lse_ptr = 0
    if lse is not None:
        if lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != index or \
                lse.shape != (tokens, hq, 2):
            raise ValueError("lse is a contiguous fp32 [tokens, num_qo_heads, 2] tensor")
        lse_ptr = lse.data_ptr()
    _call(_run, _ARGS.pack(ctypes.addressof(info), q.data_ptr(), qt, qh, tokens, k_cache.data_ptr(), kp, ks, kh,
                           v_cache.data_ptr(), vp, vs, vh, cache[0], kv_indices_dev.data_ptr(), lam.data_ptr(), w,
                           o.data_ptr(), ot, oh, lse_ptr, code, ws.int_ws.data_ptr(), ws.float_ws.data_ptr(),
                           sm_scale, norm_eps, out_scale, 0.0),
          index, stream, "fi_batch_paged_attention_run_differential")
