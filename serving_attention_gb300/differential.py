"""Python binding of differential attention over the paged cache (include/fi_diff.h).

Argument marshalling only, like the package's other bindings; there is no
fallback.  The plan is the ordinary one, made with differential=1:

    cfg = default_plan_config(0, differential=1)
    ws = Workspace(cfg)
    info = plan(ws, qo_indptr, kv_indptr, kv_indices, last_page_len, 32, 8, 128, 16, causal=1)
    differential.run(ws, info, q, k_cache, v_cache, kv_indices_dev, lam, o, lse, sm_scale)
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _DTYPE, PlanInfo, Workspace, _check, _stream_ptr, load as _load_lib

EXPORTS = ["fi_batch_paged_attention_run_differential"]

_bound = False
_Strides = ctypes.c_int64 * 3


def load() -> ctypes.CDLL:
    global _bound
    lib = _load_lib()
    if not _bound:
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        lib.fi_batch_paged_attention_run_differential.argtypes = [
            ctypes.POINTER(PlanInfo), vp, i64, i64, i32, vp, vp, vp, vp, i32, vp, vp, vp, f32, f32, vp, i64, i64, vp,
            ctypes.c_int, f32, vp, vp, vp]
        lib.fi_batch_paged_attention_run_differential.restype = ctypes.c_int
        _bound = True
    return lib


def _on_device(device: torch.device):
    """Launches go to the tensors' device, whichever is current."""
    if device.type != "cuda":
        raise TypeError("the tensors must be on a CUDA device")
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def run(ws: Workspace, info: PlanInfo, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
        kv_indices_dev: torch.Tensor, lam: torch.Tensor, o: torch.Tensor, lse: torch.Tensor | None, sm_scale: float,
        norm_weight: torch.Tensor | None = None, norm_eps: float = 1e-5, out_scale: float = 1.0, stream=None):
    """Enqueue differential attention for the current plan of `ws`.

    q, o [tokens, Hq, 128]; caches [pages, page_size, Hkv, 128]; lam fp32 [Hq];
    lse fp32 [tokens, Hq, 2] or None; norm_weight fp32 [128] or None."""
    lib = load()
    dtype = _DTYPE.get(q.dtype)
    if dtype is None or not (q.dtype == k_cache.dtype == v_cache.dtype == o.dtype):
        raise TypeError("q, k, v and o must share one 16-bit dtype")
    if kv_indices_dev.dtype != torch.int32 or not kv_indices_dev.is_contiguous():
        raise TypeError("kv_indices must be a contiguous int32 device tensor")
    f32 = (lam,) if norm_weight is None else (lam, norm_weight)
    if any(t.dtype != torch.float32 or not t.is_contiguous() for t in f32):
        raise TypeError("lam and norm_weight must be contiguous fp32")
    device = q.device
    if any(t.device != device for t in (k_cache, v_cache, kv_indices_dev, o, ws.int_ws, *f32)):
        raise TypeError("all tensors must be on one device")
    hq, hkv, tokens = info.num_qo_heads, info.num_kv_heads, q.shape[0]
    if q.shape != (tokens, hq, 128) or o.shape != q.shape or q.stride(2) != 1 or o.stride(2) != 1:
        raise ValueError("q and o are [tokens, num_qo_heads, 128], the last dimension contiguous")
    cache = (k_cache.shape[0], info.page_size, hkv, 128)
    if k_cache.shape != cache or v_cache.shape != cache or k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
        raise ValueError("the caches are [pages, page_size, num_kv_heads, 128], the last dimension contiguous")
    if lam.numel() != hq or (norm_weight is not None and norm_weight.numel() != 128):
        raise ValueError("lam has num_qo_heads entries and norm_weight 128")
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != device or
                            lse.shape != (tokens, hq, 2)):
        raise ValueError("lse is a contiguous fp32 [tokens, num_qo_heads, 2] tensor")
    with _on_device(device):
        st = lib.fi_batch_paged_attention_run_differential(
            ctypes.byref(info), q.data_ptr(), q.stride(0), q.stride(1), tokens, k_cache.data_ptr(),
            _Strides(*k_cache.stride()[:3]), v_cache.data_ptr(), _Strides(*v_cache.stride()[:3]), cache[0],
            kv_indices_dev.data_ptr(), lam.data_ptr(), norm_weight.data_ptr() if norm_weight is not None else None,
            norm_eps, out_scale, o.data_ptr(), o.stride(0), o.stride(1), lse.data_ptr() if lse is not None else None,
            dtype, sm_scale, ws.int_ws.data_ptr(), ws.float_ws.data_ptr(), _stream_ptr(stream))
    _check(st, "fi_batch_paged_attention_run_differential")
