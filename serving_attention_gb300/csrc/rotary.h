// rotary.h -- rows of queries, keys and values that the append kernels read and
// write: their descriptors, conversions and host checks.
#pragma once
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <utility>

#include "../../include/fi_step.h"
#include "ptx.cuh"

namespace fi {

struct RotaryRows {  // rows of one operand: token t (or cache slot), head h
  const uint16_t* in;
  int64_t in_tok, in_head;
  uint16_t* out;
  int64_t out_tok, out_head;  // out_tok: elements per token, or per page with slots
  int64_t out_slot;
  int32_t heads;
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
  const float2 a = Elem<T>::to_float2(u.x), b = Elem<T>::to_float2(u.y), c = Elem<T>::to_float2(u.z),
               d = Elem<T>::to_float2(u.w);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y; f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(Elem<T>::from_float2(f[0], f[1]), Elem<T>::from_float2(f[2], f[3]),
                    Elem<T>::from_float2(f[4], f[5]), Elem<T>::from_float2(f[6], f[7]));
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool stride_ok(int64_t elems) { return elems >= 0 && elems % 8 == 0; }

inline fi_status check_rotary(const fi_rotary* rot, int64_t num_tokens, int64_t num_q_heads, int64_t num_kv_heads,
                              int64_t dtype) {
  if (!rot || num_tokens < 0 || num_tokens > INT32_MAX || num_q_heads < 0 || num_kv_heads < 0)
    return FI_ERR_INVALID_ARG;
  if (rot->head_dim < 16 || rot->head_dim > 2 * FI_ROTARY_MAX_PAIRS || rot->head_dim % 8 || rot->rot_dim < 16 ||
      rot->rot_dim > rot->head_dim || rot->rot_dim % 16 || (rot->interleaved != 0 && rot->interleaved != 1))
    return FI_ERR_UNSUPPORTED;
  if (num_q_heads > 65536 || num_kv_heads > 65536) return FI_ERR_UNSUPPORTED;
  return dtype == FI_FP16 || dtype == FI_BF16 ? FI_OK : FI_ERR_UNSUPPORTED;
}

inline bool rows_ok(const fi_rows& r) {
  return aligned(r.data, 16) && stride_ok(r.stride_tok) && stride_ok(r.stride_head);
}

// Rows that are written: no two of them in one place.  The dimensions of more
// than one entry are nested: each one's stride is at least what those of smaller
// strides span.  (Sorts the dimensions; one of a single entry goes last.)
template <int N>
bool nested(int64_t (&size)[N], int64_t (&stride)[N], int64_t dim) {
  for (int i = 0; i < N; ++i)
    if (size[i] < 2) stride[i] = INT64_MAX;
  for (int i = 1; i < N; ++i)
    for (int j = i; j > 0 && stride[j] < stride[j - 1]; --j) {
      std::swap(stride[j], stride[j - 1]);
      std::swap(size[j], size[j - 1]);
    }
  int64_t span = dim, more;
  for (int i = 0; i < N && size[i] > 1; ++i)
    if (stride[i] < span || __builtin_mul_overflow(stride[i], size[i] - 1, &more) ||
        __builtin_add_overflow(span, more, &span))
      return false;
  return true;
}

// The rows of an input and an output are the same (in place) or do not meet.
// At the same strides that is exact: rows i1 and i0 places apart in the outer
// and the inner dimension meet if that is less than dim elements from how far
// the two are apart.  Other strides are left to the caller.
inline bool output_ok(const fi_rows& in, const fi_rows& out, int64_t tokens, int64_t heads, int64_t dim) {
  int64_t size[2] = {tokens, heads}, stride[2] = {out.stride_tok, out.stride_head};
  if (!nested(size, stride, dim)) return false;
  const bool same = (tokens < 2 || in.stride_tok == out.stride_tok) && (heads < 2 || in.stride_head == out.stride_head);
  if (in.data == out.data) return same;
  if (!same) return true;
  const int64_t apart = (reinterpret_cast<intptr_t>(out.data) - reinterpret_cast<intptr_t>(in.data)) / 2;
  auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0 ? 1 : 0); };
  const int64_t k1 = floor_div(apart, stride[1]);
  for (int64_t i1 = k1; i1 <= k1 + 1; ++i1) {  // no other can: the rows of one place span less than a stride
    if (i1 <= -size[1] || i1 >= size[1]) continue;
    const int64_t left = apart - i1 * stride[1], k0 = floor_div(left, stride[0]);
    for (int64_t i0 = k0; i0 <= k0 + 1; ++i0)
      if (i0 > -size[0] && i0 < size[0] && std::abs(left - i0 * stride[0]) < dim) return false;
  }
  return true;
}
inline bool cache_ok(const int64_t strides[3], int64_t pages, int64_t page_size, int64_t heads, int64_t dim) {
  int64_t size[3] = {pages, page_size, heads}, stride[3] = {strides[0], strides[1], strides[2]};
  return nested(size, stride, dim);
}

inline RotaryRows rows_of(const fi_rows& in, const fi_rows& out, int64_t heads) {
  return {static_cast<const uint16_t*>(in.data), in.stride_tok, in.stride_head, static_cast<uint16_t*>(out.data),
          out.stride_tok, out.stride_head, 0, int32_t(heads)};
}

inline RotaryRows rows_to_cache(const fi_rows& in, void* cache, const int64_t strides[3], int64_t heads) {
  return {static_cast<const uint16_t*>(in.data), in.stride_tok, in.stride_head, static_cast<uint16_t*>(cache),
          strides[0], strides[2], strides[1], int32_t(heads)};
}

// What fi_rotary_append asks of its arguments (no tokens: the shapes alone).
inline fi_status check_append(const fi_rotary_append_args* x) {
  if (!x) return FI_ERR_INVALID_ARG;
  const fi_status st = check_rotary(x->rotary, x->num_tokens, x->num_q_heads, x->num_kv_heads, x->dtype);
  if (st != FI_OK) return st;
  const int64_t P = x->page_size;
  if (x->v_dim < 0 || x->v_dim > 512 || x->v_dim % 8 || P < 1 || P > 128 || (P & (P - 1))) return FI_ERR_UNSUPPORTED;
  const bool q = x->num_q_heads > 0, v = x->v_dim > 0;
  if (x->num_tokens == 0) return FI_OK;
  if (!x->positions || !x->slots || x->num_kv_heads < 1 || x->num_pages < 1 || x->num_pages > INT32_MAX ||
      !x->k_in.data || !x->k_cache || (q && (!x->q_in.data || !x->q_out.data)) ||
      (v && (!x->v_in.data || !x->v_cache)))
    return FI_ERR_INVALID_ARG;
  if (!aligned(x->positions, 4) || !aligned(x->slots, 4) || !rows_ok(x->k_in) || !aligned(x->k_cache, 16) ||
      (q && (!rows_ok(x->q_in) || !rows_ok(x->q_out))) || (v && (!rows_ok(x->v_in) || !aligned(x->v_cache, 16))))
    return FI_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if (!stride_ok(x->k_strides[i]) || (v && !stride_ok(x->v_strides[i]))) return FI_ERR_ALIGNMENT;
  if ((q && !output_ok(x->q_in, x->q_out, x->num_tokens, x->num_q_heads, x->rotary->head_dim)) ||
      !cache_ok(x->k_strides, x->num_pages, P, x->num_kv_heads, x->rotary->head_dim) ||
      (v && !cache_ok(x->v_strides, x->num_pages, P, x->num_kv_heads, x->v_dim)))
    return FI_ERR_INVALID_ARG;
  return FI_OK;
}

// Norm weights of one operand (null: none): pointer, stride per head and eps.
inline fi_status check_weights(const float* w, int64_t stride, int64_t dim) {
  if (!w) return FI_OK;
  if (stride < 0 || (stride > 0 && stride < dim)) return FI_ERR_INVALID_ARG;
  return aligned(w, 16) && stride % 4 == 0 ? FI_OK : FI_ERR_ALIGNMENT;
}
inline bool eps_ok(double eps) { return eps >= 0.0 && std::isfinite(float(eps)); }

}  // namespace fi
