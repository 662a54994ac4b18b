// diff.cu -- C-ABI entry point of differential attention.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fi_diff.h"
#include "diff_launch.h"

namespace fi {

bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const uint64_t* dims,
              const int64_t* strides_elems, const uint32_t* box, CUtensorMapSwizzle swizzle);  // attention.cu

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool stride_ok(int64_t elems) { return elems > 0 && (elems * 2) % 16 == 0; }

}  // namespace
}  // namespace fi

using namespace fi;

extern "C" fi_status fi_batch_paged_attention_run_differential(
    const fi_plan_info* info, const void* q, int64_t q_stride_tok, int64_t q_stride_head, int32_t q_num_tokens,
    const void* k_cache, const int64_t k_strides[3], const void* v_cache, const int64_t v_strides[3],
    int32_t num_pages, const int32_t* kv_indices_dev, const float* lambda, const float* norm_weight, float norm_eps,
    float out_scale, void* o, int64_t o_stride_tok, int64_t o_stride_head, float* lse, fi_dtype dtype,
    float sm_scale, void* int_workspace_dev, void* float_workspace_dev, void* stream) {
  if (!info || !q || !o || !int_workspace_dev || !lambda) return FI_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !k_strides || !v_strides || !kv_indices_dev || num_pages < 1) return FI_ERR_INVALID_ARG;
  if (!(info->variant & 8) || info->num_ctas < 1 || q_num_tokens < 1) return FI_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale) || !std::isfinite(out_scale)) return FI_ERR_INVALID_ARG;
  if (norm_weight && !(norm_eps >= 0.f && std::isfinite(norm_eps))) return FI_ERR_INVALID_ARG;
  if (info->num_partial_rows > 0 && !float_workspace_dev) return FI_ERR_INVALID_ARG;
  if (info->head_dim != kHeadDim) return FI_ERR_UNSUPPORTED;
  if (dtype != FI_FP16 && dtype != FI_BF16) return FI_ERR_UNSUPPORTED;
  if (info->num_kv_heads < 1 || info->num_qo_heads % info->num_kv_heads) return FI_ERR_UNSUPPORTED;
  const int P = info->page_size;
  if (P < 1 || P > 128 || (P & (P - 1))) return FI_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(o) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(int_workspace_dev) ||
      (float_workspace_dev && !aligned16(float_workspace_dev)) ||
      ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(lambda) |
        reinterpret_cast<uintptr_t>(norm_weight) | reinterpret_cast<uintptr_t>(kv_indices_dev)) & 3u))
    return FI_ERR_ALIGNMENT;
  if (!stride_ok(q_stride_tok) || !stride_ok(q_stride_head) || !stride_ok(o_stride_tok) || !stride_ok(o_stride_head))
    return FI_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if (!stride_ok(k_strides[i]) || !stride_ok(v_strides[i])) return FI_ERR_ALIGNMENT;

  DiffParams dp;
  std::memset(&dp, 0, sizeof dp);
  RunParams& p = dp.run;
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride_tok = q_stride_tok;
  p.q_stride_head = q_stride_head;
  p.o = static_cast<uint16_t*>(o);
  p.o_stride_tok = o_stride_tok;
  p.o_stride_head = o_stride_head;
  p.lse = lse;
  p.iws = static_cast<int32_t*>(int_workspace_dev);
  p.fws = static_cast<float*>(float_workspace_dev);
  p.partial_o_offset = fi_partial_o_offset(info->max_partial_rows);
  p.max_partial_rows = p.fws ? info->max_partial_rows : 0;
  p.q_num_tokens = q_num_tokens;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.num_qo_heads = info->num_qo_heads;
  p.num_kv_heads = info->num_kv_heads;
  p.group = info->num_qo_heads / info->num_kv_heads;
  KvCache& kc = p.kv[0];
  kc.kv_indices = kv_indices_dev;
  kc.page_size = P;
  while ((1 << kc.log2_page) < P) ++kc.log2_page;
  kc.num_pages = num_pages;
  dp.lambda = lambda;
  dp.norm_w = norm_weight;
  dp.norm_eps = norm_eps;
  dp.out_scale = out_scale;
  dp.k = static_cast<const uint16_t*>(k_cache);
  dp.v = static_cast<const uint16_t*>(v_cache);
  for (int i = 0; i < 3; ++i) {
    dp.k_strides[i] = k_strides[i];
    dp.v_strides[i] = v_strides[i];
  }
  if (P >= kMinTmaPage) {
    const CUtensorMapDataType tt =
        dtype == FI_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t kd[4] = {uint64_t(kHeadDim), uint64_t(info->num_kv_heads), uint64_t(P), uint64_t(num_pages)};
    const int64_t ks[3] = {k_strides[2], k_strides[1], k_strides[0]};  // head, slot, page
    const int64_t vs[3] = {v_strides[2], v_strides[1], v_strides[0]};
    const uint32_t kb[4] = {64u, 1u, uint32_t(P), 1u};
    if (!make_map(&kc.tm_k, tt, k_cache, 4, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&kc.tm_v, tt, v_cache, 4, kd, vs, kb, CU_TENSOR_MAP_SWIZZLE_128B))
      return FI_ERR_UNSUPPORTED;
    kc.tc = kTileM % p.group == 0 ? 1 : 0;
    if (kc.tc) {
      const uint64_t qd[3] = {uint64_t(kHeadDim), uint64_t(info->num_qo_heads), uint64_t(q_num_tokens)};
      const int64_t qs[2] = {q_stride_head, q_stride_tok}, os[2] = {o_stride_head, o_stride_tok};
      const uint32_t qb[3] = {64u, uint32_t(p.group), uint32_t(kTileM / p.group)};
      if (!make_map(&p.tm_q, tt, q, 3, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B) ||
          !make_map(&p.tm_o, tt, o, 3, qd, os, qb, CU_TENSOR_MAP_SWIZZLE_128B))
        return FI_ERR_UNSUPPORTED;
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool mask = (info->variant & 2) != 0;
  const cudaError_t e = dtype == FI_BF16 ? (mask ? launch_diff<__nv_bfloat16, true>(dp, info->num_ctas, s)
                                                 : launch_diff<__nv_bfloat16, false>(dp, info->num_ctas, s))
                                         : (mask ? launch_diff<__half, true>(dp, info->num_ctas, s)
                                                 : launch_diff<__half, false>(dp, info->num_ctas, s));
  return e == cudaSuccess ? FI_OK : FI_ERR_CUDA;
}
