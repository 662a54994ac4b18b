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

extern "C" fi_status fi_batch_paged_attention_run_differential(const fi_differential_args* a, void* stream) {
  if (!a || !a->info) return FI_ERR_INVALID_ARG;
  const fi_plan_info* info = a->info;
  if (!a->q || !a->o || !a->int_workspace_dev || !a->lambda) return FI_ERR_INVALID_ARG;
  if (!a->k_cache || !a->v_cache || !a->kv_indices_dev || a->num_pages < 1) return FI_ERR_INVALID_ARG;
  if (!(info->variant & 8) || info->num_ctas < 1 || a->q_num_tokens < 1) return FI_ERR_INVALID_ARG;
  if (a->num_pages > INT32_MAX || a->q_num_tokens > INT32_MAX) return FI_ERR_INVALID_ARG;
  // masked logits are set to -inf before they are scaled: a factor of 0, below
  // 0, or one the hardware flushes to 0 would turn them
  const float scale_log2 = a->sm_scale * 1.4426950408889634f;
  if (!std::isnormal(scale_log2) || scale_log2 < 0.f || !std::isfinite(a->out_scale)) return FI_ERR_INVALID_ARG;
  if (a->norm_weight && !(a->norm_eps >= 0.f && std::isfinite(a->norm_eps))) return FI_ERR_INVALID_ARG;
  if (info->num_partial_rows > 0 && !a->float_workspace_dev) return FI_ERR_INVALID_ARG;
  if (info->head_dim != kHeadDim) return FI_ERR_UNSUPPORTED;
  if (a->dtype != FI_FP16 && a->dtype != FI_BF16) return FI_ERR_UNSUPPORTED;
  if (info->num_kv_heads < 1 || info->num_qo_heads < 1 || info->num_qo_heads % info->num_kv_heads)
    return FI_ERR_UNSUPPORTED;
  const int P = info->page_size;
  if (P < 1 || P > 128 || (P & (P - 1))) return FI_ERR_UNSUPPORTED;
  if (!aligned16(a->q) || !aligned16(a->o) || !aligned16(a->k_cache) || !aligned16(a->v_cache) ||
      !aligned16(a->int_workspace_dev) || !aligned16(a->float_workspace_dev) ||
      ((reinterpret_cast<uintptr_t>(a->lse) | reinterpret_cast<uintptr_t>(a->lambda) |
        reinterpret_cast<uintptr_t>(a->norm_weight) | reinterpret_cast<uintptr_t>(a->kv_indices_dev)) & 3u))
    return FI_ERR_ALIGNMENT;
  if (!stride_ok(a->q_stride_tok) || !stride_ok(a->q_stride_head) || !stride_ok(a->o_stride_tok) ||
      !stride_ok(a->o_stride_head))
    return FI_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if (!stride_ok(a->k_strides[i]) || !stride_ok(a->v_strides[i])) return FI_ERR_ALIGNMENT;

  DiffParams dp;
  std::memset(&dp, 0, sizeof dp);
  RunParams& p = dp.run;
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_stride_tok = a->q_stride_tok;
  p.q_stride_head = a->q_stride_head;
  p.o = static_cast<uint16_t*>(a->o);
  p.o_stride_tok = a->o_stride_tok;
  p.o_stride_head = a->o_stride_head;
  p.lse = a->lse;
  p.iws = static_cast<int32_t*>(a->int_workspace_dev);
  p.fws = static_cast<float*>(a->float_workspace_dev);
  p.partial_o_offset = fi_partial_o_offset(info->max_partial_rows);
  p.max_partial_rows = p.fws ? info->max_partial_rows : 0;
  p.q_num_tokens = int32_t(a->q_num_tokens);
  p.scale_log2 = scale_log2;
  p.num_qo_heads = info->num_qo_heads;
  p.num_kv_heads = info->num_kv_heads;
  p.group = info->num_qo_heads / info->num_kv_heads;
  KvCache& kc = p.kv[0];
  kc.kv_indices = a->kv_indices_dev;
  kc.page_size = P;
  while ((1 << kc.log2_page) < P) ++kc.log2_page;
  kc.num_pages = int32_t(a->num_pages);
  dp.lambda = a->lambda;
  dp.norm_w = a->norm_weight;
  dp.norm_eps = a->norm_eps;
  dp.out_scale = a->out_scale;
  dp.k = static_cast<const uint16_t*>(a->k_cache);
  dp.v = static_cast<const uint16_t*>(a->v_cache);
  for (int i = 0; i < 3; ++i) {
    dp.k_strides[i] = a->k_strides[i];
    dp.v_strides[i] = a->v_strides[i];
  }
  const CUtensorMapDataType tt =
      a->dtype == FI_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (P >= kMinTmaPage) {
    const uint64_t kd[4] = {uint64_t(kHeadDim), uint64_t(info->num_kv_heads), uint64_t(P), uint64_t(a->num_pages)};
    const int64_t ks[3] = {a->k_strides[2], a->k_strides[1], a->k_strides[0]};  // head, slot, page
    const int64_t vs[3] = {a->v_strides[2], a->v_strides[1], a->v_strides[0]};
    const uint32_t kb[4] = {64u, 1u, uint32_t(P), 1u};
    if (!make_map(&kc.tm_k, tt, a->k_cache, 4, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&kc.tm_v, tt, a->v_cache, 4, kd, vs, kb, CU_TENSOR_MAP_SWIZZLE_128B))
      return FI_ERR_UNSUPPORTED;
  }
  kc.tc = kTileM % p.group == 0 ? 1 : 0;
  if (kc.tc) {
    const uint64_t qd[3] = {uint64_t(kHeadDim), uint64_t(info->num_qo_heads), uint64_t(a->q_num_tokens)};
    const int64_t qs[2] = {a->q_stride_head, a->q_stride_tok}, os[2] = {a->o_stride_head, a->o_stride_tok};
    const uint32_t qb[3] = {64u, uint32_t(p.group), uint32_t(kTileM / p.group)};
    if (!make_map(&p.tm_q, tt, a->q, 3, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&p.tm_o, tt, a->o, 3, qd, os, qb, CU_TENSOR_MAP_SWIZZLE_128B))
      return FI_ERR_UNSUPPORTED;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool mask = (info->variant & 2) != 0;
  const cudaError_t e = a->dtype == FI_BF16 ? (mask ? launch_diff<__nv_bfloat16, true>(dp, info->num_ctas, s)
                                                 : launch_diff<__nv_bfloat16, false>(dp, info->num_ctas, s))
                                         : (mask ? launch_diff<__half, true>(dp, info->num_ctas, s)
                                                 : launch_diff<__half, false>(dp, info->num_ctas, s));
  return e == cudaSuccess ? FI_OK : FI_ERR_CUDA;
}
