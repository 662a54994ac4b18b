// kv4.cu -- C-ABI entry point of attention over the 4-bit cache.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fi_kv4.h"
#include "kv4_layout.h"
#include "kv4_params.h"
#include "rotary.h"

namespace fi {

bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const uint64_t* dims,
              const int64_t* strides_elems, const uint32_t* box, CUtensorMapSwizzle swizzle);  // attention.cu

}  // namespace fi

using namespace fi;

namespace {
inline bool row_stride_ok(int64_t elems) { return elems > 0 && elems % 8 == 0; }
}  // namespace

extern "C" fi_status fi_batch_paged_attention_run_kv4(const fi_kv4_args* a, void* stream) {
  if (!a || !a->info) return FI_ERR_INVALID_ARG;
  const fi_plan_info* info = a->info;
  if (!a->q || !a->o || !a->int_workspace_dev || !a->cache || !a->kv_indices_dev) return FI_ERR_INVALID_ARG;
  if (!(info->variant & 16) || info->num_ctas < 1 || a->q_num_tokens < 1) return FI_ERR_INVALID_ARG;
  if (a->num_pages < 1 || a->num_pages > INT32_MAX || a->q_num_tokens > INT32_MAX) return FI_ERR_INVALID_ARG;
  // masked logits are -inf before they are scaled: a factor of 0, below 0, or
  // one the hardware flushes to 0 would turn them
  const float scale_log2 = a->sm_scale * 1.4426950408889634f;
  if (!std::isnormal(scale_log2) || scale_log2 < 0.f) return FI_ERR_INVALID_ARG;
  if (info->num_partial_rows > 0 && !a->float_workspace_dev) return FI_ERR_INVALID_ARG;
  if (info->head_dim != kHeadDim || (a->dtype != FI_FP16 && a->dtype != FI_BF16)) return FI_ERR_UNSUPPORTED;
  if (info->num_kv_heads < 1 || info->num_qo_heads < 1 || info->num_qo_heads % info->num_kv_heads ||
      info->num_qo_heads / info->num_kv_heads > 16)
    return FI_ERR_UNSUPPORTED;
  const int64_t per_page = int64_t(fi_kv4_page_bytes(info->page_size));
  if (per_page == 0) return FI_ERR_UNSUPPORTED;
  if (!aligned(a->q, 16) || !aligned(a->o, 16) || !aligned(a->cache, 16) || !aligned(a->int_workspace_dev, 16) ||
      !aligned(a->float_workspace_dev, 16) || !aligned(a->lse, 4) || !aligned(a->kv_indices_dev, 4))
    return FI_ERR_ALIGNMENT;
  if (!row_stride_ok(a->q_stride_tok) || !row_stride_ok(a->q_stride_head) || !row_stride_ok(a->o_stride_tok) ||
      !row_stride_ok(a->o_stride_head) || a->cache_strides[0] % 16 || a->cache_strides[1] % 16)
    return FI_ERR_ALIGNMENT;
  if (a->cache_strides[0] < 0 || a->cache_strides[1] < 0) return FI_ERR_INVALID_ARG;

  Kv4Params kp;
  std::memset(&kp, 0, sizeof kp);
  RunParams& p = kp.run;
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
  p.late_merge = info->num_late_merge_units > 0 ? 1 : 0;  // as in the ordinary run
  KvCache& kc = p.kv[0];
  kc.kv_indices = a->kv_indices_dev;
  kc.page_size = info->page_size;
  while ((1 << kc.log2_page) < info->page_size) ++kc.log2_page;
  kc.num_pages = int32_t(a->num_pages);
  kp.cache = static_cast<const uint8_t*>(a->cache);
  kp.page_stride = a->cache_strides[0];
  kp.head_stride = a->cache_strides[1];
  kp.block_slots = kv4_block_slots(info->page_size);
  while ((1 << kp.log2_block) < kp.block_slots) ++kp.log2_block;
  kp.block_bytes = kv4_block_bytes(kp.block_slots);
  kc.tc = kTileM % p.group == 0 ? 1 : 0;  // tiles of whole tokens: Q by boxes
  if (kc.tc) {
    const uint64_t qd[3] = {uint64_t(kHeadDim), uint64_t(info->num_qo_heads), uint64_t(a->q_num_tokens)};
    const int64_t qs[2] = {a->q_stride_head, a->q_stride_tok};
    const uint32_t qb[3] = {64u, uint32_t(p.group), uint32_t(kTileM / p.group)};
    if (!make_map(&p.tm_q, a->dtype == FI_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a->q, 3,
                  qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B))
      return FI_ERR_UNSUPPORTED;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = a->dtype == FI_BF16 ? launch_kv4<__nv_bfloat16>(kp, info->num_ctas, s)
                                      : launch_kv4<__half>(kp, info->num_ctas, s);
  if (e == cudaSuccess && p.late_merge)
    e = a->dtype == FI_BF16 ? launch_late_merge<__nv_bfloat16>(p, 4 * info->num_ctas, s)
                            : launch_late_merge<__half>(p, 4 * info->num_ctas, s);
  return e == cudaSuccess ? FI_OK : FI_ERR_CUDA;
}
