/*
 * fi_diff.h -- C ABI of differential attention over the paged cache.  Same
 * conventions as fi.h (plain C types, a stream is a cudaStream_t passed as
 * void*, every entry returns an fi_status, the caller owns every buffer).
 *
 * Differential attention takes the difference of two softmax maps with a
 * learned weight, so that what both maps attend to cancels.  Query row q and
 * key k of a head are halves of 64 dims, q = [q1 | q2], k = [k1 | k2]; values
 * have 128 dims.  Per query row of head h:
 *
 *   S_i = softmax(sm_scale * q_i k_i^T + mask) V          (i = 1, 2)
 *   y   = S_1 - lambda[h] * S_2
 *   o   = out_scale * y                                    norm_weight NULL
 *   o   = out_scale * y / sqrt(mean(y^2) + norm_eps) * norm_weight
 *
 * (the mean over the 128 dims of the head).  The layer's lambda is commonly
 * exp(a1.b1) - exp(a2.b2) + lambda_init with learned vectors, computed once
 * when the weights are loaded, and out_scale 1 - lambda_init.  The caches
 * have the layout of the ordinary run ([pages, page_size, kv_heads, 128], k1
 * and k2 next to each other), so one pass over them serves both maps.
 */
#ifndef FI_DIFF_H_
#define FI_DIFF_H_

#include "fi.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fi_batch_paged_attention_run_differential -- the run of a plan made by
 * fi_plan with fi_plan_config.differential = 1 (FI_ERR_INVALID_ARG for any
 * other plan).  Batches, page tables, causal alignment, sliding window and
 * sink tokens as for fi_batch_paged_attention_run; arguments, layouts,
 * strides, alignment and dtypes too, and
 *   lambda       fp32 [num_qo_heads], device;
 *   norm_weight  fp32 [128], device, or NULL: no norm (norm_eps is then not
 *                read);
 *   sm_scale     positive (a normal fp32 number, its log2(e) multiple too);
 *   out_scale    factor on the output;
 *   lse          fp32 [q_num_tokens, num_qo_heads, 2], contiguous, the natural
 *                log-sum-exp of the two maps; may be NULL.
 * A row with no visible key gets o = 0 and lse = -inf.  Slots past the end of
 * a request's last page may hold anything, NaN included; values of its own that
 * a row's mask hides beside visible ones are read with weight 0 and have to be
 * finite (before a window: up to 127 keys ahead of it).  Page ids outside
 * [0, num_pages) read as zeros.
 *
 * Requests of up to 16 packed rows (query tokens x group) read their keys once.
 * Longer ones run on the tensor cores, tiles of 128 rows that walk their keys
 * twice (three times in a split unit), whatever the rows in them, where the
 * group divides 128; with another group (3, 5, 6, 7, ...) they run 16 rows at a
 * time and are some eight times slower (4 prompts of 1000 queries and 2000 keys:
 * 170 us with 32 query and 8 key heads, 1064 with 24 and 8).
 *
 * A row's partial states take two rows of the float workspace (one per map).
 * Two launches on `stream`: the run and the merge of split units; both read
 * their counts from the workspace, so a captured graph serves later plans.
 * A workspace that holds another kind of plan, or one that does not fit the
 * launch, records FI_ERR_DEVICE_CHECK and nothing is written.
 */
typedef struct { /* 8-byte fields but for the fp32 values at the end */
    const fi_plan_info* info;
    const void* q;
    int64_t q_stride_tok, q_stride_head, q_num_tokens;
    const void* k_cache;
    int64_t k_strides[3];
    const void* v_cache;
    int64_t v_strides[3];
    int64_t num_pages;
    const int32_t* kv_indices_dev;
    const float* lambda;
    const float* norm_weight;
    void* o;
    int64_t o_stride_tok, o_stride_head;
    float* lse;
    int64_t dtype;
    void* int_workspace_dev;
    void* float_workspace_dev;
    float sm_scale, norm_eps, out_scale, reserved;
} fi_differential_args;

fi_status fi_batch_paged_attention_run_differential(const fi_differential_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FI_DIFF_H_ */
