/*
 * fi_kv4.h -- C ABI of the paged cache held in 4 bits: the append that norms,
 * rotates and quantises a step's keys and values into it, attention over it,
 * and rows read back in 16 bits.  Same conventions as fi.h and fi_step.h
 * (plain C types, structs of 8-byte fields, a stream is a cudaStream_t passed
 * as void*, every entry returns an fi_status, the caller owns every buffer; no
 * allocation, no synchronisation, no host copy, so every call can be captured
 * in a CUDA graph).
 *
 * A head of a token is 128 values, held as
 *
 *   value_d = s (n_d - z),   n_d and z from 0 to 15,
 *
 * with s an fp16 from 0 to 4096 whose low four bits are zero; its word is the
 * bits of s with z in those four bits.  s has at most seven significant bits
 * and n - z four, so every value is an fp16 as it stands (and zero is one).
 *
 *   row    64 bytes: dim d in the low (d even) or high nibble of byte d / 2
 *   block  B = min(page_size, 32) slots of one head: B rows of k, B rows of v,
 *          B words (little endian) of k, B words of v, then zero to twelve
 *          bytes up to a multiple of 16
 *   page   of one head: page_size / B blocks after each other,
 *          fi_kv4_page_bytes(page_size) bytes (132 a slot from page size 4 on)
 *   cache  [num_pages, num_kv_heads, fi_kv4_page_bytes] bytes, its page and
 *          head strides free (multiples of 16)
 *
 * The quantiser, every operation rounded once in fp32 and to nearest, even, so
 * that equal inputs give equal bytes everywhere: with lo = min(x, 0) and
 * hi = max(x, 0) over the 128 values (a NaN is passed over),
 *
 *   s   = (hi - lo) * (1/15 in fp32), to fp16, its bits rounded up to a
 *         multiple of 16 and at most 4096's; inv = 1 / s (0 for s = 0)
 *   z   = rint(-lo * inv)               kept within 0 .. 15
 *   n_d = rint(x_d * inv) + z           kept within 0 .. 15 (a NaN: 0)
 *
 * Values beyond 15 * 4096 saturate; rows within 2^-21 of zero become zeros.
 */
#ifndef FI_KV4_H_
#define FI_KV4_H_

#include "fi_step.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FI_KV4_HEAD_DIM 128
#define FI_KV4_BLOCK 32 /* slots of a block, at most */

/* HOST only.  Bytes of one page of one head; 0 unless page_size is a power of
 * two in [1, 128]. */
size_t fi_kv4_page_bytes(int64_t page_size);

/*
 * fi_kv4_append -- one launch for a step's new tokens: q and k normed (where
 * weights are given) and rotated, q written in its own type, k and v quantised
 * into the cache, token t at slot slots[t] (page slots[t] / page_size, slot
 * slots[t] % page_size).
 *   q_in, q_out [num_tokens, num_q_heads, 128], k_in, v_in [num_tokens,
 *     num_kv_heads, 128], dtype FI_FP16 or FI_BF16, strides and alignment as
 *     for fi_rotary_append; q_out may be q_in; num_q_heads may be 0.
 *   rotary      of fi_rotary_setup with head_dim 128, or NULL: no rotation
 *     (positions is then not read).
 *   q_weight, k_weight  fp32 weights of an RMS norm before the rotation, as for
 *     fi_norm_rotary_append (NULL: none).  The sum of a head's squares is
 *     taken in pairs, in one order: dims d and d + 64, then within each group
 *     of 8 dims (e and e + 4, + 2, + 1), then over the 8 groups likewise; the
 *     factor is 1 / sqrt(sum / 128 + eps), and (x * factor) * weight the normed
 *     value.  A pair (a, b) is rotated to (a c - b s, b c + a s), each product
 *     and sum rounded by itself, with c and s the cosf and sinf of half
 *     a turn times pi.
 *   cache_strides  page and head, bytes.
 * A token whose slot is negative or not below num_pages * page_size (padding)
 * writes nothing to the cache; its q is written.  Two tokens of one call must
 * not have the same slot.  The cache must not overlap the inputs; pages and
 * heads are apart and nested (FI_ERR_INVALID_ARG).  num_tokens 0 does nothing.
 */
typedef struct {
    const fi_rotary* rotary;
    const int32_t* positions;
    const int32_t* slots;
    int64_t num_tokens;
    fi_rows q_in, q_out;
    int64_t num_q_heads;
    fi_rows k_in, v_in;
    int64_t num_kv_heads;
    const float* q_weight;
    int64_t q_weight_stride;
    const float* k_weight;
    int64_t k_weight_stride;
    void* cache;
    int64_t cache_strides[2];
    int64_t page_size, num_pages, dtype;
    double eps;
} fi_kv4_append_args;

fi_status fi_kv4_append(const fi_kv4_append_args* args, void* stream);

/*
 * fi_kv4_read -- the values held at num_rows slots, in 16 bits: row i of k_out
 * and v_out [num_rows, num_kv_heads, 128] is what slot slots[i] holds (exact in
 * fp16, rounded once in bf16), zeros for a slot outside the cache.  Either
 * output may have a NULL pointer: not written.  Slots may repeat.  Strides and
 * alignment as above.  Rows of an output are apart and nested, and outputs of the
 * same strides do not meet (FI_ERR_INVALID_ARG); that outputs of other strides do
 * not overlap each other, nor any output the cache, is the caller's to see to.
 */
typedef struct {
    const int32_t* slots;
    int64_t num_rows;
    fi_rows k_out, v_out;
    int64_t num_kv_heads;
    const void* cache;
    int64_t cache_strides[2];
    int64_t page_size, num_pages, dtype;
} fi_kv4_read_args;

fi_status fi_kv4_read(const fi_kv4_read_args* args, void* stream);

/*
 * fi_batch_paged_attention_run_kv4 -- the run of a plan made by fi_plan with
 * fi_plan_config.kv_bits = 4 (FI_ERR_INVALID_ARG for any other plan):
 * O = softmax(sm_scale * Q K^T + mask) V over the values held in the cache, and
 * the natural log-sum-exp.  Batches, page tables, causal alignment, sliding
 * window and sink tokens as for fi_batch_paged_attention_run.
 *   q, o   [q_num_tokens, num_qo_heads, 128], dtype FI_FP16 or FI_BF16
 *     (a q row enters as fp16 times a power of two: exact down to 2^-24
 *     of its largest value, which is finite and, in bf16, below 2^101).
 *   lse    fp32 [q_num_tokens, num_qo_heads], contiguous; may be NULL.
 *   sm_scale  positive (a normal fp32 number, its log2(e) multiple too).
 * Logits, exponentials and sums are fp32.  Weights p_j (in a request of at most 16
 * query tokens times query heads a key head: p_j times the scale s_j of v_j) are
 * rounded to fp16 once: off by at most 2^-11 of themselves or, where that is more, by
 * 2^-36 of the row's largest.  Those requests sum weights times codes and weights
 * times zero points apart, so every dim is off by up to about 2^-14 of
 * sum_j p_j s_j besides, which counts where the rows of weight hold zero in it.
 * A row with no visible key gets o = 0 and lse = -inf.  Slots past the end of a
 * request's last page, and keys that a row's mask hides, may hold any bytes;
 * the words of visible keys hold a finite s.  Page ids outside [0, num_pages)
 * read as zeros.  Rows of q and o behind the plan's last
 * token are left alone.
 *
 * One launch on `stream`, and behind it the merge of split prefill-class units
 * where `info` has any (a graph captured without it merges such units of later
 * plans in the run); both read their counts from the workspace, so a captured
 * graph serves later plans.  A workspace that holds another kind of plan, or one that does not fit
 * the launch, records FI_ERR_DEVICE_CHECK and nothing is written.
 */
typedef struct {
    const fi_plan_info* info;
    const void* q;
    int64_t q_stride_tok, q_stride_head, q_num_tokens;
    const void* cache;
    int64_t cache_strides[2];
    int64_t num_pages;
    const int32_t* kv_indices_dev;
    void* o;
    int64_t o_stride_tok, o_stride_head;
    float* lse;
    int64_t dtype;
    void* int_workspace_dev;
    void* float_workspace_dev;
    float sm_scale, reserved;
} fi_kv4_args;

fi_status fi_batch_paged_attention_run_kv4(const fi_kv4_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FI_KV4_H_ */
