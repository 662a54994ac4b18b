/*
 * fi_step.h -- C ABI of the operators around an attention step: the page
 * tables and slot maps of the step built on the GPU, and rotary positions
 * applied to queries and keys, with the keys and values written into the
 * paged cache.  Same conventions as fi.h (plain C types, HOST marks host
 * pointers, a stream is a cudaStream_t passed as void*, every entry returns an
 * fi_status, the caller owns every buffer; no allocation, no synchronisation,
 * no host copy, so every call can be captured in a CUDA graph).
 *
 * The calls take their many arguments in a struct of 8-byte fields (pointers
 * and int64_t), which a binding can fill in one go; the struct itself is read
 * before the call returns.
 */
#ifndef FI_STEP_H_
#define FI_STEP_H_

#include <stddef.h>
#include <stdint.h>

#include "fi.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FI_STEP_MAX_BATCH 8192
#define FI_STEP_COUNTS 8

/*
 * fi_build_step_tables -- from the lengths of a step's requests, on the GPU:
 * new pages from a free list into the requests' block table, and the page
 * table, positions and slot map that attention and the cache append read.
 *
 * Request b has qo_lens[b] new tokens and kv_lens[b] keys with them, so it
 * held kv_lens[b] - qo_lens[b] keys before the step.  With n(x) =
 * ceil(x / page_size), its row block_table[b * block_table_stride + p] holds
 * the ids of its n(old) pages; the step's n(kv_lens[b]) - n(old) further pages
 * are the next ids of free_pages from entry *free_head on, request after
 * request, and are written into the row.  Then, all int32 device arrays:
 *   qo_indptr [batch + 1]    prefix sums of qo_lens
 *   kv_indptr [batch + 1]    prefix sums of the page counts
 *   last_page_len [batch]    keys in the last page (0 without a page)
 *   kv_indices [max_pages]   page ids, request after request; entries past the
 *                            last are left as they were
 *   positions [max_tokens]   position of each new token in its request
 *   slots [max_tokens]       page id * page_size + slot of each new token (-1
 *                            for a negative page id or past INT32_MAX);
 *                            tokens past the last get position 0 and slot -1,
 *                            so that a step padded to a captured size appends
 *                            nothing for them
 *   counts [FI_STEP_COUNTS]  {tokens, pages, pages taken, *free_head + pages
 *                            taken, fi_status, 0, 0, 0}
 * counts[3] is the free_head of the next step (another counts array: counts
 * must not hold the word that free_head points to).
 *
 * Host checks: null pointers, 1 <= batch <= FI_STEP_MAX_BATCH, page_size a
 * power of two in [1, 128], sizes (FI_ERR_INVALID_ARG, FI_ERR_UNSUPPORTED).
 * max_pages and max_tokens may be 0 (the arrays are then not read).
 * free_pages and free_head may be NULL with num_free 0 (no page is given out).
 * Checked on the device: 0 <= qo_lens[b] <= kv_lens[b] <=
 * block_table_width * page_size (counts[4] = FI_ERR_INVALID_ARG otherwise),
 * and that the pages and tokens fit max_pages and max_tokens and the free list
 * holds what is taken (FI_ERR_CAPACITY).  Then counts[0..2] is what the step
 * would need (at most INT32_MAX), counts[3] = *free_head, every token gets
 * position 0 and slot -1 (so that an append behind the call in a captured step
 * writes nothing to the cache) and nothing else is written.
 */
typedef struct {
    const int32_t* qo_lens;
    const int32_t* kv_lens;
    int64_t batch, page_size;
    int32_t* block_table;
    int64_t block_table_stride, block_table_width;
    const int32_t* free_pages;
    int64_t num_free;
    const int32_t* free_head;
    int32_t* qo_indptr;
    int32_t* kv_indptr;
    int32_t* last_page_len;
    int32_t* kv_indices;
    int64_t max_pages;
    int32_t* positions;
    int32_t* slots;
    int64_t max_tokens;
    int32_t* counts;
} fi_step_tables_args;

fi_status fi_build_step_tables(const fi_step_tables_args* args, void* stream);

#define FI_ROTARY_MAX_PAIRS 128

/* How the rate f_i = theta^(-2i / rot_dim) (radians per position) of pair i is
 * changed for contexts longer than the L = original_positions that a model
 * was trained on, by a factor s:
 *   NONE      f_i
 *   LINEAR    f_i / s
 *   NTK       theta becomes theta * s^(rot_dim / (rot_dim - 2))
 *   BY_PARTS  with r_i = L f_i / (2 pi) turns over the old length: f_i where
 *             r_i >= high_turns, f_i / s where r_i <= low_turns, in between
 *             linear in r_i
 *   YARN      the same ends, in between linear in the pair's number i, from
 *             floor(d(high_turns)) to ceil(d(low_turns)) with d(r) =
 *             rot_dim ln(L / (2 pi r)) / (2 ln theta), clipped to
 *             [0, rot_dim - 1]; cos and sin are multiplied by 0.1 ln(s) + 1 */
typedef enum {
    FI_ROTARY_NONE = 0,
    FI_ROTARY_LINEAR = 1,
    FI_ROTARY_NTK = 2,
    FI_ROTARY_BY_PARTS = 3,
    FI_ROTARY_YARN = 4
} fi_rotary_scaling;

typedef struct {
    int32_t head_dim;           /* a multiple of 8, at most 256 */
    int32_t rot_dim;            /* the first rot_dim dims are rotated, the others copied: a multiple of 16,
                                   at most head_dim */
    int32_t interleaved;        /* 0: dims i and i + rot_dim / 2 form pair i; 1: dims 2i and 2i + 1 */
    int32_t scaling;            /* fi_rotary_scaling */
    double theta;               /* > 1 */
    double factor;              /* s >= 1 */
    int32_t original_positions; /* L > 0 (BY_PARTS, YARN) */
    float low_turns;            /* BY_PARTS, YARN: 0 < low_turns < high_turns */
    float high_turns;
    float amplitude;            /* > 0: factor on cos and sin; 0: 1, or YARN's own */
} fi_rotary_config;

/* Plain data made by fi_rotary_setup and passed to the calls below.  turns[i]
 * is pair i's rate in turns per position as a 64-bit binary fraction, so that
 * position * turns[i] modulo 2^64 is the exact fraction of a turn at any
 * int32 position. */
typedef struct {
    int32_t head_dim, rot_dim, interleaved, reserved;
    float amplitude;
    float reserved2;
    uint64_t turns[FI_ROTARY_MAX_PAIRS];
} fi_rotary;

/* Rows [tokens, heads, dim] of an operand: strides in elements, the last
 * dimension contiguous. */
typedef struct {
    void* data; /* an input is not written */
    int64_t stride_tok, stride_head;
} fi_rows;

/* HOST only (no CUDA call).  FI_ERR_INVALID_ARG for values outside the ranges
 * above, FI_ERR_UNSUPPORTED for dims outside them. */
fi_status fi_rotary_setup(const fi_rotary_config* cfg, fi_rotary* out);

/*
 * fi_rotary_apply -- rotate q and k rows to their positions: pair (a, b) of
 * token t becomes (a c - b s, b c + a s) with c and s the cos and sin of
 * positions[t] * f_i times the amplitude; computed in fp32 from an exact
 * angle and rounded once.
 *   q_in, q_out [num_tokens, num_q_heads, head_dim]; q_out may be q_in (same
 *   strides), otherwise they must not overlap.  num_q_heads may be 0 (q not
 *   read).
 *   k_in, k_out [num_tokens, num_kv_heads, head_dim] likewise; num_kv_heads
 *   may be 0.
 *   positions int32 [num_tokens], device; any value.
 * dtype FI_FP16 or FI_BF16; base pointers and strides are multiples of 16
 * bytes.  An input may be broadcast (stride 0).  An output's rows must be apart,
 * its dimensions nested (the larger stride at least what the other dimension
 * spans): refused otherwise (FI_ERR_INVALID_ARG), as are an output that overlaps
 * its input at the same strides without being it, and one that begins where its
 * input does at other strides.  Other overlaps are not looked for.
 * num_tokens 0 does nothing (no pointer is read or checked).
 */
typedef struct {
    const fi_rotary* rotary;
    const int32_t* positions;
    int64_t num_tokens;
    fi_rows q_in, q_out;
    int64_t num_q_heads;
    fi_rows k_in, k_out;
    int64_t num_kv_heads, dtype;
} fi_rotary_apply_args;

fi_status fi_rotary_apply(const fi_rotary_apply_args* args, void* stream);

/*
 * fi_rotary_append -- one launch for a step's new tokens: q rotated as by
 * fi_rotary_apply, k rotated into the paged cache and v copied into it, token
 * t at slot slots[t] (page slots[t] / page_size, slot slots[t] % page_size).
 *   k_cache [num_pages, page_size, num_kv_heads, head_dim] and
 *   v_cache [num_pages, page_size, num_kv_heads, v_dim], own strides k_strides
 *   and v_strides (page, slot, head; elements); v_dim a multiple of 8, at most
 *   512 (a latent cache has one head: k its rotated key, v its latent row).
 *   slots int32 [num_tokens], device.  A token whose slot is negative or not
 *   below num_pages * page_size (padding) writes nothing to the caches; its q
 *   is rotated.  Two tokens of one call must not have the same slot.
 *   num_q_heads may be 0; v_in NULL with v_dim 0 appends keys alone.
 * Other arguments, dtypes, alignment and output rows (of the caches too: pages,
 * slots and heads nested) as for fi_rotary_apply; page_size a power of two in
 * [1, 128].  The caches must not overlap the inputs.
 */
typedef struct {
    const fi_rotary* rotary;
    const int32_t* positions;
    const int32_t* slots;
    int64_t num_tokens;
    fi_rows q_in, q_out;
    int64_t num_q_heads;
    fi_rows k_in, v_in;
    int64_t v_dim, num_kv_heads;
    void* k_cache;
    int64_t k_strides[3];
    void* v_cache;
    int64_t v_strides[3];
    int64_t page_size, num_pages, dtype;
} fi_rotary_append_args;

fi_status fi_rotary_append(const fi_rotary_append_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FI_STEP_H_ */
