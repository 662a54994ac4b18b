// kv4_layout.h -- where things lie in the 4-bit cache (see fi_kv4.h).
#pragma once
#include <stdint.h>

#include "../../include/fi_kv4.h"

namespace fi {

constexpr int kKv4RowBytes = FI_KV4_HEAD_DIM / 2;
constexpr int kKv4MaxScaleBits = 0x6C00;  // 4096 as fp16

#if defined(__CUDACC__)
#define FI_HD __host__ __device__ __forceinline__
#else
#define FI_HD inline
#endif

FI_HD constexpr int kv4_block_slots(int page_size) { return page_size < FI_KV4_BLOCK ? page_size : FI_KV4_BLOCK; }
FI_HD constexpr int kv4_block_bytes(int slots) { return (132 * slots + 15) / 16 * 16; }
// Offsets in a block of `slots` slots.
FI_HD constexpr int kv4_k_row(int, int slot) { return kKv4RowBytes * slot; }
FI_HD constexpr int kv4_v_row(int slots, int slot) { return kKv4RowBytes * (slots + slot); }
FI_HD constexpr int kv4_k_word(int slots, int slot) { return 2 * kKv4RowBytes * slots + 2 * slot; }
FI_HD constexpr int kv4_v_word(int slots, int slot) { return 2 * kKv4RowBytes * slots + 2 * (slots + slot); }

#undef FI_HD

}  // namespace fi
