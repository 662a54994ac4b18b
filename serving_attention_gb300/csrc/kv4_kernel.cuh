// kv4_kernel.cuh -- attention over the paged cache held in 4 bits: the kernel and
// its 16-row tiles (kv4_prefill.cuh has the larger ones).
//
// A value is s (n - z) (fi_kv4.h).  A code n in the low nibble of a 16-bit half
// is, as it lies there, the fp16 subnormal n 2^-24, and in the next nibble n
// 2^-20; the tensor cores take subnormals exactly.  So a word of eight codes
// becomes four operand registers with four ANDs and a shift or two, no conversion,
// and scale and zero point stay out of the products:
//
//   q . k_j = s_j ( sum_d q_d n_jd - z_j sum_d q_d )
//   sum_j p_j v_j = sum_j (p_j s_j) n_j - sum_j (p_j s_j) z_j
//
// With q as A and keys as B the rows of an m16n8k16 product would be mostly
// padding; here keys are its 16 rows (S^T = K q^T, eight query rows the
// columns), and O^T = V^T P^T has the dims as rows, so eight query rows cost one
// product per 16 keys and 16 dims.  P^T comes from S^T by one 8 x 8 transpose
// per 8 keys.  The zero point's sum is one more product whose rows all are z.
// A product keeps its addends down to 2^-25 of the largest, a subnormal operand
// counting as the smallest normal number, 2^-14: codes in the lowest bits lose ten
// bits of those.  A value that a row holds as zero (n = z) has to cancel beside the
// others' values of that dim, so v's codes go in three bits up, as n 2^-21 and n
// 2^-17 (120.2 -> 120.8 us of the batch below; all as n 2^-17: 128).  k's stay where
// they are: its logits are off by up to 6 10^-5, three bits up by up to 2 10^-5 and
// the batch 4 us later.
// (tcgen05 would want the codes as 16-bit operands in shared memory, four times
// the bytes that came, for a tile of which 8 of 128 rows are used.)
//
// Twelve warps compute, in three groups.  A long chunk's keys go over all of them
// in consecutive parts; short chunks (up to kKv4GroupKeys keys), whose time is
// latency and not bytes, go to the groups in turn, three at once.  Each computing
// warp has a ring of stages of its own, 32 keys each; four loader warps fill three
// rings each, a lane a ring, one bulk copy a block (keys, values and their words lie
// together), across items.  The only barriers are those that join an item's
// states.
//
// What bounds it: the bytes of a long cache, its 132 a key and head, for up to
// eight query rows a key head; more rows go over the keys again, from L2, at half
// that rate.  Beyond a request's first 8192 keys every further one costs what its
// bytes do at 6.7 TB/s.  64 requests of 512 to 32768 keys, 32 + 8 heads: 121 us,
// 5.4 TB/s (97 us at the copy rate); two of 99991 and 131072 keys, 64 + 8 heads: 48 us
// (35).  One loader warp for all rings brought 4.4 TB/s; eight computing warps that
// widened the codes took 157 us.  Short requests are latency: four of up to 512
// keys, 8 + 2 heads, 6.4 us, of which the launch and the plan's loads are 3; 64 of
// 64 to 512 keys on pages of one token 16 us, at 144 bytes a copy.  The instance for
// blocks below 16 slots, whose addresses are uniform values instead of numbers,
// spills 120 bytes a thread at its 128 registers, and its loaders issue ring after
// ring: the batch takes 229, 221, 182 and 156 us on pages of 1, 2, 4 and 8 tokens.
#pragma once
#include <cfloat>

#include "attention_kernel.cuh"
#include "kv4_layout.h"
#include "kv4_params.h"
#include "kv4_prefill.cuh"

namespace fi {

constexpr int kKv4Threads = 512;       // warpgroup 0: loaders and MMA; 1 .. 3 compute
constexpr int kKv4FirstWarp = 4;       // first computing warp
constexpr int kKv4Warps = 12;          // computing warps of the 16-row tiles
constexpr int kKv4GroupWarps = 4;      // warps of a group
constexpr int kKv4Groups = kKv4Warps / kKv4GroupWarps;
// The longest chunk that one group takes.  152 requests of 1024 keys 41.4 us, with 512 here 57.9; 64 of 128 to 1024 keys 17.7
// and 20.2.
constexpr int kKv4GroupKeys = 1024;
constexpr int kKv4Stage = 32;          // keys of a stage
constexpr int kKv4Depth = 3;           // stages of a ring
constexpr int kKv4StageBytes = 4608;   // 32 blocks of one slot, 144 bytes each
// log2 of the smallest of the small pages that come by bulk copies, a page each; smaller ones in pieces of 16 bytes.
// 64 requests of 512 to 32768 keys, us, by bulk copies and in pieces: pages of two tokens 240 and 221, of four 182 and
// 215, of eight 156 and 210.
constexpr int kKv4BulkLog2 = 2;
constexpr int kKv4Tile = 8;            // packed query rows of a pass
constexpr int kKv4CombRow = 132;       // floats from row to row of a warp's state (128 and 4 against bank conflicts)
constexpr float kKv4NoMax = -FLT_MAX;    // the running maximum before any key
constexpr float kKv4TopUnit = 0x1p100f;  // of the weights: the largest
constexpr float kKv4TopWeight = 32768.f; // of the weights in their unit
constexpr int kKv4Barrier = 8;         // named barriers: of all computing warps, then of each group's
// Registers per thread and warpgroup; each phase's sum is the launch's.
constexpr int kKv4RegsLaunch = 128;
constexpr int kKv4RegsDecode0 = 56, kKv4RegsDecode = 152;
constexpr int kKv4RegsMma = 112, kKv4RegsWiden = 80, kKv4RegsSoftmax = 160;
static_assert(kKv4RegsDecode0 + 3 * kKv4RegsDecode <= 4 * kKv4RegsLaunch, "register split exceeds the launch");
static_assert(kKv4RegsMma + kKv4RegsWiden + 2 * kKv4RegsSoftmax <= 4 * kKv4RegsLaunch,
              "register split exceeds the launch");

struct Kv4DecodeBufs {
  alignas(128) uint8_t ring[kKv4Warps][kKv4Depth][kKv4StageBytes];
  float comb_o[kKv4Warps][kKv4Tile][kKv4CombRow];
  float comb_m[kKv4Warps][kKv4Tile];
  float comb_l[kKv4Warps][kKv4Tile];
  uint32_t good[kKv4Warps][kKv4Depth];  // keys of a stage whose page lies in the cache, a bit each
};

struct alignas(1024) Kv4Smem {
  union {
    Kv4DecodeBufs dec;
    Kv4PrefillBufs pf;
  };
  uint64_t full[kKv4Warps][kKv4Depth], empty[kKv4Warps][kKv4Depth];
  uint64_t raw_full[kKv4RawStages], raw_empty[kKv4RawStages];
  uint64_t q_raw;                   // Q's rows have landed as they are
  uint64_t q_full, q_empty, drain;  // these and the next as in RunSmem
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], o_ready[2], o_free[2], p_full[2][2];
  uint32_t tmem_base;
  volatile int abort;
  int merge_last_pf;
};
constexpr size_t kKv4SmemBytes = sizeof(Kv4Smem);
static_assert(kKv4SmemBytes <= 227 * 1024, "shared memory of the 4-bit kernel exceeds one CTA's limit");

// D += A B with A 16 x 16 and B 16 x 8 in fp16, D in fp32.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
constexpr uint32_t kNibble0 = 0x000F000Fu, kNibble1 = 0x00F000F0u;      // n 2^-24, n 2^-20
constexpr uint32_t kUpNibble0 = 0x00780078u, kUpNibble1 = 0x07800780u;  // n 2^-21, n 2^-17

// A word's two halves: the scale, and the zero point as n 2^-24 (the unit of the products).
__device__ __forceinline__ float word_scale(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w & 0xFFF0u))); }
__device__ __forceinline__ float word_zero(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w & 15u))); }

// ------------------------------------------------------------------- loads

// The warps that share an item: all computing ones, or one group's.
struct Kv4Team {
  int rank, warps, threads, bar;
};
__device__ __forceinline__ Kv4Team kv4_team(int warp, bool all) {
  if (all) return Kv4Team{warp, kKv4Warps, 32 * kKv4Warps, kKv4Barrier};
  const int g = warp / kKv4GroupWarps;
  return Kv4Team{warp % kKv4GroupWarps, kKv4GroupWarps, 32 * kKv4GroupWarps, kKv4Barrier + 1 + g};
}
// A CTA's items [begin, shorts) go to all warps, those behind to the groups in turn.
__device__ __forceinline__ int32_t kv4_next_item(int32_t i, int32_t shorts, int group) {
  if (i + 1 < shorts) return i + 1;
  return i < shorts ? shorts + group : i + kKv4Groups;
}
// First of the n stages that warp `rank` of `warps` takes: as few warps as have one each.
__device__ __forceinline__ int kv4_share(int n, int rank, int warps) {
  const int parts = min(n, warps);
  return rank < parts ? n * rank / parts : n;
}
__device__ __forceinline__ int kv4_stages(const Item& it) { return (it.kv1 - it.kv0 + kKv4Stage - 1) / kKv4Stage; }

// The loaders of the rings: lane u of a loader warp has ring first + u's place in
// its items, and a round issues a stage for every ring whose next slot is free.
// Stages of one or two blocks (kB = 32, 16) are issued by that lane, for all
// rings at once; stages of many small blocks (kB = 0) by the whole warp, ring
// after ring, a bulk copy a lane or in pieces of 16 bytes (a bulk copy for each block
// of one slot kept the copy engine busy longer than the keys did the warps).  Page
// ids are loaded a stage ahead, their lines a line ahead.
template <int kB>
__device__ void kv4_load(const Kv4Params& kp, Kv4Smem& sm, int loader, int32_t off_items, int32_t begin,
                         int32_t shorts, int32_t end) {
  constexpr int kRings = kKv4Warps / kKv4FirstWarp;
  const RunParams& p = kp.run;
  const KvCache& kc = p.kv[0];
  const int lane = threadIdx.x & 31, w = loader * kRings + lane, group = w / kKv4GroupWarps;
  const int log2_slots = kB == 32 ? 5 : kB == 16 ? 4 : kp.log2_block, bytes = kB ? kv4_block_bytes(kB) : kp.block_bytes;
  const int blocks = kKv4Stage >> log2_slots;
  const uint32_t block_keys = (2u << ((1 << log2_slots) - 1)) - 1;  // a block's keys in a stage's bits
  int32_t i = begin - 1, passes = 0, st = 0, st_begin = 0, st_end = 0, kv0 = 0, kv1 = 0, npages = 0;
  const int32_t* pages = nullptr;
  const uint8_t* head = nullptr;
  constexpr int kIds = kB == 16 ? 2 : kB == 32 ? 1 : kRings;
  int32_t ids[kIds];  // of this lane's next stage; kB = 0: this lane's block of each ring's next stage
  // kB = 0: the 16-byte pieces lane, lane + 32, .. of a stage, as block << 16 | place
  constexpr int kPieces = kKv4StageBytes / 16 / 32;
  uint32_t piece[kB ? 1 : kPieces];
  if constexpr (kB == 0)
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int x = lane + 32 * k, b = 16 * x / bytes;
      piece[k] = b < blocks ? uint32_t(b) << 16 | uint32_t(16 * x - b * bytes) : 31u << 16;
    }
  uint32_t issued = 0;
  bool done = lane >= kRings, fresh = false;  // fresh: the next stage's ids are still to be fetched
  long long seen_at = clock64();
  while (true) {
    while (!done && st == st_end) {  // this ring's next item, or the next rows of this one
      fresh = true;
      if (--passes > 0) {
        st = st_begin;
        break;
      }
      i = kv4_next_item(i, shorts, group);
      if (i >= end) {
        done = true;
        fresh = false;
        break;
      }
      const Item it = load_item(p.iws, off_items, i);
      const Kv4Team team = kv4_team(w, i < shorts);
      const int nst = kv4_stages(it);
      st = st_begin = kv4_share(nst, team.rank, team.warps);
      st_end = kv4_share(nst, team.rank + 1, team.warps);
      passes = st < st_end ? (it.row1 - it.row0 + kKv4Tile - 1) / kKv4Tile : 0;
      kv0 = it.kv0;
      kv1 = it.kv1;
      npages = (it.rq.kv_len + kc.page_size - 1) >> kc.log2_page;
      pages = kc.kv_indices + it.rq.page_start;
      head = kp.cache + it.hk * kp.head_stride;
    }
    const int32_t j0 = kv0 + kKv4Stage * st, pg0 = j0 >> kc.log2_page;
    if (fresh && (pg0 & 31) < blocks && pg0 + 32 < npages) prefetch_l1(pages + pg0 + 32);
    if constexpr (kB != 0) {
      if (fresh)
#pragma unroll
        for (int b = 0; b < kIds; ++b) ids[b] = pg0 + b < npages ? __ldg(pages + pg0 + b) : -1;
    } else {
      const uint32_t which = __ballot_sync(0xffffffffu, fresh);
#pragma unroll
      for (int u = 0; u < kRings; ++u) {
        if (!(which >> u & 1u)) continue;
        const int32_t* at = reinterpret_cast<const int32_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(pages), u));
        const int32_t pg = __shfl_sync(0xffffffffu, pg0, u) + lane, n = __shfl_sync(0xffffffffu, npages, u);
        ids[u] = lane < blocks && pg < n ? __ldg(at + pg) : -1;
      }
    }
    fresh = false;
    if (__all_sync(0xffffffffu, done)) break;
    const int slot = issued % kKv4Depth;
    const bool free_slot = !done && mbar_test_wait(&sm.empty[w][slot], ((issued / kKv4Depth) & 1) ^ 1);
    const uint32_t ready = __ballot_sync(0xffffffffu, free_slot);
    if constexpr (kB != 0) {
      if (free_slot) {
        uint8_t* dst = sm.dec.ring[w][slot];
        const uint8_t* src = head + int64_t((j0 & (kc.page_size - 1)) >> log2_slots) * bytes;
        bool ok[kIds];
        uint32_t good = 0;
        int n = 0;
#pragma unroll
        for (int b = 0; b < kIds; ++b) {
          ok[b] = uint32_t(ids[b]) < uint32_t(kc.num_pages) && j0 + b * kB < kv1;
          n += ok[b];
          good |= ok[b] ? block_keys << (b * kB) : 0u;
        }
        sm.dec.good[w][slot] = good;
        mbar_arrive_expect_tx(&sm.full[w][slot], n * bytes);
#pragma unroll
        for (int b = 0; b < kIds; ++b)
          if (ok[b]) bulk_load(dst + b * bytes, src + ids[b] * kp.page_stride, bytes, &sm.full[w][slot]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kRings; ++u) {
        if (!(ready >> u & 1u)) continue;
        const int ring = loader * kRings + u, s = __shfl_sync(0xffffffffu, slot, u);
        const int32_t key = __shfl_sync(0xffffffffu, j0, u), last = __shfl_sync(0xffffffffu, kv1, u);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(head), u));
        const bool ok = uint32_t(ids[u]) < uint32_t(kc.num_pages) && lane < blocks && key + (lane << log2_slots) < last;
        const uint32_t loads = __ballot_sync(0xffffffffu, ok);
        const uint32_t good = __ballot_sync(0xffffffffu, loads >> (lane >> log2_slots) & 1u);
        uint8_t* const dst = sm.dec.ring[ring][s];
        if (log2_slots >= kKv4BulkLog2) {
          if (ok) {
            mbar_arrive_expect_tx(&sm.full[ring][s], bytes);
            bulk_load(dst + lane * bytes, src + ids[u] * kp.page_stride, bytes, &sm.full[ring][s]);
          } else {
            mbar_arrive(&sm.full[ring][s]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kPieces; ++k) {
            const int b = piece[k] >> 16;
            const int32_t id = __shfl_sync(0xffffffffu, ids[u], b);
            if ((loads >> b & 1u) && 16 * (lane + 32 * k) < blocks * bytes)
              cp_async_16(dst + 16 * (lane + 32 * k), src + id * kp.page_stride + (piece[k] & 0xFFFFu), 16);
          }
          cp_async_mbar_arrive_noinc(&sm.full[ring][s]);
        }
        if (lane == 0) {
          sm.dec.good[ring][s] = good;
          mbar_arrive(&sm.full[ring][s]);
        }
      }
    }
    if (free_slot) {
      ++issued;
      ++st;
      fresh = st < st_end;
    }
    if (ready) {
      seen_at = clock64();
    } else {
      __nanosleep(64);
      const int stop = sm.abort != 0 ? 1 : clock64() - seen_at > kWaitBudgetClocks ? 2 : 0;
      const int how = __shfl_sync(0xffffffffu, stop, 0);
      if (how == 2) sm.abort = kStatusTimeout;
      if (how) break;
    }
  }
  // every copy has landed before the CTA leaves
  if (lane < kRings)
    for (uint32_t n = issued > kKv4Depth ? issued - kKv4Depth : 0; n < issued; ++n)
      mbar_wait_drain(&sm.full[w][n % kKv4Depth], (n / kKv4Depth) & 1);
  __syncwarp();
}

// ----------------------------------------------------------------- a stage

// Where this lane (g = lane / 4, t = lane % 4) reads in a stage.  Row r of the
// products is key r ^ (r >> 1 & 1) of a run of 8: the rows of v that lanes t = 0 ..
// 3 of a half warp read then alternate between the two halves of the 128-byte
// lines (two ways instead of four).  The next 8 and the next 16 keys lie the same
// distance on for every lane: numbers known to the compiler for blocks of kB =
// 32 and 16 slots, uniform values otherwise (kB = 0).
template <int kB>
struct Kv4Places {
  uint32_t k, w;      // of key g's row (16 bytes, dims 32 t ..) and word
  uint32_t v[2];      // of the rows of keys 2t and 2t + 1 (8 bytes, dims 16 g ..)
  uint32_t slots, bytes, log2_slots;

  __device__ explicit Kv4Places(const Kv4Params& kp)
      : slots(kB ? kB : kp.block_slots), bytes(kB ? kv4_block_bytes(kB) : kp.block_bytes),
        log2_slots(kB == 32 ? 5 : kB == 16 ? 4 : kp.log2_block) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    auto key = [](int r) { return r ^ ((r >> 1) & 1); };
    auto at = [&](int k, int row) { return (k >> log2_slots) * bytes + (k & (slots - 1)) * row; };
    k = at(key(g), kKv4RowBytes) + 16 * t;
    w = at(key(g), 2) + kv4_k_word(slots, 0);
    for (int u = 0; u < 2; ++u) v[u] = at(key(2 * t + u), kKv4RowBytes) + kv4_v_row(slots, 0) + 8 * g;
  }
  // n keys on (8 or 16 or 24), of rows of `row` bytes
  __device__ __forceinline__ uint32_t on(int n, int row) const {
    return (n >> log2_slots) * bytes + (n & (slots - 1)) * row;
  }
};

// Query row g as an operand column, and the states of rows 2t and 2t + 1.
template <typename T>
struct Kv4Rows {
  uint32_t q[8][2];  // of the 16 dims of step k
  float c[2];        // log2-domain factor of a row's products
  float qs[2];       // sum of the row's operand values
  int lim[2], lo[2];
  float m[2], l[2];
  float o[8][4];     // step i: dims 16 g + 8 (i / 4) + i % 4 (first two) and + 4 (last two)
  float z[4];
  float unit[2];     // what weights times v's scales are multiplied by
};

// This lane's part of query row g of a pass: dims 32 t .. 32 t + 31.
__device__ __forceinline__ void kv4_fetch_rows(const Kv4Params& kp, const Item& it, int pass, uint4 (&u)[4]) {
  const RunParams& p = kp.run;
  const int lane = threadIdx.x & 31, G = p.group;
  const int row = it.row0 + kKv4Tile * pass + (lane >> 2);
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = make_uint4(0u, 0u, 0u, 0u);
  if (row < it.row1) {
    const int tok = row / G;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t(it.rq.qo_start) + tok) * p.q_stride_tok +
                                                      int64_t(it.hk * G + row - tok * G) * p.q_stride_head) +
                       4 * (lane & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = __ldg(src + j);
  }
}

template <typename T>
__device__ __forceinline__ void kv4_set_rows(const Kv4Params& kp, const Item& it, int pass, int causal,
                                             const Variant& var, const uint4 (&u)[4], Kv4Rows<T>& R) {
  const RunParams& p = kp.run;
  const int lane = threadIdx.x & 31, t = lane & 3, G = p.group;
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[8];
    unpack8<T>(u[j], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // the row times a power of two, its largest value in [2^14, 2^15): fp16 has
  // room for the dims in the upper nibbles, which enter with 2^-4
  int ex = int(__float_as_uint(top) >> 23) - 127;  // -127 for rows of zeros
  ex = min(max(ex, -100), 100);
  const float up = __int_as_float((127 + 14 - ex) << 23);
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[8];
    unpack8<T>(u[j], f);
    auto put = [&](uint32_t& dst, float a, float b, float unit) {
      const __half2 h = __floats2half2_rn(a * (up * unit), b * (up * unit));
      dst = *reinterpret_cast<const uint32_t*>(&h);
      const float2 x = __half22float2(h);
      sum += (x.x + x.y) / unit;
    };
    put(R.q[2 * j][0], f[0], f[4], 1.f);
    put(R.q[2 * j][1], f[2], f[6], 1.f);
    put(R.q[2 * j + 1][0], f[1], f[5], 0.0625f);
    put(R.q[2 * j + 1][1], f[3], f[7], 0.0625f);
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  // 2^(ex - 14), and the products' 2^-24; above 0, or a hidden key's -inf would become a NaN
  const float c = fmaxf(p.scale_log2 * __int_as_float((127 + 10 + ex) << 23), FLT_MIN);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    R.qs[h] = __shfl_sync(0xffffffffu, sum, 8 * t + 4 * h);
    R.c[h] = __shfl_sync(0xffffffffu, c, 8 * t + 4 * h);
    const int r = it.row0 + kKv4Tile * pass + 2 * t + h;
    const int pos = it.rq.kv_len - it.rq.qo_len + r / G;
    R.lim[h] = r < it.row1 ? min(causal ? pos : it.rq.kv_len - 1, it.kv1 - 1) : -1;
    R.lo[h] = window_low(var, pos);
    R.m[h] = kKv4NoMax;
    R.l[h] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) R.o[i][e] = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) R.z[e] = 0.f;
  R.unit[0] = R.unit[1] = kKv4TopUnit;
}

// The 32 keys of a stage from key j0 on.  inside: every key of the stage is
// visible to every row and lies in the cache (good: one bit a key).
template <typename T, int kB>
__device__ __forceinline__ void kv4_stage(const uint8_t* stage, const Kv4Places<kB>& at, uint32_t good, int j0, bool inside,
                                          const Variant& var, Kv4Rows<T>& R) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  float s[2][4];
  float vs[2][2];
  uint32_t vz[2][2];  // zero points of v as operand rows: all of them, of two keys
#pragma unroll
  for (int b = 0; b < 2; ++b) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[b][e] = 0.f;
    const uint4 ka = *reinterpret_cast<const uint4*>(stage + at.k + at.on(16 * b, kKv4RowBytes));
    const uint4 kb = *reinterpret_cast<const uint4*>(stage + at.k + at.on(16 * b + 8, kKv4RowBytes));
    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t ha = wa[j] >> 8, hb = wb[j] >> 8;
      mma16(s[b], wa[j] & kNibble0, wb[j] & kNibble0, ha & kNibble0, hb & kNibble0, R.q[2 * j][0], R.q[2 * j][1]);
      mma16(s[b], wa[j] & kNibble1, wb[j] & kNibble1, ha & kNibble1, hb & kNibble1, R.q[2 * j + 1][0],
            R.q[2 * j + 1][1]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* word = stage + at.w + at.on(16 * b + 8 * u, 2);
      const uint32_t w = *reinterpret_cast<const uint16_t*>(word);
      const uint32_t x = *reinterpret_cast<const uint16_t*>(word + 2 * at.slots);
      const float ks = word_scale(w), kz = word_zero(w);
      vs[b][u] = word_scale(x);
      vz[b][u] = transpose8((x & 15u) * 0x00800080u);
#pragma unroll
      for (int h = 0; h < 2; ++h) s[b][2 * u + h] = fmaf(-kz, R.qs[h], s[b][2 * u + h]) * ks;
    }
  }
  if (!inside) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = 16 * b + 8 * u + (g ^ ((g >> 1) & 1)), key = j0 + k;
        const bool there = good >> k & 1u;  // other pages read as zeros
        bool any = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool sees = key <= R.lim[h] && (key >= R.lo[h] || key < var.sink);
          s[b][2 * u + h] = !sees ? -INFINITY : there ? s[b][2 * u + h] : 0.f;
          any |= sees;
        }
        if (!any || !there) vs[b][u] = 0.f;  // a weight of 0 times any bytes, infinities included
      }
  }
  // Weights p s_v as operand columns: keys 2t, 2t + 1 and 2t + 8, 2t + 9 of row g.  fp16 has few powers of two, so their
  // unit follows a row's largest p s_v, whatever scales the values of keys without weight have: where that would pass 2^15
  // it goes to 2^11, so that weights down to 2^-25 of the largest are rounded to 11 bits and those below are off by 2^-36
  // of it at most.  A running maximum moves when the logits pass it by more than 2^8; what is summed so far stays as it is
  // then, and the unit takes the factor.
  float2 x[2][2], sum;
  float pv[2][2][2], past, high;
  auto weigh = [&]() {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        x[b][u] = fma2(make_float2(s[b][2 * u], s[b][2 * u + 1]), make_float2(R.c[0], R.c[1]), make_float2(-R.m[0], -R.m[1]));
        const float2 e = make_float2(ex2(x[b][u].x), ex2(x[b][u].y));
        sum = b + u == 0 ? e : add2(sum, e);
        pv[b][u][0] = e.x * vs[b][u];
        pv[b][u][1] = e.y * vs[b][u];
      }
  };
  auto most = [](float a, float b, float c, float d) { return fmaxf(max3(a, b, c), d); };
  uint32_t w[2][2];
  auto pack = [&]() {
    const float2 unit = make_float2(R.unit[0], R.unit[1]);
    float2 y[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        y[b][u] = mul2(make_float2(pv[b][u][0], pv[b][u][1]), unit);
        w[b][u] = tc::pack2<__half>(y[b][u].x, y[b][u].y);
      }
    high = max3(most(y[0][0].x, y[0][0].y, y[0][1].x, y[0][1].y), fmaxf(y[1][0].x, y[1][0].y), fmaxf(y[1][1].x, y[1][1].y));
  };
  weigh();
  past = max3(most(x[0][0].x, x[0][0].y, x[0][1].x, x[0][1].y), fmaxf(x[1][0].x, x[1][0].y), fmaxf(x[1][1].x, x[1][1].y));
  pack();
  if (__any_sync(0xffffffffu, past > kLazyRescale || high >= kKv4TopWeight)) {
    float back[2], was[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = most(s[0][h], s[0][2 + h], s[1][h], s[1][2 + h]) * R.c[h];
#pragma unroll
      for (int y = 4; y < 32; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
      back[h] = 1.f;
      was[h] = R.unit[h];
      if (top > R.m[h] + kLazyRescale) {
        const float f = ex2(R.m[h] - top);
        R.unit[h] = fminf(R.unit[h] * ex2(top - R.m[h]), kKv4TopUnit);
        R.l[h] *= f;
        back[h] = f;
        R.m[h] = top;
      }
    }
    weigh();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = most(pv[0][0][h], pv[0][1][h], pv[1][0][h], pv[1][1][h]);
#pragma unroll
      for (int y = 4; y < 32; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
      if (top * R.unit[h] >= kKv4TopWeight)  // 2^11 over the power of two of top
        R.unit[h] = __int_as_float(((254 + 11) << 23) - int(__float_as_uint(top) & 0x7F800000u));
      back[h] *= __fdividef(R.unit[h], was[h]);
    }
    pack();
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) R.o[i][e] *= back[e & 1];
#pragma unroll
    for (int e = 0; e < 4; ++e) R.z[e] *= back[e & 1];
  }
  R.l[0] += sum.x;
  R.l[1] += sum.y;
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int u = 0; u < 2; ++u) w[b][u] = transpose8(w[b][u]);
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint32_t b0 = w[b][0], b1 = w[b][1];
    uint2 v4[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      v4[u] = *reinterpret_cast<const uint2*>(stage + at.v[u & 1] + at.on(16 * b + 8 * (u >> 1), kKv4RowBytes));
    mma16(R.z, vz[b][0], vz[b][0], vz[b][1], vz[b][1], b0, b1);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      auto word = [&](int u) { return half ? v4[u].y : v4[u].x; };
      const uint32_t a0 = __byte_perm(word(0), word(1), 0x5410), a1 = __byte_perm(word(0), word(1), 0x7632);
      const uint32_t a2 = __byte_perm(word(2), word(3), 0x5410), a3 = __byte_perm(word(2), word(3), 0x7632);
      const uint32_t l0 = a0 << 3, l1 = a1 << 3, l2 = a2 << 3, l3 = a3 << 3;
      const uint32_t h0 = a0 >> 5, h1 = a1 >> 5, h2 = a2 >> 5, h3 = a3 >> 5;
      mma16(R.o[4 * half], l0 & kUpNibble0, l1 & kUpNibble0, l2 & kUpNibble0, l3 & kUpNibble0, b0, b1);
      mma16(R.o[4 * half + 1], l0 & kUpNibble1, l1 & kUpNibble1, l2 & kUpNibble1, l3 & kUpNibble1, b0, b1);
      mma16(R.o[4 * half + 2], h0 & kUpNibble0, h1 & kUpNibble0, h2 & kUpNibble0, h3 & kUpNibble0, b0, b1);
      mma16(R.o[4 * half + 3], h0 & kUpNibble1, h1 & kUpNibble1, h2 & kUpNibble1, h3 & kUpNibble1, b0, b1);
    }
  }
}

// This warp's state of the pass into shared memory: o (not yet divided), max, sum.
template <typename T>
__device__ __forceinline__ void kv4_put_state(Kv4Smem& sm, int warp, Kv4Rows<T>& R) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float up = __fdividef(131072.f, R.unit[h]);  // 2^17: zero points came in as n 2^-17, codes as that or n 2^-21
    float l = R.l[h];
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    const int row = 2 * t + h;
    if (g == 0) {
      sm.dec.comb_m[warp][row] = R.m[h];
      sm.dec.comb_l[warp][row] = l;
    }
    float* dst = &sm.dec.comb_o[warp][row][16 * g];
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ((i & 1 ? 1.f : 16.f) * R.o[4 * half + i][2 * hi + h] - R.z[h]) * up;
        *reinterpret_cast<float4*>(dst + 8 * half + 4 * hi) = make_float4(x[0], x[1], x[2], x[3]);
      }
  }
}

// One row of a split unit from its chunks' partial states, in chunk order, by a
// warp: lane c has chunk c's log-sum-exp (32 at a time), eight chunks' partial
// outputs are in flight.
template <typename T>
__device__ __forceinline__ void kv4_merge_row(const RunParams& p, const Item& it, int r, int n, int64_t base) {
  const int lane = threadIdx.x & 31, nrows = it.row1 - it.row0;
  const float* lse = p.fws + base + r;
  const float4* part = reinterpret_cast<const float4*>(p.fws + p.partial_o_offset + (base + r) * kHeadDim) + lane;
  const int64_t step = int64_t(nrows) * (kHeadDim / 4);
  float M = -INFINITY;
  for (int c = lane; c < n; c += 32) M = fmaxf(M, __ldcg(lse + int64_t(c) * nrows));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M != -INFINITY) {
    for (int c0 = 0; c0 < n; c0 += 32) {
      const float mine = c0 + lane < n ? ex2((__ldcg(lse + int64_t(c0 + lane) * nrows) - M) * 1.4426950408889634f) : 0.f;
      for (int c1 = c0; c1 < min(n, c0 + 32); c1 += 8) {
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = c1 + u < n ? __ldcg(part + (c1 + u) * step) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float w = __shfl_sync(0xffffffffu, mine, (c1 + u) & 31);
          L += w;
          acc.x += w * v[u].x;
          acc.y += w * v[u].y;
          acc.z += w * v[u].z;
          acc.w += w * v[u].w;
        }
      }
    }
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const int row = it.row0 + r, t = row / p.group, head = it.hk * p.group + row - t * p.group;
  const int64_t tok = int64_t(it.rq.qo_start) + t;
  uint2 packed;
  packed.x = Elem<T>::from_float2(acc.x * inv, acc.y * inv);
  packed.y = Elem<T>::from_float2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.o + tok * p.o_stride_tok + int64_t(head) * p.o_stride_head + 4 * lane) = packed;
  if (lane == 0 && p.lse) p.lse[tok * p.num_qo_heads + head] = L > 0.f ? M + __logf(L) : -INFINITY;
}

// Rows [kKv4Tile pass, ..) of an item, by its team.  u: this lane's part of them;
// on return of those of pass `next_pass` of item `next_i` (on their way while the
// states are joined).  `after`: the team whose states of the pass before may still
// be being joined; its barrier comes before this warp's next state, so that a warp
// without a row to join goes on.  A row of a split unit is merged by the warp that
// brings its last chunk, by a counter for each row: no warp waits for another's.
template <typename T, int kB>
__device__ __forceinline__ void kv4_pass(const Kv4Params& kp, Kv4Smem& sm, int warp, const Kv4Places<kB>& at,
                                         const Item& it, int pass, int32_t off_items, int32_t next_i, int next_pass,
                                         int32_t end, const Kv4Team& team, Kv4Team& after, int32_t off_merge,
                                         int32_t off_rows, int causal, const Variant& var, uint32_t& used,
                                         uint4 (&u)[4]) {
  const RunParams& p = kp.run;
  const int lane = threadIdx.x & 31, G = p.group;
  const int rows = min(kKv4Tile, it.row1 - it.row0 - kKv4Tile * pass);
  const int nst = kv4_stages(it), parts = min(nst, team.warps);
  if (team.rank < parts) {
    Kv4Rows<T> R;
    kv4_set_rows<T>(kp, it, pass, causal, var, u, R);
    // keys that every row of the pass sees
    const int r0 = it.row0 + kKv4Tile * pass, r1 = r0 + rows - 1, pos = it.rq.kv_len - it.rq.qo_len;
    const int lim = min(causal ? pos + r0 / G : it.rq.kv_len - 1, it.kv1 - 1), lo = window_low(var, pos + r1 / G);
    const int s1 = kv4_share(nst, team.rank + 1, team.warps);
    bool ok = __shfl_sync(0xffffffffu, sm.abort ? 0 : 1, 0);
    for (int st = kv4_share(nst, team.rank, team.warps); st < s1 && ok; ++st) {
      const int slot = used % kKv4Depth;
      ok = warp_wait(&sm.full[warp][slot], (used / kKv4Depth) & 1, &sm.abort);
      if (!ok) break;
      ++used;
      const int j0 = it.kv0 + kKv4Stage * st;
      const uint32_t good = sm.dec.good[warp][slot];
      const bool inside = good == 0xffffffffu && j0 + kKv4Stage - 1 <= lim && j0 >= lo;
      kv4_stage<T, kB>(sm.dec.ring[warp][slot], at, good, j0, inside, var, R);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[warp][slot]);
    }
    if (after.warps) named_barrier_sync(after.bar, after.threads);
    kv4_put_state<T>(sm, warp, R);
  } else if (after.warps) {
    named_barrier_sync(after.bar, after.threads);
  }
  if (next_i < end) kv4_fetch_rows(kp, load_item(p.iws, off_items, next_i), next_pass, u);
  named_barrier_sync(team.bar, team.threads);
  const int w0 = warp - team.rank;  // the team's first warp
  if (!sm.abort) {
    for (int r = team.rank; r < rows; r += team.warps) {
      // lane w has warp w's maximum and sum
      const float m = lane < parts ? sm.dec.comb_m[w0 + lane][r] : -INFINITY;
      float M = m;
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
      M = __shfl_sync(0xffffffffu, M, 0);
      const float f = m != -INFINITY ? ex2(m - M) : 0.f;
      float L = lane < parts ? f * sm.dec.comb_l[w0 + lane][r] : 0.f;
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
      L = __shfl_sync(0xffffffffu, L, 0);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < parts; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(&sm.dec.comb_o[w0 + w][r][4 * lane]);
        const float fw = __shfl_sync(0xffffffffu, f, w);
        acc.x += fw * v.x;
        acc.y += fw * v.y;
        acc.z += fw * v.z;
        acc.w += fw * v.w;
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;
      const float lse = L > 0.f ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
      const int prow = kKv4Tile * pass + r;
      if (it.part < 0) {
        const int row = it.row0 + prow, t = row / G, head = it.hk * G + row - t * G;
        const int64_t tok = int64_t(it.rq.qo_start) + t;
        uint2 packed;
        packed.x = Elem<T>::from_float2(acc.x * inv, acc.y * inv);
        packed.y = Elem<T>::from_float2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(p.o + tok * p.o_stride_tok + int64_t(head) * p.o_stride_head + 4 * lane) = packed;
        if (lane == 0 && p.lse) p.lse[tok * p.num_qo_heads + head] = lse;
      } else {
        const int64_t part = int64_t(it.part) + prow;
        *(reinterpret_cast<float4*>(p.fws + p.partial_o_offset + part * kHeadDim) + lane) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (lane == 0) p.fws[part] = lse;
        const int32_t* unit = p.iws + off_merge + FI_MERGE_INTS * it.merge;
        const int n = __ldg(unit + 4);
        const int64_t base = __ldg(unit + 5);
        int32_t* const count = p.iws + off_rows + FI_KV4_ROW_COUNTERS * it.merge + prow;
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0) last = atomicAdd(count, 1) == n - 1;
        if (__shfl_sync(0xffffffffu, last, 0)) {
          __threadfence();
          kv4_merge_row<T>(p, it, prow, n, base);
          if (lane == 0) *count = 0;  // ready for the next run of this plan
        }
      }
    }
  }
  after = team;
}

// The items [begin, end) of a CTA, by computing warp `warp`.
template <typename T, int kB>
__device__ void kv4_consume(const Kv4Params& kp, Kv4Smem& sm, int warp, int32_t begin, int32_t shorts, int32_t end,
                            int32_t off_items, int32_t off_merge, int32_t off_rows, int causal, const Variant& var) {
  const RunParams& p = kp.run;
  const Kv4Places<kB> at(kp);
  const int group = warp / kKv4GroupWarps;
  uint32_t used = 0;
  Kv4Team after{0, 0, 0, 0};
  int32_t i = kv4_next_item(begin - 1, shorts, group);
  if (i >= end) return;
  int pass = 0;
  uint4 u[4];
  kv4_fetch_rows(kp, load_item(p.iws, off_items, i), 0, u);
  while (i < end) {
    const Item it = load_item(p.iws, off_items, i);
    const bool last = kKv4Tile * (pass + 1) >= it.row1 - it.row0;
    const int32_t next_i = last ? kv4_next_item(i, shorts, group) : i;
    const int next_pass = last ? 0 : pass + 1;
    kv4_pass<T, kB>(kp, sm, warp, at, it, pass, off_items, next_i, next_pass, end, kv4_team(warp, i < shorts), after,
                    off_merge, off_rows, causal, var, used, u);
    i = next_i;
    pass = next_pass;
  }
  named_barrier_sync(after.bar, after.threads);
}

// A CTA's items come prefill-class first, longest first in a class.  mid: the
// first of [begin, end) of at most FI_TILE_DECODE packed rows; shorts: the first
// from there on that one group takes alone (a last one goes to all warps).  Whole
// warps; lane l looks at item i0 + l.
__device__ __forceinline__ void kv4_phases(const RunParams& p, int32_t begin, int32_t end, int32_t off_items, int32_t& mid,
                                           int32_t& shorts) {
  const int lane = threadIdx.x & 31;
  mid = shorts = end;
  for (int32_t i0 = begin; i0 < end && shorts == end; i0 += 32) {
    bool small = false, is_short = false;
    if (i0 + lane < end) {
      const int32_t* item = p.iws + off_items + FI_ITEM_INTS * (i0 + lane);
      const int2 kv = __ldg(reinterpret_cast<const int2*>(item + 4));
      small = __ldg(item + 9) * p.group <= FI_TILE_DECODE;
      is_short = small && kv.y - kv.x <= kKv4GroupKeys;
    }
    const unsigned m = __ballot_sync(0xffffffffu, small), ms = __ballot_sync(0xffffffffu, is_short);
    if (mid == end && m) mid = i0 + __ffs(m) - 1;
    if (ms) shorts = i0 + __ffs(ms) - 1;
  }
  if (shorts + 1 >= end) shorts = end;
}

template <typename T, int kB>
__global__ void __launch_bounds__(kKv4Threads, 1) kv4_attention_kernel(const __grid_constant__ Kv4Params kp) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Kv4Smem& sm = *reinterpret_cast<Kv4Smem*>(smem_raw);
  if (threadIdx.x == 0) let_dependents_start();
  const RunParams& p = kp.run;
  const int32_t* iws = p.iws;
  // The plan in the workspace has to be one over the 4-bit cache and fit this
  // launch: nothing is written otherwise.  (A plan's CTA offsets and items lie
  // where this grid has them: their loads do not wait for the header's.)
  constexpr int32_t off_cta = FI_HEADER_INTS;
  const int32_t off_items = off_cta + ((int32_t(gridDim.x) + 4) & ~3);
  const int32_t begin = __ldg(iws + off_cta + blockIdx.x), end = __ldg(iws + off_cta + blockIdx.x + 1);
  const int32_t h_rows = ws_header(iws, FI_H_PARTIAL_ROWS), h_qo = ws_header(iws, FI_H_TOTAL_QO);
  const bool bad = ws_header(iws, FI_H_MAGIC) != FI_PLAN_MAGIC_KV4 ||
                   ws_header(iws, FI_H_NUM_CTAS) != int32_t(gridDim.x) || ws_header(iws, FI_H_OFF_CTA) != off_cta ||
                   ws_header(iws, FI_H_OFF_ITEMS) != off_items || h_rows < 0 || h_rows > p.max_partial_rows ||
                   h_qo < 0 || h_qo > p.q_num_tokens || ws_header(iws, FI_H_NUM_QO_HEADS) != p.num_qo_heads ||
                   ws_header(iws, FI_H_NUM_KV_HEADS) != p.num_kv_heads ||
                   ws_header(iws, FI_H_PAGE_SIZE) != p.kv[0].page_size || (smem_u32(smem_raw) & 1023u) != 0 ||
                   begin < 0 || end < begin || end > ws_header(iws, FI_H_NUM_ITEMS);
  if (bad) {
    if (threadIdx.x == 0) atomicOr(p.iws + FI_H_STATUS, kStatusBadPlan);
    return;
  }
  const int32_t off_merge = ws_header(iws, FI_H_OFF_MERGE), off_cnt = ws_header(iws, FI_H_OFF_COUNTERS);
  const int32_t off_rows = off_cnt + ((ws_header(iws, FI_H_NUM_MERGE) + 3) & ~3);
  const int causal = ws_header(iws, FI_H_CAUSAL);
  Variant var;
  var.window_left = ws_header(iws, FI_H_WINDOW_LEFT);
  var.sink = ws_header(iws, FI_H_SINK_TOKENS);
  var.cap_a = var.cap_b = 0.f;
  var.rope_table = nullptr;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x < kKv4Warps * kKv4Depth) {
    mbar_init(&sm.full[0][threadIdx.x], kB ? 1 : 33);  // the copies' bytes; or every copying lane, and one for the bits
    mbar_init(&sm.empty[0][threadIdx.x], 1);
  }
  if (threadIdx.x == kKv4Warps * kKv4Depth) {
    for (int s = 0; s < kKv4RawStages; ++s) {
      mbar_init(&sm.raw_full[s], 1);
      mbar_init(&sm.raw_empty[s], kKv4QuantWarps / kKv4RawStages);  // the warps of a stage's keys
    }
    mbar_init(&sm.q_full, 2 + kKv4QuantWarps);  // every warp that turns rows of it
    mbar_init(&sm.q_raw, kp.run.kv[0].tc ? 1 : 2);  // its load, or the warps that copy it
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.drain, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.k_full[s], kKv4QuantWarps);
      mbar_init(&sm.v_full[s], kKv4QuantWarps);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_empty[s], 1);
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.o_ready[s], 1);
      mbar_init(&sm.o_free[s], 4);  // the warps of an M tile's softmax
      mbar_init(&sm.p_full[s][0], 4);
      mbar_init(&sm.p_full[s][1], 4);
    }
    sm.abort = 0;
    sm.merge_last_pf = 0;
  }
  fence_mbar_init();
  int32_t mid, shorts;
  kv4_phases(p, begin, end, off_items, mid, shorts);
  const bool prefill = mid > begin;
  if (prefill && warp == kMmaWarp) {
    tc::tmem_alloc(&sm.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // Every warpgroup leaves the first phase with the launch's registers: those
  // that had more give them up before its barrier, the others take theirs behind
  // it.
  if (prefill) {
    if (warp < kKv4QuantWarp0) {
      tc::setmaxnreg_dec<kKv4RegsMma>();
      if (warp == 0) {
        kv4_pf_load<kB>(kp, sm, begin, mid, off_items);
      } else if (warp == kMmaWarp) {
        pf_mma<__half, false>(p, sm, begin, mid, off_items);
        __syncwarp();
      } else {
        kv4_pf_queries<T>(kp, sm, warp - 2, begin, mid, off_items);
        __syncwarp();
      }
      fence_proxy_async_smem();  // the second phase's copies go where these tiles were
      tc::fence_before_sync();
      named_barrier_sync_unaligned(kPhaseBarrier, kKv4Threads);
      tc::fence_after_sync();
      tc::setmaxnreg_inc<kKv4RegsLaunch>();
    } else if (warp < kKv4SoftmaxWarp0) {
      tc::setmaxnreg_dec<kKv4RegsWiden>();
      kv4_pf_widen<T, kB>(kp, sm, begin, mid, off_items);
      __syncwarp();
      fence_proxy_async_smem();
      named_barrier_sync_unaligned(kPhaseBarrier, kKv4Threads);
      tc::setmaxnreg_inc<kKv4RegsLaunch>();
    } else {
      tc::setmaxnreg_inc<kKv4RegsSoftmax>();
      if (var.window_left >= 0)
        kv4_pf_softmax<T, true>(p, sm, begin, mid, off_items, off_merge, off_cnt, causal, var);
      else
        kv4_pf_softmax<T, false>(p, sm, begin, mid, off_items, off_merge, off_cnt, causal, var);
      tc::setmaxnreg_dec<kKv4RegsLaunch>();
      fence_proxy_async_smem();
      tc::fence_before_sync();
      named_barrier_sync_unaligned(kPhaseBarrier, kKv4Threads);
      tc::fence_after_sync();
    }
  }
  if (mid < end) {
    if (warp < kKv4FirstWarp) {
      tc::setmaxnreg_dec<kKv4RegsDecode0>();
      kv4_load<kB>(kp, sm, warp, off_items, mid, shorts, end);
    } else {
      tc::setmaxnreg_inc<kKv4RegsDecode>();
      kv4_consume<T, kB>(kp, sm, warp - kKv4FirstWarp, mid, shorts, end, off_items, off_merge, off_rows, causal, var);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (prefill && warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(sm.tmem_base, kTmemCols);
  }
  if (threadIdx.x == 0 && sm.abort) atomicOr(p.iws + FI_H_STATUS, sm.abort);
}

}  // namespace fi
