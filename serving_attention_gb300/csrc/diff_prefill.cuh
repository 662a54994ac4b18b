// diff_prefill.cuh -- prefill-class items of differential attention on the
// 5th-generation tensor cores.
//
// An item is up to 128 packed query rows against a chunk of keys.  Map m
// multiplies dims 64 m .. 64 m + 63 of the one Q tile and of K; with the two
// maps' weights w_1, w_2 the output is (w_1 - lambda w_2) V.  The keys are
// walked twice:
//   pass 0  logits of both maps, their references and sums;
//   pass 1  logits again, now with the normalisers known: one weight
//           w_1 - lambda w_2 per key, rounded once, and one product with V.
// The maps' common part cancels before any rounding, so the error is half a
// step of the weights' type relative to the difference, however much of the
// maps cancels (1.38 times the error of rounding the result alone, at random
// keys); with each map's weights rounded on their own it was 1.53 times, and
// more the more the maps agree.  It also takes fewer tensor cycles than two
// accumulators would: per 128 keys 512 in pass 0 and 512 + 512 in pass 1,
// against 512 + 1024, or 512 + 2048 with weights of two terms; the second walk
// costs 128 exponentials a thread, which overlap with them.
// A split unit's chunk needs both maps' outputs, each to be weighed by its own
// map's share of the chunk: pass 1 walks the keys for map 1 alone and pass 2 for
// map 2, with weights of two 16-bit terms, p = hi + lo, so that what the maps
// have in common cancels in the merge too (1.00 times the error of rounding the
// result alone).  With S_1 - lambda S_2 in pass 1 and S_2 in pass 2, weights of
// one term, a prompt part of 600 queries behind 20000 keys took 121 us for 131,
// but S_1 then had the rounding of map 2's weights in the chunk, at full size
// where map 2 looks at other chunks.
//
// Roles: warp 0 loads Q (two buffers) and K, warp 2 V, by TMA (pages below 8
// tokens: by copies, with warp 3), into one ring of four tiles (two rings of two
// tiles hold less of what is needed next); warp 1 issues the products;
// warpgroups of warps 4..7, 8..11, 12..15 and 16..19 take 32 keys each of
// every 128-key tile, for both maps (thread = row = tensor-memory lane).
// Tensor memory: S of both maps (256 columns), O (128), two P buffers (64
// each); in pass 0, which needs neither O nor P, their columns are a second S
// buffer, and where a pass has one map alone the other map's S columns hold the
// second terms of P.  A thread takes its 64 logits into registers and
// gives S back, so the next tile's S runs while it computes; P has columns of
// its own, so S does not wait for P V either.  Four softmax warps on each
// scheduler: with two (64 keys each) a warp's waits, loads and stores were
// not covered.
//
// What bounds it (556 us for 12161 queries of 8 prompts, 32 query heads, up to
// 3756 keys; its tiles' products alone would take 293): a tile takes some 3200 cycles of both passes, of which the
// products read 160 KB of operands and TMA writes 96 KB through shared memory's
// 128 bytes a cycle (2050 cycles), and the MMA and softmax warps hand S and P
// to one another; leaving the arithmetic of either pass out gains 6 %.  An item
// ends in some 6000 cycles from its last weights to the next one's first sums.
#pragma once
#include "attention_kernel.cuh"
#include "diff_params.h"

namespace fi {

constexpr int kDiffThreads = 640;
constexpr int kDiffGroups = 4;                         // softmax warpgroups
constexpr int kDiffKeys = kTileN / kDiffGroups;        // keys of a tile, and dims of the output, of each
constexpr int kDiffSoftmaxThreads = 128 * kDiffGroups;
constexpr int kDiffBarrier = 6;  // all softmax warpgroups (1: decode, 3: end of phase, 4 and 5: two warpgroups)
constexpr int kDiffStages = 4;   // K and V tiles in one ring
constexpr int kDiffCopyBarrier = 8;  // named barrier of the two warps that copy K tiles of small pages
constexpr int kDiffTmemO = 256, kDiffTmemP = 384;
constexpr float kWeightScale = 13.f;  // softmax weights are multiplied by 2^13 before they are rounded
// Register budgets, per thread (see kRegsLaunch): in the tensor-core phase
// warps 0..3 and the softmax warpgroups, in the decode phase its consumers
// (two warpgroups) and the other twelve warps.
constexpr int kDiffRegsLaunch = 96;
constexpr int kDiffRegsLoader = 64, kDiffRegsSoftmax = 104;
constexpr int kDiffRegsOther = 48, kDiffRegsConsumer = 168;
static_assert(kDiffRegsLoader * 128 + kDiffRegsSoftmax * 512 <= kDiffRegsLaunch * kDiffThreads, "exceeds the launch");
static_assert(kDiffRegsOther * 384 + kDiffRegsConsumer * 256 <= kDiffRegsLaunch * kDiffThreads, "exceeds the launch");

struct DiffPrefillBufs {  // every [128][64] block is a 128-byte swizzled operand half (see PrefillBufs)
  uint16_t q[2][2][kTileM][64];  // [buffer][d half = map][row][dim]; an item's output leaves through its Q buffer
  uint16_t kv[kDiffStages][2][kTileN][64];  // [stage][d half][token][dim]
  float stats[kDiffGroups][4][kTileM];  // [warpgroup][max 1, sum 1, max 2, sum 2][row] over its keys
  float sq[kDiffGroups][kTileM];        // [dim quarter][row] sum of squares
  float4 norm_w[kHeadDim / 4];
};

struct DiffPrefillBars {
  uint64_t q_full[2], q_empty[2], kv_full[kDiffStages], kv_empty[kDiffStages];
  uint64_t v_clear[kDiffStages];  // a tile's V rows past the request's end cleared
  uint64_t v_go[2];               // [Q buffer] the K loader is past the item's pass 0
  uint64_t s_full[2], s_free[2];  // [S buffer]
  uint64_t p_full[2];             // [buffer]
  uint64_t o_ready, o_free, drain;
};

// An item with the tiles of its sink: lead tiles from key 0 on, then those of
// [kv0, kv1).
struct DiffItem : Item {
  int32_t lead;
};
__device__ __forceinline__ DiffItem load_diff_item(const int32_t* iws, int32_t off_items, int32_t i) {
  return DiffItem{load_item(iws, off_items, i), __ldg(iws + off_items + FI_ITEM_INTS * i + FI_ITEM_LEAD)};
}
__device__ __forceinline__ int diff_tiles(const DiffItem& it) { return it.lead + item_kv_tiles(it); }
__device__ __forceinline__ int diff_tile_key(const DiffItem& it, int j) {  // first key of tile j
  return j < it.lead ? j * kTileN : it.kv0 + (j - it.lead) * kTileN;
}

static_assert(FI_MIN_TMA_PAGE == kMinTmaPage, "the planner's smallest page of this path's boxes");

// Passes of an item behind pass 0: pass 1, and of a split unit's chunk pass 2.
__device__ __forceinline__ int pv_passes(const Item& it) { return it.part >= 0 ? 2 : 1; }

// Whether the item's last KV tile reaches past the end of the request inside
// a page: the V rows there may hold anything (0 * NaN would not be 0).
__device__ __forceinline__ bool item_v_tail(const Item& it, int page_size) {
  return page_size >= kMinTmaPage && (it.rq.kv_len & (page_size - 1)) != 0 &&
         it.kv0 + item_kv_tiles(it) * kTileN > it.rq.kv_len;
}

// Pages below 8 tokens, whose boxes would start inside a swizzle atom: a tile's
// rows are copied 16 bytes at a time into the boxes' layout, K by warps 0 and 3,
// 64 rows each, V by warp 2, and handed on once they have landed.  4 prompts of
// 300 to 512 queries: 38 us on pages of one token, 26 on pages of 16.
template <bool kV>
__device__ __forceinline__ void diff_pf_copy(const DiffParams& dp, const DiffItem& it, uint16_t (*buf)[kTileN][64],
                                             int key0, int row0, int rows) {
  const KvCache& kc = dp.run.kv[0];
  const int lane = threadIdx.x & 31, c16 = lane & 15, hw = lane >> 4;
  const int lp = kc.log2_page, P = kc.page_size;
  const int32_t* pages = kc.kv_indices + it.rq.page_start;
  const int64_t page_stride = kV ? dp.v_strides[0] : dp.k_strides[0];
  const int64_t slot_stride = kV ? dp.v_strides[1] : dp.k_strides[1];
  const uint16_t* head = (kV ? dp.v : dp.k) + it.hk * (kV ? dp.v_strides[2] : dp.k_strides[2]) + 8 * c16;
  auto page_of = [&](int row) -> int32_t {  // of this lane's row
    const int key = key0 + row + lane;
    const int32_t id = key < it.rq.kv_len ? __ldg(pages + (key >> lp)) : -1;
    return uint32_t(id) < uint32_t(kc.num_pages) ? id : -1;
  };
  int32_t next = page_of(row0);
  for (int g = row0; g < row0 + rows; g += 32) {
    const int64_t my_row = next >= 0 ? next * page_stride + ((key0 + g + lane) & (P - 1)) * slot_stride : -1;
    if (g + 32 < row0 + rows) next = page_of(g + 32);
#pragma unroll 8
    for (int r = 0; r < 16; ++r) {
      const int tt = 2 * r + hw, row = g + tt;
      const int64_t at = __shfl_sync(0xffffffffu, my_row, tt);
      cp_async_16(&buf[c16 >> 3][row][((c16 & 7) ^ (row & 7)) * 8], head + (at >= 0 ? at : 0), at >= 0 ? 16u : 0u);
    }
  }
  cp_async_wait_all();
  fence_proxy_async_smem();
  __syncwarp();
}

// Warp 0 (kV false): Q and K tiles; warp 2 (kV true): V tiles.  K and V tiles
// share one ring, in the order in which the MMA warp takes them: in pass 0 all
// its stages hold K.  With t the item's first place, and pending = 1 behind an
// item (whose last V comes after this item's first K):
//   pass 0            K(0) t, K(j) t + pending + j
//   pass 1            from t1 = t + pending + tiles: K(0) t1, K(j) t1 + 2j - 1,
//                     V(j) t1 + 2j + 2
//   the next item     t1 + 2 tiles - 1.
// The passes 1 and 2 of a split unit's chunk leave nothing pending: their last V
// has the place before, and the pass or item behind them begins 2 tiles on.
// Returns which stages this warp loaded, and above them the phases of the last
// loads.
template <bool kV, bool kCopies>
__device__ uint32_t diff_pf_produce(const DiffParams& dp, DiffPrefillBufs& pf, DiffPrefillBars& bar,
                                    volatile int* abort, int32_t b0, int32_t b1, int32_t off_items) {
  const RunParams& p = dp.run;
  const int lane = threadIdx.x & 31;
  const bool second = kCopies && !kV && threadIdx.x >= 32;  // warp 3, which only copies
  const KvCache& kc = p.kv[0];
  const int G = p.group, lp = kc.log2_page, P = kc.page_size, ppt = kTileN >> lp;
  const CUtensorMap* map = kV ? &kc.tm_v : &kc.tm_k;
  if (lane == 0) {
    if (!kCopies) tc::prefetch_tensormap(map);
    if (!kV) tc::prefetch_tensormap(&p.tm_q);
  }
  uint32_t t = 0, ni = 0;  // an item's first place, items
  int pending = 0;
  uint32_t armed = 0, armed_phase = 0;  // bit st: this warp loaded into stage st, and the phase of the last load
  int q_armed[2] = {-1, -1};
  DiffItem ahead = load_diff_item(p.iws, off_items, b0);
  for (int32_t i = b0; i < b1; ++i) {
    const DiffItem it = ahead;
    if (i + 1 < b1) ahead = load_diff_item(p.iws, off_items, i + 1);
    const int ntiles = diff_tiles(it);
    if (ntiles == 0) continue;
    const int32_t* pages = kc.kv_indices + it.rq.page_start;
    const int npages = (it.rq.kv_len + P - 1) >> lp;
    auto page_of = [&](int j) -> int32_t {
      const int pg = (diff_tile_key(it, j) >> lp) + lane;
      return lane < ppt && pg < npages ? __ldg(pages + pg) : kc.num_pages;  // out of bounds -> zeros
    };
    int32_t next = page_of(0);
    if (!kV && !second) {
      const int qb = ni & 1;
      const uint32_t ph = (ni >> 1) & 1;
      if (warp_wait(&bar.q_empty[qb], ph ^ 1, abort)) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar.q_full[qb], kQTileBytes);
          const int c1 = it.hk * G, c2 = it.rq.qo_start + it.row0 / G;
          tc::tma_load_3d(&pf.q[qb][0][0][0], &p.tm_q, &bar.q_full[qb], 0, c1, c2);
          tc::tma_load_3d(&pf.q[qb][1][0][0], &p.tm_q, &bar.q_full[qb], 64, c1, c2);
        }
        q_armed[qb] = ph;
      }
    }
    const bool split = it.part >= 0;
    const int steps = ntiles * pv_passes(it);
    const uint32_t t1 = t + pending + ntiles;
    int j = 0;
    for (int n = kV ? ntiles : 0; n < ntiles + steps; ++n) {
      const int q = n - ntiles, tile = j;       // step of the passes behind pass 0
      const uint32_t tp = t1 + 2 * (q - tile);  // first place of its pass
      const uint32_t at = q < 0 ? t + (n > 0 ? pending + n : 0) : kV ? tp + 2 * tile + 2 - (split && tile + 1 == ntiles)
                                                                           : tp + (tile > 0 ? 2 * tile - 1 : 0);
      const uint32_t st = at % kDiffStages, ph = (at / kDiffStages) & 1;
      const int32_t cur = next;
      j = j + 1 < ntiles ? j + 1 : 0;
      next = page_of(j);
      // A parity tells a phase from the next alone, so the V loads of an item
      // begin once the K loads are that far: at K(0) behind pass 0, the tiles
      // before t1 - 4 have been taken, and V(0)'s stage is at the phase before.
      // One barrier an item, two in turn: the arrival for item i + 2 follows
      // this warp's wait for Q buffer i & 1, so the output of item i, so its V
      // tiles, so the V loader's wait for item i, which cannot miss a phase.
      // The wait is as long as a pass 0, some 1600 cycles a tile of at most 2^24
      // tiles, and has that for its bound: a K loader that gives up ends it.
      if (q == 0) {
        if (kV)
          warp_wait<32 * kWaitBudgetClocks>(&bar.v_go[ni & 1], (ni >> 1) & 1, abort);
        else if (!second && lane == 0)
          mbar_arrive(&bar.v_go[ni & 1]);
      }
      const bool free = warp_wait(&bar.kv_empty[st], ph ^ 1, abort);
      if (kCopies) {
        if (free) diff_pf_copy<kV>(dp, it, pf.kv[st], diff_tile_key(it, tile), second ? 64 : 0, kV ? kTileN : 64);
        if (!kV) named_barrier_sync(kDiffCopyBarrier, 64);
        if (free && lane == 0 && !second) mbar_arrive(&bar.kv_full[st]);
        continue;
      }
      if (!free) continue;
      if (lane == 0) mbar_arrive_expect_tx(&bar.kv_full[st], kKVBytes);
      __syncwarp();
      uint16_t(*buf)[kTileN][64] = pf.kv[st];
      if (lane < ppt) {
        tc::tma_load_4d(&buf[0][lane * P][0], map, &bar.kv_full[st], 0, it.hk, 0, cur);
        tc::tma_load_4d(&buf[1][lane * P][0], map, &bar.kv_full[st], 64, it.hk, 0, cur);
      }
      armed |= 1u << st;
      armed_phase = (armed_phase & ~(1u << st)) | (ph << st);
      // The rows past the request's end are cleared once they have landed,
      // and the MMA warp waits for that instead.  This warp does it because
      // it alone starts the stage's next phase, so its wait cannot miss this
      // one.
      if (kV && tile + 1 == ntiles && item_v_tail(it, P) && warp_wait(&bar.kv_full[st], ph, abort)) {
        for (int row = it.rq.kv_len - diff_tile_key(it, tile) + (lane >> 4); row < kTileN; row += 2)
          *reinterpret_cast<uint4*>(&buf[(lane >> 3) & 1][row][8 * (lane & 7)]) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_clear[st]);
      }
    }
    t = t1 + 2 * steps - (split ? 0 : 1);
    pending = split ? 0 : 1;
    ++ni;
  }
  if (!kV && lane == 0) {  // every Q load has landed before the CTA moves on
    for (int s = 0; s < 2; ++s)
      if (q_armed[s] >= 0) mbar_wait_drain(&bar.q_full[s], q_armed[s]);
  }
  __syncwarp();
  return armed | armed_phase << kDiffStages;
}

// After a phase that gave up: the tiles still on their way into the ring have
// to land before its memory is used again.  (Otherwise the MMA warp has taken
// them all.)  A wait for a phase that the other loader's tile has followed
// runs into its bound.
__device__ __forceinline__ void diff_pf_drain(DiffPrefillBars& bar, uint32_t loads) {
  if ((threadIdx.x & 31) == 0)
    for (int st = 0; st < kDiffStages; ++st)
      if (loads >> st & 1) mbar_wait_drain(&bar.kv_full[st], (loads >> (kDiffStages + st)) & 1);
  __syncwarp();
}

// Waits for two phases, bounded as warp_wait is, but the warp keeps polling:
// the wake-up of a sleeping wait is on the critical path of the products.  Odd
// lanes poll the second.
__device__ __forceinline__ bool poll_wait(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, volatile int* abort) {
  const bool odd = threadIdx.x & 1;
  const uint32_t bar = odd ? b1 : b0, ph = odd ? p1 : p0;
  auto done = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(ph)
        : "memory");
    return __all_sync(0xffffffffu, ok != 0) != 0;
  };
  if (done()) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
      if (done()) return true;
    const int st = __shfl_sync(0xffffffffu, (*abort != 0 ? 2 : 0) | (clock64() - t0 > kWaitBudgetClocks ? 4 : 0), 0);
    if (st & 2) return false;
    if (st & 4) {
      *abort = kStatusTimeout;
      return false;
    }
  }
}

// Four products D (+)= A B of K 16 each behind one election; the operands
// advance by constants.  A in shared memory (64 dims of Q) or, with kTmemA, in
// tensor memory (64 keys' weights); B 64 dims of K, or 64 keys of V.
template <bool kTmemA>
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a_desc, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                     uint32_t accumulate) {
  if (kTmemA)
    asm volatile(
        "{\n\t.reg .pred p, t, e;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %3, %3;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %3, %3;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The MMA warp shares its scheduler with four softmax warps, and an
// instruction of it takes 5 to 10 cycles: a step's few hundred instructions
// are what a step takes.  So its waits and products are kept short, and the
// blocks large: 8 products of S behind one wait, 8 of P V behind another.
template <typename T>
__device__ void diff_pf_mma(const RunParams& p, DiffPrefillBufs& pf, DiffPrefillBars& bar, volatile int* abort,
                            uint32_t tmem, int32_t b0, int32_t b1, int32_t off_items) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t idesc_s = tc::idesc_f16(kBf16, false, kTileM, kTileN);
  constexpr uint32_t idesc_pv = tc::idesc_f16(kBf16, true, kTileM, kHeadDim);
  const int lane = threadIdx.x & 31;
  // Start addresses count 16-byte units: a 64-dim half is 1024, a stage or Q
  // buffer 2048, 16 dims along a swizzled row 2, 16 V rows 128.
  const uint64_t dq = tc::smem_desc_sw128(smem_u32(&pf.q[0][0][0][0]), 16, 1024);
  const uint64_t dk = tc::smem_desc_sw128(smem_u32(&pf.kv[0][0][0][0]), 16, 1024);
  const uint64_t dv = tc::smem_desc_sw128(smem_u32(&pf.kv[0][0][0][0]), 64 * kTileN * 2, 1024);
  const uint32_t kv_full = smem_u32(&bar.kv_full[0]), v_clear = smem_u32(&bar.v_clear[0]);
  const uint32_t s_free = smem_u32(&bar.s_free[0]), p_full = smem_u32(&bar.p_full[0]), o_free = smem_u32(&bar.o_free);
  uint32_t t = 0, ni = 0, no = 0;           // tiles taken from the ring, items, uses of O so far
  uint32_t ps = 3, pp = 0;                  // bit b: parity that the next use of S, P buffer b waits for
  uint32_t cleared = 0;                     // bit st: parity of the cleared tails of V stage st
  bool ok = true, issued = false;  // after a wait that ran out nothing more is issued
  // S of a step in buffer x, of the maps m0 .. m1
  auto do_s = [&](uint64_t a, int x, int m0, int m1) {
    const uint32_t st = t % kDiffStages;
    ok = ok && poll_wait(s_free + 8 * x, (ps >> x) & 1, kv_full + 8 * st, (t / kDiffStages) & 1, abort);
    if (!ok) return;
    tc::fence_after_sync();
    const uint64_t b = dk + 2048u * st;
    const uint32_t d = tmem + 2 * kTileN * x;
    if (m0 == 0) mma4<false>(d, a, 0, b, idesc_s, 0);
    if (m1 == 1) mma4<false>(d + kTileN, a + 1024u, 0, b + 1024u, idesc_s, 0);
    tc::mma_commit_warp(&bar.s_full[x]);
    tc::mma_commit_warp(&bar.kv_empty[st]);
    ps ^= 1u << x;
    ++t;
    issued = true;
  };
  // P V of a step, weights in buffer b, second terms (or none) at column lo
  constexpr uint32_t kNoLo = ~0u;
  const uint32_t o_col = tmem + kDiffTmemO;
  auto do_pv = [&](uint32_t lo, int b, bool first, bool last, bool tail) {
    const uint32_t st = t % kDiffStages;
    if (first) ok = ok && poll_wait(o_free, (no & 1) ^ 1, o_free, (no & 1) ^ 1, abort);
    ok = ok && poll_wait(p_full + 8 * b, (pp >> b) & 1, (tail ? v_clear : kv_full) + 8 * st,
                         tail ? (cleared >> st) & 1 : (t / kDiffStages) & 1, abort);
    if (!ok) return;
    tc::fence_after_sync();
    const uint64_t v = dv + 2048u * st;
    const uint32_t w = tmem + kDiffTmemP + 64 * b;
    mma4<true>(o_col, 0, w, v, idesc_pv, first ? 0u : 1u);
    mma4<true>(o_col, 0, w + 32, v + 512u, idesc_pv, 1u);
    if (lo != kNoLo) {
      mma4<true>(o_col, 0, lo + 64 * b, v, idesc_pv, 1u);
      mma4<true>(o_col, 0, lo + 64 * b + 32, v + 512u, idesc_pv, 1u);
    }
    tc::mma_commit_warp(&bar.kv_empty[st]);
    if (last) {
      tc::mma_commit_warp(&bar.o_ready);
      ++no;
    }
    if (tail) cleared ^= 1u << st;
    pp ^= 1u << b;
    ++t;
  };
  // The P V of a step follows the S of the next step: what is pending behind
  // an item, if anything.
  struct {
    bool any, first, tail;
    int b;
  } pv{false, false, false, 0};
  auto flush = [&] {
    if (pv.any) do_pv(kNoLo, pv.b, pv.first, true, pv.tail);
    pv.any = false;
  };
  auto wait_o = [&] { ok = ok && poll_wait(o_free, (no & 1) ^ 1, o_free, (no & 1) ^ 1, abort); };
  bool split_before = false;
  DiffItem next = load_diff_item(p.iws, off_items, b0);
  for (int32_t i = b0; i < b1 && ok; ++i) {
    const DiffItem it = next;
    if (i + 1 < b1) next = load_diff_item(p.iws, off_items, i + 1);
    const int ntiles = diff_tiles(it);
    if (ntiles == 0) continue;
    const bool tail = item_v_tail(it, p.kv[0].page_size);
    const uint32_t qb = ni & 1, q_full = smem_u32(&bar.q_full[0]) + 8 * qb;
    const uint64_t a = dq + 2048u * qb;
    ok = poll_wait(q_full, (ni >> 1) & 1, q_full, (ni >> 1) & 1, abort);
    if (split_before) wait_o();  // its second terms are where S goes
    split_before = it.part >= 0;
    do_s(a, 0, 0, 1);
    flush();
    for (int j = 1; j < ntiles && ok; ++j) {
      if (j == 1) wait_o();  // S buffer 1: O's and P's columns, once the item before is read out
      do_s(a, j & 1, 0, 1);
    }
    if (it.part < 0) {
      do_s(a, 0, 0, 1);
      for (int j = 1; j < ntiles && ok; ++j) {
        do_s(a, 0, 0, 1);
        do_pv(kNoLo, (j - 1) & 1, j == 1, false, false);
      }
      pv = {true, ntiles == 1, tail, (ntiles - 1) & 1};
    } else {
      for (int x = 0; x < 2 && ok; ++x) {
        if (x == 1) wait_o();  // map 1's second terms are where map 2's S goes
        const uint32_t lo = tmem + (x == 0 ? kTileN : 0);
        do_s(a, 0, x, x);
        for (int j = 1; j < ntiles && ok; ++j) {
          do_s(a, 0, x, x);
          do_pv(lo, (j - 1) & 1, j == 1, false, false);
        }
        do_pv(lo, (ntiles - 1) & 1, ntiles == 1, true, tail);
      }
    }
    ++ni;
  }
  if (pv.any) ++t;  // the place of the first K that a next item would have
  flush();
  if (issued) {  // no product may still run when the CTA leaves the phase
    tc::mma_commit_warp(&bar.drain);
    if (lane == 0) mbar_wait_drain(&bar.drain, 0);
    __syncwarp();
  }
}

// 1 / sqrt(mean square of a head's 128 dims + eps); 0 where both are 0.
__device__ __forceinline__ float rms_factor(float sum_sq, float eps) {
  const float ms = sum_sq * (1.f / kHeadDim) + eps;
  return ms > 0.f ? rsqrtf(ms) : 0.f;
}

// Largest of a thread's 32 logits: eight chains of three-input maxima.
__device__ __forceinline__ float max32(const uint32_t (&v)[32]) {
  auto val = [&](int e) { return __uint_as_float(v[e]); };
  float mx[8];
#pragma unroll
  for (int a = 0; a < 8; ++a) mx[a] = max3(val(a), val(8 + a), val(16 + a));
#pragma unroll
  for (int a = 0; a < 8; ++a) mx[a] = fmaxf(mx[a], val(24 + a));
  return max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
}

// The softmax warpgroups and the end of the items.
template <typename T, bool kMask>
__device__ void diff_pf_softmax(const DiffParams& dp, DiffPrefillBufs& pf, DiffPrefillBars& bar, volatile int* abort,
                                uint32_t tmem, int32_t b0, int32_t b1, int32_t off_items, int causal,
                                const Variant var) {
  const RunParams& p = dp.run;
  const int sw = (threadIdx.x >> 5) - kSoftmaxWarp0, wg = sw >> 2, lane = threadIdx.x & 31;
  const int r = 32 * (sw & 3) + lane;
  const uint32_t tl = tmem + (uint32_t(32 * (sw & 3)) << 16);
  const bool elected = (threadIdx.x & 255) == 128;  // one thread of each pair of warpgroups
  const int half = wg >> 1;                          // of the keys, and of the output's dims
  const int G = p.group, log2_g = __ffs(G) - 1;  // G divides 128 on this path
  const float sc = p.scale_log2;
  const float2 cc = make_float2(sc, sc);
  uint32_t s_phase = 0, no = 0, ni = 0;  // bit x: parity of S buffer x's next tile; uses of O, items
  int q_held = -1;  // the Q buffer that this warpgroup's output store may still be reading
  if (dp.norm_w && sw < 4) reinterpret_cast<float*>(pf.norm_w)[r] = __ldg(dp.norm_w + r);
  named_barrier_sync(kDiffBarrier, kDiffSoftmaxThreads);
  // Lane l holds word l of the next item's descriptor.
  auto item_word = [&](int32_t i) {
    return lane <= FI_ITEM_LEAD && i < b1 ? __ldg(p.iws + off_items + FI_ITEM_INTS * i + lane) : 0;
  };
  int32_t ahead = item_word(b0);
  for (int32_t i = b0; i < b1; ++i) {
    auto word = [&](int w) { return __shfl_sync(0xffffffffu, ahead, w); };
    const DiffItem item{Item{word(0), word(1), word(2), word(3), word(4), word(5), word(6), word(7),
                             Request{word(8), word(9), word(10), word(11)}, 1},
                        word(FI_ITEM_LEAD)};
    ahead = item_word(i + 1);
    const Request& rq = item.rq;
    const int nrows = item.row1 - item.row0, ntiles = diff_tiles(item);
    const int row = item.row0 + r, tq = row >> log2_g, head = item.hk * G + (row & (G - 1));
    const int64_t tok = int64_t(rq.qo_start) + tq;
    const int pos = rq.kv_len - rq.qo_len + tq;
    const bool live = r < nrows;
    // visible keys [lo, lim] and the sink (a padding row, never stored, sees
    // all of the chunk, so that it does not make its warp mask every tile)
    const int lim = live && causal ? min(pos, item.kv1 - 1) : item.kv1 - 1;
    const int lo = kMask && live ? window_low(var, pos) : 0;
    // tiles [c0, c1) need no mask for any row of the warp's keys; past c2 no
    // row of the warp sees any
    const int first = item.kv0 + kDiffKeys * wg;  // this warpgroup's first key behind the sink's tiles
    const int c1 = item.lead + __reduce_min_sync(0xffffffffu, (lim + 1 - first - kDiffKeys + kTileN) >> 7);
    const int c2 = item.lead + __reduce_max_sync(0xffffffffu, (lim - first + kTileN) >> 7);
    const int c0 = kMask ? item.lead + ((max(__reduce_max_sync(0xffffffffu, lo) - first, 0) + kTileN - 1) >> 7) : 0;
    uint16_t* out = p.o + tok * p.o_stride_tok + int64_t(head) * p.o_stride_head + kDiffKeys * wg;
    if (ntiles == 0) {  // no key: the output and log-sum-exps of an empty row
      if (live && item.part < 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c) reinterpret_cast<uint4*>(out)[c] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse && wg < 2) p.lse[(tok * p.num_qo_heads + head) * 2 + wg] = -INFINITY;
      }
      continue;
    }
    bool ok = true;
    const float lam = live ? __ldg(dp.lambda + head) : 0.f;
    // This warpgroup's 32 logits of a tile in S buffer x, of both maps or (into
    // a) of map mp alone; S goes back to the MMA warp.
    auto load_s = [&](int x, bool both, int mp, uint32_t (&a)[32], uint32_t (&b)[32]) {
      const uint32_t ph = (s_phase >> x) & 1;
      if (!__all_sync(0xffffffffu, mbar_try_wait(&bar.s_full[x], ph))) ok = ok && warp_wait(&bar.s_full[x], ph, abort);
      s_phase ^= 1u << x;
      tc::fence_after_sync();
      const uint32_t col = tl + 2 * kTileN * x + kDiffKeys * wg;
      tc::tmem_ld32(col + kTileN * mp, a);
      if (both) tc::tmem_ld32(col + kTileN, b);
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.s_free[x]);
    };
    // Bit e: key e of this warpgroup's 32 of tile j is visible to the row (tests
    // of the keys one by one took twice as long as the tile's sums).
    auto visible = [&](int j) -> uint32_t {
      const int key0 = diff_tile_key(item, j) + kDiffKeys * wg;
      auto below = [&](int end) -> uint32_t {  // keys before end
        const int n = end - key0;
        return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
      };
      return kMask ? below(lim + 1) & (~below(lo) | below(var.sink)) : below(lim + 1);
    };
    auto mask = [&](uint32_t seen, uint32_t (&v)[32]) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!(seen >> e & 1)) v[e] = 0xff800000u;
    };
    // This thread's weights are in P buffer b, the other one of the step before.
    // It was free: the step's S was issued behind the P V of two steps before,
    // and a commit stands for everything issued before it.
    auto signal_p = [&](int b) {
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[b]);
    };
    // ---- pass 0: a reference m and the sum of 2^(s - m) per map.  The
    // reference is the maximum of the first tile that the row sees; it only
    // moves when a sum passes 2^100, so the loop has no maximum to take.
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool have_m = false;  // of every row of the warp
    for (int j = 0; j < ntiles; ++j) {
      uint32_t s[2][32];
      load_s(j & 1, true, 0, s[0], s[1]);
      if (j >= c2) continue;
      if (j < c0 || j >= c1) {
        const uint32_t seen = visible(j);
        mask(seen, s[0]);
        mask(seen, s[1]);
      }
      for (bool move = !have_m;; move = true) {
        if (move) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float top = max32(s[x]) * sc;
            if (top > m[x] + kLazyRescale) {
              l[x] *= ex2(m[x] - top);  // 0 * 0 before the first key
              m[x] = top;
            }
          }
          have_m = __all_sync(0xffffffffu, m[0] != -INFINITY && m[1] != -INFINITY);
        }
        const float ms0 = m[0] == -INFINITY ? 0.f : m[0], ms1 = m[1] == -INFINITY ? 0.f : m[1];
        const float2 n0 = make_float2(-ms0, -ms0), n1 = make_float2(-ms1, -ms1);
        float2 sum[2][2];
#pragma unroll
        for (int a = 0; a < 2; ++a) sum[0][a] = sum[1][a] = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = fma2(make_float2(__uint_as_float(s[0][2 * e]), __uint_as_float(s[0][2 * e + 1])), cc, n0);
          const float2 y = fma2(make_float2(__uint_as_float(s[1][2 * e]), __uint_as_float(s[1][2 * e + 1])), cc, n1);
          sum[0][e & 1] = add2(sum[0][e & 1], make_float2(ex2(x.x), ex2(x.y)));
          sum[1][e & 1] = add2(sum[1][e & 1], make_float2(ex2(y.x), ex2(y.y)));
        }
        const float2 t0 = add2(sum[0][0], sum[0][1]), t1 = add2(sum[1][0], sum[1][1]);
        const float l0 = l[0] + (t0.x + t0.y), l1 = l[1] + (t1.x + t1.y);
        if (move || !__any_sync(0xffffffffu, !(fmaxf(l0, l1) < 1.2676506e30f))) {  // 2^100
          l[0] = l0;
          l[1] = l1;
          break;
        }
      }
    }
    // The warpgroups' statistics of a row together, in the same order in all.
    // (`stats` of the item before has been read: this item's S needed its
    // readers' loads.)
    if (elected && q_held >= 0) {
      tc::bulk_wait_read_all();
      mbar_arrive(&bar.q_empty[q_held]);
    }
    q_held = -1;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      pf.stats[wg][2 * x][r] = m[x];
      pf.stats[wg][2 * x + 1][r] = l[x];
    }
    named_barrier_sync(kDiffBarrier, kDiffSoftmaxThreads);
    float log2l[2], lse = -INFINITY;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float mw[kDiffGroups], mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kDiffGroups; ++w) mm = fmaxf(mm, mw[w] = pf.stats[w][2 * x][r]);
#pragma unroll
      for (int w = 0; w < kDiffGroups; ++w)
        if (mw[w] != -INFINITY) ll += pf.stats[w][2 * x + 1][r] * ex2(mw[w] - mm);
      l[x] = ll;
      m[x] = mm == -INFINITY ? 0.f : mm;  // an empty row: every weight is 2^-inf
      log2l[x] = ll > 0.f ? __log2f(ll) : 0.f;
      if (wg == x && ll > 0.f) lse = (m[x] + log2l[x]) * 0.69314718055994531f;
    }

    uint32_t y[32];  // this warpgroup's 32 dims of a row of the accumulator, which goes back to the MMA warp
    auto val = [&](int e) { return __uint_as_float(y[e]); };
    auto load_o = [&] {
      ok = ok && warp_wait(&bar.o_ready, no & 1, abort);
      ++no;
      tc::fence_after_sync();
      tc::tmem_ld32(tl + kDiffTmemO + kDiffKeys * wg, y);
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.o_free);
    };
    if (item.part >= 0) {
      // ---- passes 1 and 2 of a split unit's chunk: one map's weights, scaled by
      // 2^13, in two terms that keep 16 (bf16) or 22 (fp16) bits; its partial state
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        const float a = (x ? m[1] + log2l[1] : m[0] + log2l[0]) - kWeightScale;
        const float2 n = make_float2(-a, -a);
        const uint32_t lo_col = tl + (x ? 0 : kTileN) + 16 * wg;
        for (int j = 0; j < ntiles; ++j) {
          uint32_t s[32], hi[16], lo[16];
          load_s(0, false, x, s, s);
          if (j < c0 || j >= c1) mask(visible(j), s);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 z = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), cc, n);
            const float w0 = ex2(z.x), w1 = ex2(z.y);
            hi[e] = tc::pack2<T>(w0, w1);
            const float2 h = Elem<T>::to_float2(hi[e]);
            lo[e] = tc::pack2<T>(w0 - h.x, w1 - h.y);
          }
          tc::tmem_st16(tl + kDiffTmemP + 64 * (j & 1) + 16 * wg, hi);
          tc::tmem_st16(lo_col + 64 * (j & 1), lo);
          signal_p(j & 1);
        }
        load_o();
        if (live && !*abort) {
          const float unscale = l[0] > 0.f ? ex2(-kWeightScale) : 0.f;  // both maps see the same keys
          const int64_t prw = int64_t(item.part) + x * nrows + r;
          float4* const dst = reinterpret_cast<float4*>(p.fws + p.partial_o_offset + prw * kHeadDim + kDiffKeys * wg);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(val(4 * e) * unscale, val(4 * e + 1) * unscale, val(4 * e + 2) * unscale,
                                 val(4 * e + 3) * unscale);
          if (wg == x) p.fws[prw] = lse;
        }
      }
      if (elected) mbar_arrive(&bar.q_empty[ni & 1]);
      ++ni;
      continue;
    }

    // ---- pass 1: weights w_1 - lambda w_2, scaled by 2^sigma so that they
    // stay below 2^14 and small ones inside an fp16's normal range
    const float sigma = kWeightScale - (fabsf(lam) > 1.f ? __log2f(fabsf(lam)) : 0.f);
    const float a1 = m[0] + log2l[0] - sigma, a2 = m[1] + log2l[1] - sigma;
    const float2 n1 = make_float2(-a1, -a1), n2 = make_float2(-a2, -a2), nl = make_float2(-lam, -lam);
    for (int j = 0; j < ntiles; ++j) {
      const int b = j & 1;
      uint32_t s1[32], s2[32], pk[16];
      load_s(0, true, 0, s1, s2);
      if (j < c0 || j >= c1) {
        const uint32_t seen = visible(j);
        mask(seen, s1);
        mask(seen, s2);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 x = fma2(make_float2(__uint_as_float(s1[2 * e]), __uint_as_float(s1[2 * e + 1])), cc, n1);
        const float2 y = fma2(make_float2(__uint_as_float(s2[2 * e]), __uint_as_float(s2[2 * e + 1])), cc, n2);
        const float2 w = fma2(make_float2(ex2(y.x), ex2(y.y)), nl, make_float2(ex2(x.x), ex2(x.y)));
        pk[e] = tc::pack2<T>(w.x, w.y);
      }
      tc::tmem_st16(tl + kDiffTmemP + 64 * b + 16 * wg, pk);
      signal_p(b);
    }
    if (p.lse && wg < 2 && live && !*abort) p.lse[(tok * p.num_qo_heads + head) * 2 + wg] = lse;
    const float unscale = l[0] > 0.f ? ex2(-sigma) : 0.f;
    load_o();
    // ---- the output
    float f = unscale * dp.out_scale;
    if (dp.norm_w) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) ss += val(e) * val(e);
      pf.sq[wg][r] = ss * unscale * unscale;
      named_barrier_sync(kDiffBarrier, kDiffSoftmaxThreads);
      f *= rms_factor((pf.sq[0][r] + pf.sq[1][r]) + (pf.sq[2][r] + pf.sq[3][r]), dp.norm_eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 w = pf.norm_w[kDiffKeys / 4 * wg + e];
        y[4 * e] = __float_as_uint(val(4 * e) * w.x);
        y[4 * e + 1] = __float_as_uint(val(4 * e + 1) * w.y);
        y[4 * e + 2] = __float_as_uint(val(4 * e + 2) * w.z);
        y[4 * e + 3] = __float_as_uint(val(4 * e + 3) * w.w);
      }
    }
    auto pack8 = [&](int e) {
      return make_uint4(tc::pack2<T>(val(e) * f, val(e + 1) * f), tc::pack2<T>(val(e + 2) * f, val(e + 3) * f),
                        tc::pack2<T>(val(e + 4) * f, val(e + 5) * f), tc::pack2<T>(val(e + 6) * f, val(e + 7) * f));
    };
    const int qb = ni & 1;
    if (nrows == kTileM) {  // a whole tile leaves through the item's Q halves, by one TMA store each
      uint16_t* stage = &pf.q[qb][half][0][0];
      uint4* my_row = reinterpret_cast<uint4*>(stage + r * 64);
#pragma unroll
      for (int c = 0; c < 4; ++c) my_row[(4 * (wg & 1) + c) ^ (r & 7)] = pack8(8 * c);
      fence_proxy_async_smem();
      named_barrier_sync(kEpilogueBarrier0 + half, 256);
      if (elected && !*abort) {
        tc::tma_store_3d(&p.tm_o, stage, 64 * half, item.hk * G, rq.qo_start + item.row0 / G);
        tc::bulk_commit();
      }
      q_held = qb;
    } else {
      if (elected) mbar_arrive(&bar.q_empty[qb]);
      if (live && !*abort) {
#pragma unroll
        for (int c = 0; c < 4; ++c) reinterpret_cast<uint4*>(out)[c] = pack8(8 * c);
      }
    }
    ++ni;
  }
  if (elected) tc::bulk_wait_all();  // output tiles written before the CTA moves on
  fence_proxy_async_smem();          // the decode ring's copies land in this phase's buffers
}

}  // namespace fi
