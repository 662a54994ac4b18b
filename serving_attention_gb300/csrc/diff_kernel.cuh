// diff_kernel.cuh -- persistent kernel of differential attention over the
// paged cache.
//
// A query row of head h is q = [q1 | q2], a key k = [k1 | k2], halves of 64
// dims; values have 128.  With S_i = softmax(scale * q_i k_i^T + mask) V
//
//   y = S_1 - lambda_h S_2,   o = out_scale * y                        or
//   o = out_scale * y / sqrt(mean(y^2) + eps) * w   (RMS norm over the 128 dims)
//
// Both maps read the same V rows, so the row tiles below read K and V once:
// the cache layout, its bytes and the work list are those of the ordinary run; a
// row's two maps are kept apart as two rows of the matrix products.  Requests of
// more than 16 packed rows walk their keys twice or three times (see
// diff_prefill.cuh) where the group divides 128; other groups take the row
// tiles, 16 rows a pass over the chunk.
//
// Row tiles (mma.sync m16n8k16; this path is bound by the cache's bytes, 8
// query rows fill the 16 rows of the smallest product exactly):
//  * up to 8 packed rows: row g of the tile is map 1, row g + 8 map 2 of
//    packed row g.  Q is [q1 | 0] and [0 | q2], so one chain of eight K16
//    steps gives both maps' logits and one P V product both outputs, and a
//    thread holds both maps of its row.
//  * 9 to 16 rows: a warp takes one map of all 16 rows; warps 0..3 map 1,
//    warps 4..7 map 2 of the same tokens.
// Measured: 64 requests of 512 to 32768 keys, 2.52 GB of cache, 371 us (99 %
// of the copy rate); 64 requests of 64 to 512 keys on pages of one token,
// 55 MB, 24 us, there bound by an item's chain of some 9000 cycles.
#pragma once
#include "attention_kernel.cuh"
#include "diff_params.h"
#include "diff_prefill.cuh"

namespace fi {

// Stages hold 128 tokens as two 64-dim halves of 128-byte rows, 16-byte
// chunks XOR-ed with the row (the layout of the 128-byte TMA swizzle), so
// that ldmatrix reads 8 rows without bank conflicts.
struct DiffBufs {
  uint16_t k[kStages][2][kStageTokens][64];
  uint16_t v[kStages][2][kStageTokens][64];
  float comb[kConsumerWarps][16][64];  // one half (64 dims) of the warps' O rows at a time
};

struct alignas(1024) DiffSmem {
  union {
    DiffBufs dec;
    DiffPrefillBufs pf;
  };
  float2 comb_ml[kConsumerWarps][16];  // (running max, sum) of the warps' rows
  uint64_t full[kStages], empty[kStages];
  DiffPrefillBars bars;
  uint32_t tmem_base;
  volatile int abort;  // set by the role whose bounded wait ran out
};
constexpr size_t kDiffSmemBytes = sizeof(DiffSmem);
static_assert(kDiffSmemBytes <= 227 * 1024, "shared memory of the differential kernel exceeds one CTA's limit");

// 16-bit products with fp32 sums: D (16 x 8) += A (16 x 16) * B (16 x 8).
template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t saddr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t saddr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// Passes of an item through the row tiles: one of up to 8 rows, or tiles of 16.
__device__ __forceinline__ int diff_passes(int nrows) { return (nrows + 15) / 16; }

// ---------------------------------------------------------------- producers

// Eight warps copy a stage's rows with 16-byte asynchronous copies, any page
// size and strides: 32 tokens each, warps 0..3 of K and the first four behind
// the consumers of V (a stage took four warps, both tensors each, 4900 cycles,
// most of them between the instructions of a warp).  Lane l holds the page id
// of token l (the next stage's loaded one stage ahead); half a warp copies one
// 256-byte row.  Tokens past the chunk and pages outside the cache arrive as
// zeros.
constexpr int kCopyWarps = 8;
__device__ __forceinline__ int diff_copy_warp(int warp) {
  constexpr int behind = kFirstConsumerWarp + kConsumerWarps;
  return warp < kFirstConsumerWarp ? warp : warp >= behind && warp < behind + 4 ? warp - behind + 4 : -1;
}

template <bool kV>
__device__ void diff_produce(const DiffParams& dp, DiffSmem& sm, int pw, int32_t item_begin, int32_t item_end,
                             int32_t off_items) {
  const RunParams& p = dp.run;
  const KvCache& kc = p.kv[0];
  const int lane = threadIdx.x & 31;
  const int c16 = lane & 15, hw = lane >> 4;
  const int lp = kc.log2_page, P = kc.page_size;
  const int64_t page_stride = kV ? dp.v_strides[0] : dp.k_strides[0];
  const int64_t slot_stride = kV ? dp.v_strides[1] : dp.k_strides[1];
  uint32_t it = 0;
  for (int32_t i = item_begin; i < item_end; ++i) {
    const Item item = load_item(p.iws, off_items, i);
    const int nst = (item.kv1 - item.kv0 + kStageTokens - 1) >> kLog2StageTokens;
    const int32_t* pages = kc.kv_indices + item.rq.page_start;
    const uint16_t* head = (kV ? dp.v : dp.k) + item.hk * (kV ? dp.v_strides[2] : dp.k_strides[2]) + 8 * c16;
    auto token_page = [&](int st) -> int32_t {
      const int tok = item.kv0 + st * kStageTokens + 32 * pw + lane;
      const int32_t id = tok < item.kv1 ? __ldg(pages + (tok >> lp)) : -1;
      return uint32_t(id) < uint32_t(kc.num_pages) ? id : -1;
    };
    const int passes = diff_passes(item.row1 - item.row0);
    for (int pass = 0; pass < passes; ++pass) {
      int32_t next = nst > 0 ? token_page(0) : -1;
      for (int st = 0; st < nst; ++st, ++it) {
        const int s = it % kStages;
        const int32_t cur = next;
        if (st + 1 < nst) next = token_page(st + 1);
        if (!warp_wait(&sm.empty[s], ((it / kStages) & 1) ^ 1, &sm.abort)) continue;
        const int tok0 = item.kv0 + st * kStageTokens + 32 * pw;
        // lane l: where token l's row begins
        const int64_t my_row = cur >= 0 ? cur * page_stride + ((tok0 + lane) & (P - 1)) * slot_stride : -1;
        uint16_t(*half)[64] = (kV ? sm.dec.v : sm.dec.k)[s][c16 >> 3];
#pragma unroll 8
        for (int r = 0; r < 16; ++r) {
          const int tt = 2 * r + hw, row = 32 * pw + tt;
          const int64_t at = __shfl_sync(0xffffffffu, my_row, tt);
          cp_async_16(&half[row][((c16 & 7) ^ (row & 7)) * 8], head + (at >= 0 ? at : 0), at >= 0 ? 16u : 0u);
        }
        cp_async_mbar_arrive_noinc(&sm.full[s]);
      }
    }
  }
  cp_async_wait_all();
}

// Smallest page whose stages come by TMA boxes: with 8-token pages the 64 boxes
// of a stage took 186.8 us for 753 MB of cache, the copies above 129.1.
constexpr int kDiffMinBoxPage = 16;

// Larger pages: warp 0 brings a stage with one 128-byte swizzled
// TMA box (64 dims, 1 head, P slots, 1 page) per page, half and tensor -- the
// boxes of the tensor-core path, in the layout that the copies above write by
// hand.  Lane l issues pages l, l + 32, ...; the next stage's page ids are
// loaded one stage ahead; pages past the chunk are addressed out of bounds and
// arrive as zeros.
static __device__ void diff_produce_tma(const DiffParams& dp, DiffSmem& sm, int32_t item_begin, int32_t item_end,
                                        int32_t off_items) {
  const RunParams& p = dp.run;
  const KvCache& kc = p.kv[0];
  DiffBufs& bufs = sm.dec;
  const int lane = threadIdx.x & 31;
  const int lp = kc.log2_page, P = kc.page_size, boxes = kStageTokens >> lp;  // 1 to 8
  if (lane == 0) {
    tc::prefetch_tensormap(&kc.tm_k);
    tc::prefetch_tensormap(&kc.tm_v);
  }
  uint32_t it = 0;
  int armed[kStages];
#pragma unroll
  for (int s = 0; s < kStages; ++s) armed[s] = -1;
  for (int32_t i = item_begin; i < item_end; ++i) {
    const Item item = load_item(p.iws, off_items, i);
    const int nst = (item.kv1 - item.kv0 + kStageTokens - 1) >> kLog2StageTokens;
    const int npages = (item.kv1 + P - 1) >> lp;  // of the request, up to the chunk's end
    const int32_t* pages = kc.kv_indices + item.rq.page_start;
    auto page_of = [&](int st) -> int32_t {
      const int pg = ((item.kv0 + st * kStageTokens) >> lp) + lane;
      return lane < boxes && pg < npages ? __ldg(pages + pg) : kc.num_pages;
    };
    const int passes = diff_passes(item.row1 - item.row0);
    for (int pass = 0; pass < passes; ++pass) {
      int32_t next = page_of(0);
      for (int st = 0; st < nst; ++st, ++it) {
        const int s = it % kStages;
        const uint32_t ph = (it / kStages) & 1;
        const int32_t cur = next;
        if (st + 1 < nst) next = page_of(st + 1);
        if (!warp_wait(&sm.empty[s], ph ^ 1, &sm.abort)) continue;
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[s], 2u * kStageTokens * kHeadDim * 2u);
        __syncwarp();
        if (lane < boxes) {
          const int row = lane << lp;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tc::tma_load_4d(&bufs.k[s][h][row][0], &kc.tm_k, &sm.full[s], 64 * h, item.hk, 0, cur);
            tc::tma_load_4d(&bufs.v[s][h][row][0], &kc.tm_v, &sm.full[s], 64 * h, item.hk, 0, cur);
          }
        }
        armed[s] = ph;
      }
    }
  }
  // Every load this warp armed has landed before the CTA leaves.
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s)
      if (armed[s] >= 0) mbar_wait_drain(&sm.full[s], armed[s]);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- consumers

// The 16-token slice of a stage at stage row tok0 (its first key: key0)
// against the warp's 16 tile rows: logits, online softmax, O += P V.
// kWide: the tile's rows are 16 packed rows of map `map`; otherwise rows g are
// map 1 and rows g + 8 map 2 of packed row g.
struct DiffRows {
  float m[2], l[2];        // of tile rows g and g + 8: running max (log2 domain) and this thread's share of the sum
  int lim[2], lo[2];       // visible keys [lo, lim], and those under the sink
};

template <typename T, bool kWide>
__device__ __forceinline__ void diff_slice(const uint16_t* ks, const uint16_t* vs, int tok0, int key0, int map,
                                           float scale_log2, int sink, int kv_end, const uint32_t (&qf)[16],
                                           DiffRows& rw, float (&o)[16][4]) {
  constexpr int kHalf = kStageTokens * 64;  // elements of a 64-dim half
  const int lane = threadIdx.x & 31, t = lane & 3;
  float s[2][4];
#pragma unroll
  for (int nb = 0; nb < 2; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[nb][e] = 0.f;
  // K: one ldmatrix brings 8 tokens x 32 dims (two K16 steps)
#pragma unroll
  for (int c = 0; c < (kWide ? 2 : 4); ++c) {
    const int half = kWide ? map : c >> 1, ch = (kWide ? c : c & 1) * 4 + (lane >> 3);
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
      const int row = tok0 + 8 * nb + (lane & 7);
      uint32_t b[4];
      ldmatrix_x4(b, smem_u32(ks + half * kHalf + row * 64 + ((ch ^ (row & 7)) * 8)));
      if (kWide) {
        mma_16816<T>(s[nb], qf[8 * c], qf[8 * c + 1], qf[8 * c + 2], qf[8 * c + 3], b[0], b[1]);
        mma_16816<T>(s[nb], qf[8 * c + 4], qf[8 * c + 5], qf[8 * c + 6], qf[8 * c + 7], b[2], b[3]);
      } else if (c < 2) {
        mma_16816<T>(s[nb], qf[4 * c], 0u, qf[4 * c + 1], 0u, b[0], b[1]);
        mma_16816<T>(s[nb], qf[4 * c + 2], 0u, qf[4 * c + 3], 0u, b[2], b[3]);
      } else {
        mma_16816<T>(s[nb], 0u, qf[4 * c], 0u, qf[4 * c + 1], b[0], b[1]);
        mma_16816<T>(s[nb], 0u, qf[4 * c + 2], 0u, qf[4 * c + 3], b[2], b[3]);
      }
    }
  }
  float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int nb = 0; nb < 2; ++nb)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = key0 + 8 * nb + 2 * t + (e & 1), x = e >> 1;
      const bool seen = key <= rw.lim[x] && (key >= rw.lo[x] || key < sink);
      s[nb][e] = seen ? s[nb][e] * scale_log2 : -INFINITY;
      mx[x] = fmaxf(mx[x], s[nb][e]);
    }
  float alpha[2];
  bool moved = false;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    mx[x] = quad_max(mx[x]);
    const float m_new = mx[x] > rw.m[x] + kLazyRescale ? mx[x] : rw.m[x];
    alpha[x] = m_new == rw.m[x] ? 1.f : ex2(rw.m[x] - m_new);
    moved |= m_new != rw.m[x];
    rw.m[x] = m_new;
    rw.l[x] *= alpha[x];
  }
  if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      o[n][0] *= alpha[0];
      o[n][1] *= alpha[0];
      o[n][2] *= alpha[1];
      o[n][3] *= alpha[1];
    }
  }
  // P as two 16-bit terms, p = hi + lo: the weights keep 16 (bf16) or 22 (fp16)
  // bits, so that the difference of the two maps carries no rounding of P;
  // the second product costs nothing here (the cache's bytes bound this path).
  uint32_t ph[4], pl[4];
#pragma unroll
  for (int nb = 0; nb < 2; ++nb)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float ms = rw.m[x] == -INFINITY ? 0.f : rw.m[x];
      const float p0 = ex2(s[nb][2 * x] - ms), p1 = ex2(s[nb][2 * x + 1] - ms);
      rw.l[x] += p0 + p1;
      const uint32_t h = Elem<T>::from_float2(p0, p1);
      const float2 hf = Elem<T>::to_float2(h);
      ph[2 * nb + x] = h;
      pl[2 * nb + x] = Elem<T>::from_float2(p0 - hf.x, p1 - hf.y);
    }
  // V rows at or past the chunk's end are not the request's: whatever they
  // hold (NaN and infinities included) is cleared, as 0 * NaN would not be 0
  const bool tail = key0 + 16 > kv_end;
  uint32_t keep[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int key = key0 + 8 * h + 2 * t;
    keep[h] = (key < kv_end ? 0x0000ffffu : 0u) | (key + 1 < kv_end ? 0xffff0000u : 0u);
  }
  const int vrow = tok0 + (lane & 15);
#pragma unroll
  for (int c = 0; c < 8; ++c) {  // 16 dims: two 8-dim column blocks x 16 tokens
    const int ch = 2 * c + (lane >> 4);
    uint32_t b[4];
    ldmatrix_x4_trans(b, smem_u32(vs + (ch >> 3) * kHalf + vrow * 64 + (((ch & 7) ^ (vrow & 7)) * 8)));
    if (tail) {
      b[0] &= keep[0];
      b[1] &= keep[1];
      b[2] &= keep[0];
      b[3] &= keep[1];
    }
    mma_16816<T>(o[2 * c], ph[0], ph[1], ph[2], ph[3], b[0], b[1]);
    mma_16816<T>(o[2 * c + 1], ph[0], ph[1], ph[2], ph[3], b[2], b[3]);
    mma_16816<T>(o[2 * c], pl[0], pl[1], pl[2], pl[3], b[0], b[1]);
    mma_16816<T>(o[2 * c + 1], pl[0], pl[1], pl[2], pl[3], b[2], b[3]);
  }
}

// y = S_1 - lambda S_2 of one (token, head) row held by a warp, float2 v[h] of
// each map at dims 64 h + 2 lane: the norm, the scale and the store.
template <typename T>
__device__ __forceinline__ void diff_store_row(const DiffParams& dp, const float2 (&s1)[2], const float2 (&s2)[2],
                                               float lam, int64_t tok, int head) {
  const RunParams& p = dp.run;
  const int lane = threadIdx.x & 31;
  float y[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    y[2 * h] = s1[h].x - lam * s2[h].x;
    y[2 * h + 1] = s1[h].y - lam * s2[h].y;
  }
  float f[4] = {dp.out_scale, dp.out_scale, dp.out_scale, dp.out_scale};
  if (dp.norm_w) {
    const float ss = warp_sum(y[0] * y[0] + y[1] * y[1] + y[2] * y[2] + y[3] * y[3]);
    const float r = rms_factor(ss, dp.norm_eps) * dp.out_scale;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f[2 * h] = r * __ldg(dp.norm_w + 64 * h + 2 * lane);
      f[2 * h + 1] = r * __ldg(dp.norm_w + 64 * h + 2 * lane + 1);
    }
  }
  uint16_t* dst = p.o + tok * p.o_stride_tok + int64_t(head) * p.o_stride_head + 2 * lane;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *reinterpret_cast<uint32_t*>(dst + 64 * h) = Elem<T>::from_float2(y[2 * h] * f[2 * h], y[2 * h + 1] * f[2 * h + 1]);
}

// One pass of an item's packed rows [prow0, prow0 + prows): the queries as
// product operands, the item's stages, then the merge of the eight warps'
// states and the output (or the fp32 partial states).
template <typename T, bool kWide>
__device__ __forceinline__ uint32_t diff_pass(const DiffParams& dp, DiffSmem& sm, const Item& item, int prow0,
                                              int prows, uint32_t it, int causal, const Variant& var) {
  const RunParams& p = dp.run;
  DiffBufs& bufs = sm.dec;
  const int cw = (threadIdx.x >> 5) - kFirstConsumerWarp;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = p.group;
  const Request& rq = item.rq;
  const int nst = (item.kv1 - item.kv0 + kStageTokens - 1) >> kLog2StageTokens;
  const int map = kWide ? cw >> 2 : 0;

  uint32_t qf[16];
  DiffRows rw;
  {
    const uint16_t* src[2];
    bool live[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = kWide ? g + 8 * x : g;  // packed row of tile row g + 8 x
      live[x] = r < prows;
      const int row = item.row0 + prow0 + (live[x] ? r : 0);
      const int tq = row / G, head = item.hk * G + (row - tq * G);
      src[x] = p.q + int64_t(rq.qo_start + tq) * p.q_stride_tok + int64_t(head) * p.q_stride_head + 2 * t;
      const int pos = rq.kv_len - rq.qo_len + tq;
      rw.lim[x] = live[x] ? min(causal ? pos : rq.kv_len - 1, item.kv1 - 1) : -1;
      rw.lo[x] = window_low(var, pos);
      rw.m[x] = -INFINITY;
      rw.l[x] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      // narrow: the pair of step e / 2 at offset 8 (e % 2), both maps in a row;
      // wide: steps of 64 dims of this map, rows g and g + 8 in turn
      const int x = kWide ? e & 1 : 0;
      const int dim = kWide ? 64 * map + 16 * (e >> 2) + 8 * ((e >> 1) & 1) : 16 * (e >> 1) + 8 * (e & 1);
      qf[e] = live[x] ? __ldg(reinterpret_cast<const uint32_t*>(src[x] + dim)) : 0u;
    }
  }
  float o[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

  for (int st = 0; st < nst; ++st, ++it) {
    const int s = it % kStages;
    const int j0 = item.kv0 + st * kStageTokens;
    if (warp_wait(&sm.full[s], (it / kStages) & 1, &sm.abort)) {
      const uint16_t *ks = &bufs.k[s][0][0][0], *vs = &bufs.v[s][0][0][0];
#pragma unroll
      for (int sl = 0; sl < (kWide ? 2 : 1); ++sl) {
        const int tok0 = kWide ? 32 * (cw & 3) + 16 * sl : 16 * cw;
        if (j0 + tok0 < item.kv1)
          diff_slice<T, kWide>(ks, vs, tok0, j0 + tok0, map, p.scale_log2, var.sink, item.kv1, qf, rw, o);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[s]);
  }

  // Merge of the warps' states, 64 dims at a time through shared memory.
  // Warp w finishes packed row w (and w + 8 of a wide tile).
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const float l = quad_sum(rw.l[x]);
    if (t == 0) sm.comb_ml[cw][g + 8 * x] = make_float2(rw.m[x], l);
  }
  constexpr int kRows = kWide ? 2 : 1, kParts = kWide ? 4 : 8;
  float2 acc[kRows][2][2];  // [row][map][64-dim half]
  float wsum[kRows][2], mmax[kRows][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int nb = 0; nb < 8; ++nb) {
      const int col = (nb ^ g) * 8 + 2 * t;
      *reinterpret_cast<float2*>(&bufs.comb[cw][g][col]) = make_float2(o[8 * h + nb][0], o[8 * h + nb][1]);
      *reinterpret_cast<float2*>(&bufs.comb[cw][g + 8][col]) = make_float2(o[8 * h + nb][2], o[8 * h + nb][3]);
    }
    named_barrier_sync(1, 32 * kConsumerWarps);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (cw + 8 * k < prows) {
#pragma unroll
        for (int mp = 0; mp < 2; ++mp) {
          const int tr = kWide ? cw + 8 * k : cw + 8 * mp;  // tile row
          const int w0 = kWide ? 4 * mp : 0;                // first warp that holds it
          float M = -INFINITY;
#pragma unroll
          for (int i = 0; i < kParts; ++i) M = fmaxf(M, sm.comb_ml[w0 + i][tr].x);
          float2 a = make_float2(0.f, 0.f);
          float L = 0.f;
          if (M != -INFINITY) {
            const int col = ((lane >> 2) ^ (tr & 7)) * 8 + 2 * (lane & 3);
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
              const float2 ml = sm.comb_ml[w0 + i][tr];
              const float w = ex2(ml.x - M);
              const float2 x = *reinterpret_cast<const float2*>(&bufs.comb[w0 + i][tr][col]);
              L += w * ml.y;
              a.x += w * x.x;
              a.y += w * x.y;
            }
          }
          const float inv = L > 0.f ? 1.f / L : 0.f;
          acc[k][mp][h] = make_float2(a.x * inv, a.y * inv);
          mmax[k][mp] = M;
          wsum[k][mp] = L;
        }
      }
    }
    named_barrier_sync(1, 32 * kConsumerWarps);
  }
  if (!sm.abort) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int pr = cw + 8 * k;
      if (pr >= prows) continue;
      const int prow = prow0 + pr, row = item.row0 + prow;
      const int tq = row / G, head = item.hk * G + (row - tq * G);
      const int64_t tok = int64_t(rq.qo_start) + tq;
      const int nrows = item.row1 - item.row0;
      if (item.part < 0) diff_store_row<T>(dp, acc[k][0], acc[k][1], __ldg(dp.lambda + head), tok, head);
#pragma unroll
      for (int mp = 0; mp < 2; ++mp) {
        const float lse = wsum[k][mp] > 0.f ? (mmax[k][mp] + __log2f(wsum[k][mp])) * 0.69314718055994531f : -INFINITY;
        if (item.part < 0) {
          if (p.lse && lane == 0) p.lse[(tok * p.num_qo_heads + head) * 2 + mp] = lse;
        } else {
          const int64_t prw = int64_t(item.part) + mp * nrows + prow;
          float* dst = p.fws + p.partial_o_offset + prw * kHeadDim + 2 * lane;
#pragma unroll
          for (int h = 0; h < 2; ++h) *reinterpret_cast<float2*>(dst + 64 * h) = acc[k][mp][h];
          if (lane == 0) p.fws[prw] = lse;
        }
      }
    }
  }
  return it;
}

template <typename T>
__device__ void diff_consume(const DiffParams& dp, DiffSmem& sm, int32_t item_begin, int32_t item_end,
                             int32_t off_items, int causal, const Variant& var) {
  uint32_t it = 0;
  for (int32_t i = item_begin; i < item_end; ++i) {
    const Item item = load_item(dp.run.iws, off_items, i);
    const int nrows = item.row1 - item.row0;
    for (int prow0 = 0; prow0 < nrows; prow0 += 16) {
      const int prows = min(16, nrows - prow0);
      if (prows <= 8)
        it = diff_pass<T, false>(dp, sm, item, prow0, prows, it, causal, var);
      else
        it = diff_pass<T, true>(dp, sm, item, prow0, prows, it, causal, var);
    }
  }
}

// ---------------------------------------------------------------- kernel

// Where the CTA's items leave the tensor cores: at the first of a request of
// at most 16 packed rows, or, on pages below 8 tokens, of at most 32, which the
// decode path takes in two passes: 16 requests on pages of one token took
// 143 us with 32 rows each (on the tensor cores, where a tile is copied row by
// row, 162), but 209 with 48 (164) and 341 with 80 (165).  The planner puts
// these behind the CTA's larger items.
__device__ __forceinline__ int32_t diff_first_decode_item(const RunParams& p, int32_t begin, int32_t end,
                                                          int32_t off_items) {
  const int lane = threadIdx.x & 31;
  const int most = p.kv[0].page_size < kMinTmaPage ? FI_DIFF_SMALL_PAGE_ROWS : FI_TILE_DECODE;
  for (int32_t i0 = begin; i0 < end; i0 += 32) {
    const bool decode = i0 + lane >= end || !p.kv[0].tc ||
                        __ldg(p.iws + off_items + FI_ITEM_INTS * (i0 + lane) + 9) * p.group <= most;  // its qo_len
    const unsigned m = __ballot_sync(0xffffffffu, decode);
    if (m) return min(end, i0 + __ffs(m) - 1);
  }
  return end;
}

template <typename T, bool kMask>
__global__ void __launch_bounds__(kDiffThreads, 1) diff_attention_kernel(const __grid_constant__ DiffParams dp) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  DiffSmem& sm = *reinterpret_cast<DiffSmem*>(smem_raw);
  const RunParams& p = dp.run;
  if (threadIdx.x == 0) let_dependents_start();
  const int32_t* iws = p.iws;
  // The plan in the workspace has to fit this launch (see the run kernel).
  const int32_t magic = ws_header(iws, FI_H_MAGIC), n_items = ws_header(iws, FI_H_NUM_ITEMS);
  const int32_t n_ctas = ws_header(iws, FI_H_NUM_CTAS), off_cta = ws_header(iws, FI_H_OFF_CTA);
  const int32_t h_rows = ws_header(iws, FI_H_PARTIAL_ROWS), h_qo = ws_header(iws, FI_H_TOTAL_QO);
  const int32_t h_hq = ws_header(iws, FI_H_NUM_QO_HEADS), h_hkv = ws_header(iws, FI_H_NUM_KV_HEADS);
  const int32_t h_page = ws_header(iws, FI_H_PAGE_SIZE);
  bool bad = magic != FI_PLAN_MAGIC_DIFF || n_ctas != int32_t(gridDim.x) || (smem_u32(smem_raw) & 1023u) != 0 ||
             h_rows < 0 || h_rows > p.max_partial_rows || h_qo < 0 || h_qo > p.q_num_tokens ||
             h_hq != p.num_qo_heads || h_hkv != p.num_kv_heads || h_page != p.kv[0].page_size ||
             (!kMask && ws_header(iws, FI_H_WINDOW_LEFT) >= 0);
  int32_t begin = 0, end = 0;
  if (!bad) {
    begin = __ldg(iws + off_cta + blockIdx.x);
    end = __ldg(iws + off_cta + blockIdx.x + 1);
    bad = begin < 0 || end < begin || end > n_items;
  }
  if (bad) {
    if (threadIdx.x == 0) atomicOr(p.iws + FI_H_STATUS, kStatusBadPlan);
    return;
  }
  const int32_t off_items = ws_header(iws, FI_H_OFF_ITEMS);
  const int causal = ws_header(iws, FI_H_CAUSAL);
  Variant var;
  var.window_left = ws_header(iws, FI_H_WINDOW_LEFT);
  var.sink = ws_header(iws, FI_H_SINK_TOKENS);
  var.cap_a = var.cap_b = 0.f;
  var.rope_table = nullptr;
  const int warp = threadIdx.x >> 5;
  const int32_t mid = diff_first_decode_item(p, begin, end, off_items);
  const bool tc_phase = mid > begin;
  const bool boxes = p.kv[0].page_size >= kDiffMinBoxPage;
  DiffPrefillBars& bar = sm.bars;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], boxes ? 1 : 32 * kCopyWarps);  // the producer, or every copying thread
      mbar_init(&sm.empty[s], kConsumerWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.q_full[s], 1);
      mbar_init(&bar.q_empty[s], 2);  // one thread of each pair of softmax warpgroups
      mbar_init(&bar.v_go[s], 1);
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.s_free[s], 4 * kDiffGroups);  // every softmax warp
      mbar_init(&bar.p_full[s], 4 * kDiffGroups);
    }
    for (int s = 0; s < kDiffStages; ++s) {
      mbar_init(&bar.kv_full[s], 1);
      mbar_init(&bar.kv_empty[s], 1);
      mbar_init(&bar.v_clear[s], 1);
    }
    mbar_init(&bar.o_ready, 1);
    mbar_init(&bar.o_free, 4 * kDiffGroups);
    mbar_init(&bar.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (tc_phase && warp == kMmaWarp) {
    tc::tmem_alloc(&sm.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // Each branch returns to the launch's registers before the code paths meet
  // (an increase waits for the other warpgroups' release).
  if (tc_phase) {
    uint32_t loads = 0;
    if (warp < kSoftmaxWarp0) {
      tc::setmaxnreg_dec<kDiffRegsLoader>();
      const bool copies = p.kv[0].page_size < kMinTmaPage;
      if (copies && (warp == 0 || warp == 3)) {
        diff_pf_produce<false, true>(dp, sm.pf, bar, &sm.abort, begin, mid, off_items);
      } else if (copies && warp == kVWarp) {
        diff_pf_produce<true, true>(dp, sm.pf, bar, &sm.abort, begin, mid, off_items);
      } else if (warp == 0) {
        loads = diff_pf_produce<false, false>(dp, sm.pf, bar, &sm.abort, begin, mid, off_items);
      } else if (warp == kMmaWarp) {
        diff_pf_mma<T>(p, sm.pf, bar, &sm.abort, sm.tmem_base, begin, mid, off_items);
        __syncwarp();
      } else if (warp == kVWarp) {
        loads = diff_pf_produce<true, false>(dp, sm.pf, bar, &sm.abort, begin, mid, off_items);
      }
      tc::fence_before_sync();
      named_barrier_sync_unaligned(kPhaseBarrier, kDiffThreads);
      tc::fence_after_sync();
      tc::setmaxnreg_inc<kDiffRegsLaunch>();
    } else {
      tc::setmaxnreg_inc<kDiffRegsSoftmax>();
      diff_pf_softmax<T, kMask>(dp, sm.pf, bar, &sm.abort, sm.tmem_base, begin, mid, off_items, causal, var);
      tc::setmaxnreg_dec<kDiffRegsLaunch>();
      tc::fence_before_sync();
      named_barrier_sync_unaligned(kPhaseBarrier, kDiffThreads);
      tc::fence_after_sync();
    }
    if (sm.abort) {  // no role is left that could set it: all threads take this branch or none
      diff_pf_drain(bar, loads);
      named_barrier_sync_unaligned(kPhaseBarrier, kDiffThreads);
    }
  }
  if (mid < end) {
    if (warp >= kFirstConsumerWarp && warp < kFirstConsumerWarp + kConsumerWarps) {
      tc::setmaxnreg_inc<kDiffRegsConsumer>();
      diff_consume<T>(dp, sm, mid, end, off_items, causal, var);
    } else {
      tc::setmaxnreg_dec<kDiffRegsOther>();
      const int copier = diff_copy_warp(warp);
      if (boxes) {
        if (warp == 0) diff_produce_tma(dp, sm, mid, end, off_items);
      } else if (copier >= 4) {
        diff_produce<true>(dp, sm, copier - 4, mid, end, off_items);
      } else if (copier >= 0) {
        diff_produce<false>(dp, sm, copier, mid, end, off_items);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (tc_phase && warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(sm.tmem_base, kTmemCols);
  }
  if (threadIdx.x == 0 && sm.abort) atomicOr(p.iws + FI_H_STATUS, sm.abort);
}

constexpr int kMergeAhead = 4;  // chunks whose partial outputs a warp has in flight

// Merge of split units, launched behind the run: one warp per packed row, its
// chunks' partial states of both maps in chunk order, then the row's output.
// Counts come from the workspace, so a captured graph serves later plans.
template <typename T>
__global__ void __launch_bounds__(256) diff_merge_kernel(const __grid_constant__ DiffParams dp) {
  const RunParams& p = dp.run;
  const int32_t* iws = p.iws;
  const int lane = threadIdx.x & 31;
  const int32_t rows_max = iws[FI_H_CASCADE_ROWS_MAX], units = iws[FI_H_NUM_MERGE];
  const int4* merge = reinterpret_cast<const int4*>(iws + iws[FI_H_OFF_MERGE]);
  const int32_t* reqs = iws + iws[FI_H_OFF_REQUESTS];
  if (iws[FI_H_MAGIC] != FI_PLAN_MAGIC_DIFF || units < 1 || rows_max < 1) {
    grid_dependency_wait();
    return;
  }
  // Row pr of a unit per warp, rows_max rows a unit.  A unit's words are
  // fetched a task ahead, the first before the run has ended.
  const int32_t warps = int32_t(gridDim.x * (blockDim.x >> 5));
  const int32_t me = int32_t(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5));
  const int32_t unit_step = warps / rows_max, row_step = warps % rows_max;
  int32_t unit = me / rows_max, row = me % rows_max;
  int4 next0 = make_int4(0, 0, 0, 0), next1 = next0;
  auto fetch = [&] {
    if (unit < units) {
      next0 = __ldg(merge + FI_MERGE_INTS / 4 * int64_t(unit));
      next1 = __ldg(merge + FI_MERGE_INTS / 4 * int64_t(unit) + 1);
    }
  };
  fetch();
  grid_dependency_wait();
  if (iws[FI_H_STATUS] != 0) return;
  while (unit < units) {
    const int4 u0 = next0, u1 = next1;  // {b, hk, row0, row1}, {n, base, late, 0}
    const int pr = row, nrows = u0.w - u0.z, n = u1.x;
    unit += unit_step;
    row += row_step;
    if (row >= rows_max) {
      row -= rows_max;
      ++unit;
    }
    fetch();
    if (pr >= nrows) continue;
    const int qrow = u0.z + pr, tq = qrow / p.group, head = u0.y * p.group + (qrow - tq * p.group);
    const float lam = __ldg(dp.lambda + head);
    const int64_t tok = int64_t(__ldg(reqs + FI_REQ_INTS * u0.x)) + tq;
    // Partial row of chunk c: row0[map] + c step.  Lane c holds chunk c's two
    // log-sum-exps (32 at a time); kMergeAhead chunks' partial outputs are in
    // flight, the first of them beside the log-sum-exps.
    const int64_t step = 2 * nrows, row0[2] = {int64_t(u1.y) + pr, int64_t(u1.y) + nrows + pr};
    float2 v[kMergeAhead][2][2];
    auto load = [&](int c) {
#pragma unroll
      for (int u = 0; u < kMergeAhead; ++u)
#pragma unroll
        for (int mp = 0; mp < 2; ++mp) {
          const float2* src = reinterpret_cast<const float2*>(
                                  p.fws + p.partial_o_offset + (row0[mp] + (c + u) * step) * kHeadDim) + lane;
          v[u][mp][0] = c + u < n ? __ldcg(src) : make_float2(0.f, 0.f);
          v[u][mp][1] = c + u < n ? __ldcg(src + 32) : make_float2(0.f, 0.f);
        }
    };
    load(0);
    auto lse_of = [&](int c, int mp) { return c < n ? __ldcg(p.fws + row0[mp] + c * step) : -INFINITY; };
    const float e0[2] = {lse_of(lane, 0), lse_of(lane, 1)};
    float M[2] = {e0[0], e0[1]}, L[2] = {0.f, 0.f};
    for (int c = lane + 32; c < n; c += 32) {
      M[0] = fmaxf(M[0], lse_of(c, 0));
      M[1] = fmaxf(M[1], lse_of(c, 1));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      M[0] = fmaxf(M[0], __shfl_xor_sync(0xffffffffu, M[0], off));
      M[1] = fmaxf(M[1], __shfl_xor_sync(0xffffffffu, M[1], off));
    }
    float2 a[2][2];
#pragma unroll
    for (int mp = 0; mp < 2; ++mp) a[mp][0] = a[mp][1] = make_float2(0.f, 0.f);
    float w[2] = {0.f, 0.f};
    for (int c = 0; c < n; c += kMergeAhead) {
      if ((c & 31) == 0) {
#pragma unroll
        for (int mp = 0; mp < 2; ++mp) {
          const float e = c == 0 ? e0[mp] : lse_of(c + lane, mp);
          w[mp] = M[mp] != -INFINITY ? ex2((e - M[mp]) * 1.4426950408889634f) : 0.f;
          L[mp] += w[mp];
        }
      }
#pragma unroll
      for (int u = 0; u < kMergeAhead; ++u)
#pragma unroll
        for (int mp = 0; mp < 2; ++mp) {
          const float wu = __shfl_sync(0xffffffffu, w[mp], (c + u) & 31);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a[mp][h].x += wu * v[u][mp][h].x;
            a[mp][h].y += wu * v[u][mp][h].y;
          }
        }
      if (c + kMergeAhead < n) load(c + kMergeAhead);
    }
    float2 s[2][2];
    float lse[2];
#pragma unroll
    for (int mp = 0; mp < 2; ++mp) {
      const float sum = warp_sum(L[mp]), inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) s[mp][h] = make_float2(a[mp][h].x * inv, a[mp][h].y * inv);
      lse[mp] = sum > 0.f ? M[mp] + __logf(sum) : -INFINITY;
    }
    diff_store_row<T>(dp, s[0], s[1], lam, tok, head);
    if (p.lse && lane < 2) p.lse[(tok * p.num_qo_heads + head) * 2 + lane] = lane ? lse[1] : lse[0];
  }
}

}  // namespace fi
