// kv4_prefill.cuh -- prefill-class items over the 4-bit cache, on the 5th-
// generation tensor cores.
//
// Items, tiles and the order of the products are those of prefill_kernel.cuh: up
// to two 128-row M tiles against 128-key tiles, S = Q K^T into tensor memory, P
// over it as 16-bit pairs, O += P V.  What differs is where the operands come
// from.  A value s (n - z) has seven significant bits of s times four of n - z:
// eleven, an fp16 as it stands (fi_kv4.h), so K and V tiles are exact fp16 tiles;
// a bf16 row of Q is brought into fp16 by a power of two of its own, which its
// softmax takes back.  (K as n - z in bf16 beside Q as it is, each key's s
// multiplied to its column of S, was slower: the widening, whose warps are the
// busiest, doubled for K.)
//
//  * warp 0 brings the pages' blocks, 64 keys a stage, a raw stage for each half
//    of a tile (a bulk copy a block, page ids a stage ahead);
//  * warps 4 .. 7 are the 128 keys of a tile: a thread has its key's scale and
//    zero point in registers and turns its two rows of 64 bytes into 256 bytes
//    each, in the 128-byte swizzle that the products read: for eight codes one
//    shift, four (x & m) | c (1024 + n and 64 + n as fp16), four subtractions of
//    the same with z, four products with s.  The codes come out in the order 0, 4,
//    1, 5, 2, 6, 3, 7 of each eight dims; Q's rows are put in it too, and the
//    output right where it is stored.  Reads and writes of a quarter warp meet no
//    bank twice: lane l starts with quarter l / 2 of its row;
//  * warp 2 loads Q (one TMA box a 64-dim half of an M tile where the group
//    divides 128, else warps 2 and 3 copy its rows), and warps 4 .. 7 turn the rows
//    of M tile A, warps 2 and 3 those of B, a thread a row, in place;
//  * warp 1 issues the products (pf_mma), warps 8 .. 15 the softmax.
//
// What bounds it: no one unit, but the chain of a tile of 128 keys, 3.3 thousand
// clocks.  An M tile's S has no second buffer in tensor memory, so its softmax
// (2.1 thousand) and its P V and next S (1.1) follow one another, the other M tile's
// between them; widening a tile takes 2.3.  Tensor cores are busy half of that time,
// issue slots for 59 %.  Eight prompts of 128 to 2048 tokens behind up to 2048,
// 32 + 8 heads: 318 us (in fp16 304), 1.1 PFLOP/s (188 us at the rate of plain bf16
// products; 285 us from a cache in 16 bits, four times the memory).  What it took:
// straight code as short as can be (the roles' loops together are longer than the
// instruction cache: the widening unrolled cost 80 us), one row sum (22 us), hidden
// keys as bits and once a tile, and output by four lanes a row (together 22 us, and 6
// of every short call).  Not kept: units of 64 keys with S two units ahead, whose
// products read Q twice as often and need half again the instructions (364 us).
#pragma once
#include <cfloat>

#include "kv4_params.h"
#include "attention_kernel.cuh"
#include "kv4_layout.h"

namespace fi {

constexpr int kKv4RawKeys = 64;     // keys of a raw stage
constexpr int kKv4RawStages = kTileN / kKv4RawKeys;  // a stage's readers are the same two warps, tile after tile
constexpr int kKv4RawBytes = 9216;  // 64 blocks of one slot, 144 bytes each
constexpr int kKv4QuantWarp0 = 4, kKv4QuantWarps = 4;
constexpr int kKv4SoftmaxWarp0 = 8;
constexpr float kKv4Lazy = 4.f, kKv4Room = 11.f;  // log2, of the weights: see kv4_pf_softmax
static_assert(kKv4Lazy + kKv4Room <= 15.f, "weights pass fp16's end");

struct Kv4PrefillBufs {
  uint16_t q[2][2][kTileM][64];  // [M tile][d half][row][dim], and so on as in PrefillBufs
  uint16_t k[2][2][kTileN][64];
  uint16_t v[2][2][kTileN][64];
  alignas(128) uint8_t raw[kKv4RawStages][kKv4RawBytes];
  float q_scale[2][2 * kTileM];  // [item's parity][row]: log2-domain factor of the row's products, FLT_MIN at least (a hidden
                                 // key's -inf times 0 would be a NaN; logits that small are 0)
  uint32_t good[kKv4RawStages][2];  // keys of a raw stage whose page lies in the cache, a bit each
};

// The raw stages of items [b0, b1), whole warp.
template <int kB, typename Smem>
__device__ void kv4_pf_load(const Kv4Params& kp, Smem& sm, int32_t b0, int32_t b1, int32_t off_items) {
  const RunParams& p = kp.run;
  const KvCache& kc = p.kv[0];
  const int lane = threadIdx.x & 31;
  const int log2_slots = kB == 32 ? 5 : kB == 16 ? 4 : kp.log2_block, bytes = kB ? kv4_block_bytes(kB) : kp.block_bytes;
  const int blocks = kKv4RawKeys >> log2_slots;  // 2 .. 64: up to two a lane
  uint32_t n = 0;
  bool ok = true;
  for (int32_t i = b0; i < b1 && ok; ++i) {
    const Item it = load_item(p.iws, off_items, i);
    const int stages = 2 * item_kv_tiles(it);  // a tile's second half may have no key
    const int npages = (it.rq.kv_len + kc.page_size - 1) >> kc.log2_page;
    const int32_t* pages = kc.kv_indices + it.rq.page_start;
    const uint8_t* head = kp.cache + it.hk * kp.head_stride;
    int32_t next[2];
    auto fetch = [&](int st) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int b = lane + 32 * u, key = kKv4RawKeys * st + (b << log2_slots);
        const int pg = (it.kv0 + key) >> kc.log2_page;
        next[u] = b < blocks && key < it.kv1 - it.kv0 && pg < npages ? __ldg(pages + pg) : -1;
      }
    };
    if (stages > 0) fetch(0);
    for (int st = 0; st < stages; ++st, ++n) {
      const int slot = n % kKv4RawStages;  // the half of the tile
      const int32_t id[2] = {next[0], next[1]};
      if (st + 1 < stages) fetch(st + 1);
      ok = warp_wait(&sm.raw_empty[slot], ((n / kKv4RawStages) & 1) ^ 1, &sm.abort);
      if (!ok) break;
      const bool in0 = uint32_t(id[0]) < uint32_t(kc.num_pages), in1 = uint32_t(id[1]) < uint32_t(kc.num_pages);
      const uint32_t m0 = __ballot_sync(0xffffffffu, in0), m1 = __ballot_sync(0xffffffffu, in1);
      auto has = [&](int key) {
        const int b = key >> log2_slots;
        return ((b < 32 ? m0 : m1) >> (b & 31)) & 1u;
      };
      const uint32_t g0 = __ballot_sync(0xffffffffu, has(lane)), g1 = __ballot_sync(0xffffffffu, has(32 + lane));
      if (lane == 0) {
        sm.pf.good[slot][0] = g0;
        sm.pf.good[slot][1] = g1;
        mbar_arrive_expect_tx(&sm.raw_full[slot], (__popc(m0) + __popc(m1)) * bytes);
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int b = lane + 32 * u, key = it.kv0 + kKv4RawKeys * st + (b << log2_slots);
        if (u ? in1 : in0)
          bulk_load(&sm.pf.raw[slot][b * bytes],
                    head + id[u] * kp.page_stride + int64_t((key & (kc.page_size - 1)) >> log2_slots) * bytes, bytes,
                    &sm.raw_full[slot]);
      }
    }
  }
  // every copy has landed before the CTA moves on
  if (lane == 0)
    for (uint32_t x = n > kKv4RawStages ? n - kKv4RawStages : 0; x < n; ++x)
      mbar_wait_drain(&sm.raw_full[x % kKv4RawStages], (x / kKv4RawStages) & 1);
  __syncwarp();
}

// One row of 64 bytes of codes to 256 bytes of fp16 in row r of the tile at `tile`
// (shared-memory address); c0 .. c3: quarters lane / 2 .. lane / 2 + 3 modulo 4.
// A loop of one quarter: its warps share the instruction caches with the softmax's,
// whose loop is long.
__device__ __forceinline__ void kv4_widen(uint4 c0, uint4 c1, uint4 c2, uint4 c3, uint32_t scale, uint32_t z,
                                          uint32_t tile, int r) {
  const int lane = threadIdx.x & 31;
  auto twice = [](uint32_t x) {
    x |= x << 16;
    return *reinterpret_cast<const __half2*>(&x);
  };
  const __half2 s = twice(scale), z0 = twice(0x6400u + z), z1 = twice(0x5400u + (z << 4));
  auto value = [&](uint32_t codes, __half2 zero) {
    const __half2 x = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&codes), zero), s);
    return *reinterpret_cast<const uint32_t*>(&x);
  };
  const uint32_t row = tile + r * 128 + 16 * (r & 7);  // 16-byte chunk c of the row lies at 16 (c ^ r % 8)
#pragma unroll 1
  for (int u = 0; u < 4; ++u) {
    const int quarter = (u + (lane >> 1)) & 3;
    const uint32_t w[4] = {c0.x, c0.y, c0.z, c0.w};
    const uint32_t at = (row ^ (64 * (quarter & 1))) + (quarter >> 1) * (kTileN * 128);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t h = w[e] >> 8;
      const uint4 out = make_uint4(value((w[e] & 0x000F000Fu) | 0x64006400u, z0), value((w[e] & 0x00F000F0u) | 0x54005400u, z1),
                                   value((h & 0x000F000Fu) | 0x64006400u, z0), value((h & 0x00F000F0u) | 0x54005400u, z1));
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (16 * e)), "r"(out.x), "r"(out.y), "r"(out.z),
                   "r"(out.w)
                   : "memory");
    }
    c0 = c1;
    c1 = c2;
    c2 = c3;
  }
}

// Row r of an M tile in place: the dims of each eight in the order 0, 4, 1, 5, ..,
// and a bf16 row times a power of two that brings its largest value into [2^14,
// 2^15), as fp16; returns the factor that takes it back.
template <typename T>
__device__ __forceinline__ float kv4_turn_query(uint16_t (*tile)[kTileM][64], int r) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  float up = 1.f, back = 1.f;
  if constexpr (kBf16) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    auto larger = [](uint32_t a, uint32_t b) {
      const __nv_bfloat162 m =
          __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    };
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 16; ++c) {  // chunk order does not matter: c ^ r is every chunk once
      const uint4 u = *reinterpret_cast<const uint4*>(tile[c >> 3][r] + 8 * ((c & 7) ^ (r & 7)));
      top = larger(top, larger(larger(u.x & kAbs, u.y & kAbs), larger(u.z & kAbs, u.w & kAbs)));
    }
    top = larger(top, top >> 16);
    const int ex = min(max(int(top >> 7 & 0xFF) - 127, -100), 100);
    up = __int_as_float((127 + 14 - ex) << 23);
    back = __int_as_float((127 - 14 + ex) << 23);
  }
#pragma unroll 4
  for (int c = 0; c < 16; ++c) {
    uint4* const at = reinterpret_cast<uint4*>(tile[c >> 3][r] + 8 * ((c & 7) ^ (r & 7)));
    const uint4 u = *at;
    if constexpr (kBf16) {
      float f[8];
      unpack8<T>(u, f);
      *at = make_uint4(tc::pack2<__half>(f[0] * up, f[4] * up), tc::pack2<__half>(f[1] * up, f[5] * up),
                       tc::pack2<__half>(f[2] * up, f[6] * up), tc::pack2<__half>(f[3] * up, f[7] * up));
    } else {
      *at = make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                       __byte_perm(u.y, u.w, 0x7632));
    }
  }
  return back;
}

// K and V tiles of items [b0, b1), thread = key of a tile; and M tile A's rows.
template <typename T, int kB, typename Smem>
__device__ void kv4_pf_widen(const Kv4Params& kp, Smem& sm, int32_t b0, int32_t b1, int32_t off_items) {
  const int r = threadIdx.x - 32 * kKv4QuantWarp0, lane = threadIdx.x & 31, half = r / kKv4RawKeys;
  const int slots = kB ? kB : kp.block_slots, log2_slots = kB == 32 ? 5 : kB == 16 ? 4 : kp.log2_block;
  const int bytes = kB ? kv4_block_bytes(kB) : kp.block_bytes;
  const int key = r % kKv4RawKeys, place = key & (slots - 1);
  const uint8_t* const raw = sm.pf.raw[half] + (key >> log2_slots) * bytes;
  uint32_t kt = 0, pe = 0;
  for (int32_t i = b0; i < b1; ++i) {
    const Item it = load_item(kp.run.iws, off_items, i);
    const int ntiles = item_kv_tiles(it);
    for (int j = 0; j < ntiles; ++j, ++kt) {
      const int st = kt & 1;
      if (!warp_wait(&sm.raw_full[half], kt & 1, &sm.abort)) return;
      // the words, with a finite scale whatever the bytes; 0 outside the cache
      const uint32_t good = sm.pf.good[half][key >> 5] >> (key & 31) & 1u ? 0xFFF0u : 0u;
      const uint32_t kw = *reinterpret_cast<const uint16_t*>(raw + kv4_k_word(slots, place));
      const uint32_t vw = *reinterpret_cast<const uint16_t*>(raw + kv4_v_word(slots, place));
      uint4 k[4], v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = 16 * ((u + (lane >> 1)) & 3);
        k[u] = *reinterpret_cast<const uint4*>(raw + kv4_k_row(slots, place) + at);
        v[u] = *reinterpret_cast<const uint4*>(raw + kv4_v_row(slots, place) + at);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.raw_empty[half]);
      if (!warp_wait(&sm.k_empty[st], ((kt >> 1) & 1) ^ 1, &sm.abort)) return;
      kv4_widen(k[0], k[1], k[2], k[3], min(kw & good, uint32_t(kKv4MaxScaleBits)), kw & 15u, smem_u32(sm.pf.k[st]), r);
      fence_proxy_async_smem();  // read by the tensor core
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.k_full[st]);
      if (j == 0) {
        if (!warp_wait(&sm.q_raw, pe & 1, &sm.abort)) return;
        sm.pf.q_scale[pe & 1][r] = fmaxf(kp.run.scale_log2 * kv4_turn_query<T>(sm.pf.q[0], r), FLT_MIN);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full);
        ++pe;
      }
      if (!warp_wait(&sm.v_empty[st], ((kt >> 1) & 1) ^ 1, &sm.abort)) return;
      kv4_widen(v[0], v[1], v[2], v[3], min(vw & good, uint32_t(kKv4MaxScaleBits)), vw & 15u, smem_u32(sm.pf.v[st]), r);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.v_full[st]);
    }
  }
}

// Q of items [b0, b1) by warps 2 and 3 (which = 0, 1): its load, and M tile B's rows.
template <typename T, typename Smem>
__device__ void kv4_pf_queries(const Kv4Params& kp, Smem& sm, int which, int32_t b0, int32_t b1, int32_t off_items) {
  const RunParams& p = kp.run;
  const int lane = threadIdx.x & 31, c = lane & 15, G = p.group;
  const bool boxes = p.kv[0].tc != 0;
  uint32_t pe = 0;
  int armed = -1;  // parity of the last load
  for (int32_t i = b0; i < b1; ++i) {
    const Item it = load_item(p.iws, off_items, i);
    if (item_kv_tiles(it) == 0) continue;
    const int nrows = it.row1 - it.row0, nm = item_m_tiles(it);
    bool ok = warp_wait(&sm.q_empty, (pe & 1) ^ 1, &sm.abort);
    if (!ok) break;
    if (boxes) {
      if (which == 0) {
        if (lane == 0) {
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(&sm.q_raw, nm * kQTileBytes);
          for (int m = 0; m < nm; ++m) {
            const int c1 = it.hk * G, c2 = it.rq.qo_start + (it.row0 + m * kTileM) / G;
            tc::tma_load_3d(&sm.pf.q[m][0][0][0], &p.tm_q, &sm.q_raw, 0, c1, c2);
            tc::tma_load_3d(&sm.pf.q[m][1][0][0], &p.tm_q, &sm.q_raw, 64, c1, c2);
          }
        }
        armed = pe & 1;
      }
    } else {
      const int first = it.row0 + 2 * which + (lane >> 4);
      int tok = first / G, g = first - tok * G;
      for (int row = 2 * which + (lane >> 4); row < nm * kTileM; row += 4) {
        const uint16_t* src = row < nrows ? p.q + (int64_t(it.rq.qo_start) + tok) * p.q_stride_tok +
                                                int64_t(it.hk * G + g) * p.q_stride_head + 8 * c
                                          : p.q;
        cp_async_16(&sm.pf.q[row / kTileM][c >> 3][row % kTileM][8 * ((c & 7) ^ (row & 7))], src, row < nrows ? 16u : 0u);
        for (g += 4; g >= G; g -= G) ++tok;
      }
      cp_async_wait_all();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_raw);
    }
    ok = warp_wait(&sm.q_raw, pe & 1, &sm.abort);
    if (!ok) break;
    if (nm == 2)
      for (int r = 32 * which + lane; r < kTileM; r += 64)
        sm.pf.q_scale[pe & 1][kTileM + r] = fmaxf(p.scale_log2 * kv4_turn_query<T>(sm.pf.q[1], r), FLT_MIN);
    fence_proxy_async_smem();  // read by the tensor core
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);
    ++pe;
  }
  if (armed >= 0 && lane == 0) mbar_wait_drain(&sm.q_raw, armed);
  __syncwarp();
}

// The first n of 32 bits.
__device__ __forceinline__ uint32_t kv4_below(int n) {
  uint32_t rest;
  asm("shl.b32 %0, %1, %2;" : "=r"(rest) : "r"(0xffffffffu), "r"(max(n, 0)));  // 0 from 32 on
  return ~rest;
}

// The softmax of the M tiles (see pf_softmax): thread = row = TMEM lane.
template <typename T, bool kMask, typename Smem>
__device__ void kv4_pf_softmax(const RunParams& p, Smem& sm, int32_t b0, int32_t b1, int32_t off_items,
                               int32_t off_merge, int32_t off_cnt, int causal, const Variant var) {
  const int sw = (threadIdx.x >> 5) - kKv4SoftmaxWarp0, mt = sw >> 2, w = sw & 3, lane = threadIdx.x & 31;
  const int r = 32 * w + lane, tid = mt * kTileM + r;
  const uint32_t tl = sm.tmem_base + (uint32_t(32 * w) << 16);
  const uint32_t s_cols = tl + mt * kTileN, o_cols = tl + kTmemO + mt * kHeadDim;
  const int G = p.group;
  uint32_t tiles = 0, items = 0, seq = 0;  // phases of s_full[mt] and o_ready[mt]; items with keys
  for (int32_t i = b0; i < b1; ++i) {
    const Item item = load_item(p.iws, off_items, i);
    const Request& rq = item.rq;
    const int nrows = item.row1 - item.row0;
    const int ntiles = item_kv_tiles(item);
    const int prow = mt * kTileM + r;  // packed row within the item
    if (mt < item_m_tiles(item)) {
      // visible keys of this row: [lo, lim] and the sink (a padding row, which is not stored: all, so that its warp has
      // no key to hide)
      int lim = INT32_MAX - 1, lo = 0;
      if (prow < nrows) {
        const int pos = rq.kv_len - rq.qo_len + (item.row0 + prow) / G;
        lim = min(causal ? pos : rq.kv_len - 1, item.kv1 - 1);
        if (kMask) lo = window_low(var, pos);
      }
      // lrun: sum of the fp32 P.  The product takes them in fp16, each off by at most half a step, 2^-11 of itself (what the
      // roundings of a row have in common does not cancel, as it would in the sum of the rounded ones; that sum beside this
      // one took 7 % of the time).  fp16 has few powers of two, so a row's P are held 2^kKv4Room up: those down to
      // 2^-(14 + kKv4Room) of the largest are rounded to 11 bits, those below off by 2^-(25 + kKv4Room) at most.  Their
      // largest is 2^(kKv4Lazy + kKv4Room), for the running maximum moves when the logits pass it by more than 2^kKv4Lazy.
      float mrun = -INFINITY, lrun = 0.f, c = 0.f;
      bool ok = true;
      for (int j = 0; j < ntiles; ++j) {
        ok = ok && warp_wait(&sm.s_full[mt], tiles & 1, &sm.abort);
        ++tiles;
        if (!ok) continue;
        tc::fence_after_sync();
        if (j == 0) c = sm.pf.q_scale[seq & 1][prow];
        const int kbase = item.kv0 + j * kTileN;
        // causal diagonal, chunk end, window
        const bool edge = __any_sync(0xffffffffu, kbase + kTileN - 1 > lim || (kMask && kbase < lo));
        uint32_t sv[2][32];
        auto load = [&](int half) {  // 64 columns of S
          tc::tmem_ld32(s_cols + 64 * half, sv[0]);
          tc::tmem_ld32(s_cols + 64 * half + 32, sv[1]);
          tc::tmem_ld_wait();
        };
        // row max in four independent chains of three-input maxima
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          load(half);
          if (edge) {  // the hidden keys' columns -inf, here and for the second pass over them
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k0 = kbase + 64 * half + 32 * h;
              uint32_t seen = kv4_below(lim - k0 + 1);
              if (kMask) seen &= ~kv4_below(lo - k0) | kv4_below(var.sink - k0);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(seen & (1u << e))) sv[h][e] = 0xff800000u;  // -inf
              tc::tmem_st32(s_cols + 64 * half + 32 * h, sv[h]);
            }
          }
#pragma unroll
          for (int e = 0; e < 64; e += 8)
#pragma unroll
            for (int a = 0; a < 4; ++a)
              mx4[a] = max3(mx4[a], __uint_as_float(sv[e >> 5][(e & 31) + a]), __uint_as_float(sv[e >> 5][(e & 31) + 4 + a]));
        }
        if (edge) tc::tmem_st_wait();
        const float mx = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]) * c;
        const float m_old = mrun;
        const float m_new = (mx > m_old + kKv4Lazy) ? mx : m_old;
        const bool rescale = (m_new != m_old) && j > 0;
        if (__any_sync(0xffffffffu, rescale)) {
          // O holds P V of every earlier tile (covered by this S's commit)
          const float alpha = rescale ? ex2(m_old - m_new) : 1.f;
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            tc::tmem_ld32(o_cols + 32 * h, sv[0]);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[0][e] = __float_as_uint(__uint_as_float(sv[0][e]) * alpha);
            tc::tmem_st32(o_cols + 32 * h, sv[0]);
          }
          tc::tmem_st_wait();
          if (rescale) lrun *= alpha;
        }
        // P = 2^(s c - m + kKv4Room) as fp16 pairs over the first 64 columns of the S
        // buffer, published in two halves of 64 keys each
        const float msub = (m_new == -INFINITY) ? 0.f : m_new - kKv4Room;
        const float2 cc = make_float2(c, c), nms = make_float2(-msub, -msub);
        float2 sum4[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) sum4[a] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          load(half);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 x = fma2(make_float2(__uint_as_float(sv[h][2 * e]), __uint_as_float(sv[h][2 * e + 1])), cc, nms);
              const float2 pe = make_float2(ex2(x.x), ex2(x.y));
              sum4[e & 3] = add2(sum4[e & 3], pe);
              pk[e] = tc::pack2<__half>(pe.x, pe.y);
            }
            tc::tmem_st16(s_cols + 32 * half + 16 * h, pk);
          }
          tc::tmem_st_wait();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[mt][half]);
        }
        const float2 s01 = add2(sum4[0], sum4[1]), s23 = add2(sum4[2], sum4[3]), s4 = add2(s01, s23);
        lrun += s4.x + s4.y;
        mrun = m_new;
      }
      bool have_o = false;
      if (ntiles > 0) {
        ok = ok && warp_wait(&sm.o_ready[mt], items & 1, &sm.abort);
        ++items;
        have_o = ok;
      }
      // The row's values go back to tensor memory in their type, and from there to the lanes that store them: four lanes a
      // row, 64 contiguous bytes (a lane a row met a cache line of its own in every store: 3 us an item).
      const float inv = lrun > 0.f ? 1.f / lrun : 0.f;
      const bool partial = item.part >= 0;
      int64_t at = -1;  // of the row, in bytes
      if (prow < nrows && !sm.abort) {
        const float lse = lrun > 0.f ? (mrun - kKv4Room + __log2f(lrun)) * 0.69314718055994531f : -INFINITY;
        const int row = item.row0 + prow, t = row / G, head = item.hk * G + (row - t * G);
        const int64_t tok = int64_t(rq.qo_start) + t, part = int64_t(item.part) + prow;
        if (partial) {
          at = 4 * kHeadDim * part;
          p.fws[part] = lse;
        } else {
          at = 2 * (tok * p.o_stride_tok + int64_t(head) * p.o_stride_head);
          if (p.lse) p.lse[tok * p.num_qo_heads + head] = lse;
        }
      }
      if (have_o) tc::fence_after_sync();
      // Word 4 i + e (e < 4) of 16 goes to column 2 i + e (e < 2) or 2 i + e + 6.  Dim d of each eight of O lies in column
      // 2 d (d < 4) or 2 d - 7.
      constexpr auto word_of = [](int column) { return (column & ~15) + 4 * ((column >> 1) & 3) + 2 * (column >> 3 & 1) + (column & 1); };
      constexpr auto column_of = [](int dim) { return (dim & ~7) + ((dim & 7) < 4 ? 2 * (dim & 7) : 2 * (dim & 7) - 7); };
      uint32_t ov[2][32], out[32];
#pragma unroll
      for (int e = 0; e < 64; ++e) ov[e >> 5][e & 31] = 0u;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (have_o) {
          tc::tmem_ld32(o_cols + 64 * h, ov[0]);
          tc::tmem_ld32(o_cols + 64 * h + 32, ov[1]);
          tc::tmem_ld_wait();
        }
        auto dim = [&](int d) { return __uint_as_float(ov[column_of(d) >> 5][column_of(d) & 31]) * inv; };
        if (partial) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int e = 0; e < 32; ++e) out[e] = __float_as_uint(dim(word_of(32 * u + e)));
            tc::tmem_st32(o_cols + 64 * h + 32 * u, out);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) out[e] = tc::pack2<T>(dim(2 * word_of(e)), dim(2 * word_of(e) + 1));
          tc::tmem_st32(o_cols + 32 * h, out);
        }
      }
      tc::tmem_st_wait();
      uint8_t* const rows = partial ? reinterpret_cast<uint8_t*>(p.fws + p.partial_o_offset) : reinterpret_cast<uint8_t*>(p.o);
#pragma unroll 1
      for (int n = 0; n < (partial ? 4 : 2); ++n) {  // 16 rows, 256 bytes of each
        tc::tmem_ld_quads(o_cols + (uint32_t(16 * (n & 1)) << 16) + 64 * (n >> 1), out);
        tc::tmem_ld_wait();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int64_t to = __shfl_sync(0xffffffffu, at, 16 * (n & 1) + 8 * u + (lane >> 2));
          if (to >= 0) {
            uint4* const dst = reinterpret_cast<uint4*>(rows + to + 256 * (n >> 1)) + (lane & 3);
#pragma unroll
            for (int g = 0; g < 4; ++g)
              dst[4 * g] = make_uint4(out[8 * g + 2 * u], out[8 * g + 2 * u + 1], out[8 * g + 4 + 2 * u], out[8 * g + 5 + 2 * u]);
          }
          __syncwarp();
        }
      }
      if (have_o) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_free[mt]);
      }
    }
    if (ntiles > 0) ++seq;
    if (item.merge >= 0)
      merge_split_unit<T>(p, item, rq, off_merge, off_cnt, tid, kSoftmaxThreads, 2, &sm.merge_last_pf, sm.abort);
  }
}

}  // namespace fi
