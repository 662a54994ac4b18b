// diff_prefill.cuh -- prefill-class items of differential attention on the
// 5th-generation tensor cores.
//
// An item is up to 128 packed query rows against a chunk of keys; its two M
// tiles are the two softmax maps of the same rows.  Map m multiplies dims
// 64 m .. 64 m + 63 of the one Q tile and of K, and both multiply the same V.
// K and V arrive in 128-key tiles and are used in sub-tiles of 64 keys.
//
// Roles: warp 0 loads Q (two buffers) and K, warp 2 V, by TMA; warp 1 issues
// the products; warps 4..7 take the softmax of map 1, warps 8..11 that of map
// 2 (thread = row = tensor-memory lane).  Tensor memory: per map two S
// buffers of 64 columns and O of 128.  The S product runs two sub-tiles ahead
// of P V, across items: while a warpgroup works on S(n), S(n + 1) is there
// already, so the only chain is a map's own softmax.
//
// P is kept as two 16-bit terms, hi + lo, both multiplied with V: the output
// is a difference, in which the maps' common part cancels and the rounding of
// the weights does not (with P of one term the output was 1.5 times further
// from the 64-bit result than its own rounding, at random keys; more where
// the maps agree more).  A sub-tile's hi and lo fill the columns of its S.
//
// Per 64 keys and map: S 4 and P V 8 products of M128 K16, 128 + 512 cycles
// of the tensor pipe; both maps 1280.  The softmax of a sub-tile is some 350
// instructions a warp, two warps on each scheduler.
#pragma once
#include "attention_kernel.cuh"
#include "diff_params.h"

namespace fi {

constexpr int kSubKeys = 64;
constexpr int kDiffBarrier = 6;  // both softmax warpgroups (1: decode, 3: end of phase, 4 and 5: one warpgroup)

struct DiffPrefillBufs {  // every [128][64] block is a 128-byte swizzled operand half (see PrefillBufs)
  uint16_t q[2][2][kTileM][64];    // [buffer][d half = map][row][dim]
  uint16_t k[2][2][kTileN][64];    // [stage][d half][token][dim]
  uint16_t v[2][2][kTileN][64];
  uint16_t ostage[2][kTileM][64];  // [d half][row][dim]: an output half on its way to a TMA store
};

struct DiffPrefillBars {
  uint64_t q_full[2], q_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t v_clear[2];    // a tile's rows past the request's end cleared
  uint64_t s_full[2][2];  // [map][buffer]
  uint64_t p_full[2][2];
  uint64_t pv_done[2][2];  // [map][buffer]: P V of a sub-tile has completed
  uint64_t o_ready[2];    // [map]: and of an item's last one
  uint64_t o_free[2];
  uint64_t drain;
};

__device__ __forceinline__ int item_subs(const Item& it) { return (it.kv1 - it.kv0 + kSubKeys - 1) / kSubKeys; }

// Whether the item's last KV tile reaches past the end of the request inside
// a page: the V rows there may hold anything (0 * NaN would not be 0).
__device__ __forceinline__ bool item_v_tail(const Item& it, int page_size) {
  return (it.rq.kv_len & (page_size - 1)) != 0 && it.kv0 + item_kv_tiles(it) * kTileN > it.rq.kv_len;
}

// Warp 0 (kV false): Q and K tiles; warp 2 (kV true): V tiles.
template <bool kV>
__device__ void diff_pf_produce(const RunParams& p, DiffPrefillBufs& pf, DiffPrefillBars& bar, volatile int* abort,
                                int32_t b0, int32_t b1, int32_t off_items) {
  const int lane = threadIdx.x & 31;
  const KvCache& kc = p.kv[0];
  const int G = p.group, lp = kc.log2_page, P = kc.page_size, ppt = kTileN >> lp;
  const CUtensorMap* map = kV ? &kc.tm_v : &kc.tm_k;
  uint64_t *full = kV ? bar.v_full : bar.k_full, *empty = kV ? bar.v_empty : bar.k_empty;
  if (lane == 0) {
    tc::prefetch_tensormap(map);
    if (!kV) tc::prefetch_tensormap(&p.tm_q);
  }
  uint32_t kt = 0, ni = 0;
  int armed[2] = {-1, -1}, q_armed[2] = {-1, -1};
  for (int32_t i = b0; i < b1; ++i) {
    const Item it = load_item(p.iws, off_items, i);
    const int ntiles = item_kv_tiles(it);
    if (ntiles == 0) continue;
    const int32_t* pages = kc.kv_indices + it.rq.page_start;
    const int npages = (it.rq.kv_len + P - 1) >> lp;
    auto page_of = [&](int j) -> int32_t {
      const int pg = ((it.kv0 + j * kTileN) >> lp) + lane;
      return lane < ppt && pg < npages ? __ldg(pages + pg) : kc.num_pages;  // out of bounds -> zeros
    };
    int32_t next = page_of(0);
    if (!kV) {
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
      ++ni;
    }
    for (int j = 0; j < ntiles; ++j, ++kt) {
      const int st = kt & 1;
      const uint32_t ph = (kt >> 1) & 1;
      const int32_t cur = next;
      if (j + 1 < ntiles) next = page_of(j + 1);
      if (!warp_wait(&empty[st], ph ^ 1, abort)) continue;
      if (lane == 0) mbar_arrive_expect_tx(&full[st], kKVBytes);
      __syncwarp();
      uint16_t(*buf)[kTileN][64] = kV ? pf.v[st] : pf.k[st];
      if (lane < ppt) {
        tc::tma_load_4d(&buf[0][lane * P][0], map, &full[st], 0, it.hk, 0, cur);
        tc::tma_load_4d(&buf[1][lane * P][0], map, &full[st], 64, it.hk, 0, cur);
      }
      armed[st] = ph;
      // The rows past the request's end are cleared once they have landed, and
      // the MMA warp waits for that instead.  This warp does it because it
      // alone starts the stage's next phase, so its wait cannot miss this one.
      if (kV && j + 1 == ntiles && item_v_tail(it, P) && warp_wait(&full[st], ph, abort)) {
        for (int row = it.rq.kv_len - (it.kv0 + j * kTileN) + (lane >> 4); row < kTileN; row += 2)
          *reinterpret_cast<uint4*>(&buf[(lane >> 3) & 1][row][8 * (lane & 7)]) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_clear[st]);
      }
    }
  }
  if (lane == 0) {  // every load this warp armed has landed before the CTA moves on
    for (int s = 0; s < 2; ++s) {
      if (armed[s] >= 0) mbar_wait_drain(&full[s], armed[s]);
      if (!kV && q_armed[s] >= 0) mbar_wait_drain(&bar.q_full[s], q_armed[s]);
    }
  }
  __syncwarp();
}

// A place in the CTA's stream of sub-tiles (items without keys have none).
struct SubCursor {
  int32_t i, end;
  Item it;
  int u, subs;          // sub-tile of the item, and how many it has
  uint32_t tile, item;  // K/V tile and non-empty item in the stream

  __device__ __forceinline__ bool live() const { return i < end; }
  __device__ __forceinline__ void settle(const int32_t* iws, int32_t off_items) {
    for (; i < end; ++i) {
      it = load_item(iws, off_items, i);
      subs = item_subs(it);
      if (subs > 0) break;
    }
    u = 0;
  }
  __device__ __forceinline__ void advance(const int32_t* iws, int32_t off_items) {
    if ((u & 1) || u + 1 == subs) ++tile;
    if (++u < subs) return;
    ++item;
    ++i;
    settle(iws, off_items);
  }
  __device__ __forceinline__ bool tile_begins() const { return (u & 1) == 0; }
  __device__ __forceinline__ bool tile_ends() const { return (u & 1) || u + 1 == subs; }
};

template <typename T>
__device__ void diff_pf_mma(const RunParams& p, DiffPrefillBufs& pf, DiffPrefillBars& bar, volatile int* abort,
                            uint32_t tmem, int32_t b0, int32_t b1, int32_t off_items) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t idesc_s = tc::idesc_f16(kBf16, false, kTileM, kSubKeys);
  constexpr uint32_t idesc_pv = tc::idesc_f16(kBf16, true, kTileM, kHeadDim);
  const int lane = threadIdx.x & 31, P = p.kv[0].page_size;
  // Start addresses count 16-byte units: a 64-dim half is 1024, a stage or Q
  // buffer 2048, 64 rows 512, 16 dims along a swizzled row 2, 16 V rows 128.
  const uint64_t dq = tc::smem_desc_sw128(smem_u32(&pf.q[0][0][0][0]), 16, 1024);
  const uint64_t dk = tc::smem_desc_sw128(smem_u32(&pf.k[0][0][0][0]), 16, 1024);
  const uint64_t dv = tc::smem_desc_sw128(smem_u32(&pf.v[0][0][0][0]), 64 * kTileN * 2, 1024);
  SubCursor s{b0, b1}, c{b0, b1};  // the next S, the next P V
  s.tile = s.item = c.tile = c.item = 0;
  s.settle(p.iws, off_items);
  c.settle(p.iws, off_items);
  uint32_t n = 0;        // sub-tiles through P V
  uint32_t cleared = 0;  // bit st: parity of the cleared tails of V stage st
  bool issued = false;
  // S of map m at cursor s into buffer buf; m = 0 waits for its operands, m = 1 releases them
  auto issue_s = [&](int m, int buf) {
    const int st = s.tile & 1, qb = s.item & 1;
    if (m == 0 && s.tile_begins()) {
      const bool q = s.u == 0;
      if (!warp_wait_all(2, &bar.k_full[st], (s.tile >> 1) & 1, q ? &bar.q_full[qb] : &bar.k_full[st],
                         q ? (s.item >> 1) & 1 : (s.tile >> 1) & 1, nullptr, 0, nullptr, 0, abort))
        return false;
      tc::fence_after_sync();
    }
    const uint64_t a = dq + 2048u * qb + 1024u * m, b = dk + 2048u * st + 1024u * m + 512u * (s.u & 1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      tc::mma_ss_warp(tmem + (2 * m + buf) * kSubKeys, a + 2u * kk, b + 2u * kk, idesc_s, kk > 0 ? 1u : 0u);
    tc::mma_commit_warp(&bar.s_full[m][buf]);
    issued = true;
    if (m == 1) {
      if (s.tile_ends()) tc::mma_commit_warp(&bar.k_empty[st]);
      if (s.u + 1 == s.subs) tc::mma_commit_warp(&bar.q_empty[qb]);
    }
    return true;
  };
  bool ok = true;
  for (int a = 0; a < 2 && ok && s.live(); ++a) {
    ok = issue_s(0, a) && issue_s(1, a);
    s.advance(p.iws, off_items);
  }
  for (; ok && c.live(); ++n) {
    const int buf = n & 1, st = c.tile & 1;
    const uint32_t pp = (n >> 1) & 1;
    const bool v_tail = c.tile_begins() && c.u + 2 >= c.subs && item_v_tail(c.it, P);
    for (int m = 0; m < 2 && ok; ++m) {
      uint64_t* const pb = &bar.p_full[m][buf];
      const bool v = m == 0 && c.tile_begins(), first = c.u == 0;
      uint64_t* const vb = v_tail ? &bar.v_clear[st] : &bar.v_full[st];
      const uint32_t vp = v_tail ? (cleared >> st) & 1 : (c.tile >> 1) & 1;
      ok = warp_wait_all(3, pb, pp, v ? vb : pb, v ? vp : pp, first ? &bar.o_free[m] : pb,
                         first ? (c.item & 1) ^ 1 : pp, nullptr, 0, abort);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t pcol = tmem + (2 * m + buf) * kSubKeys, o = tmem + kTmemO + m * kHeadDim;
      const uint64_t b = dv + 2048u * st + 512u * (c.u & 1);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)  // hi of keys 16 kk .. 16 kk + 15: columns 8 kk .. 8 kk + 7
        tc::mma_ts_warp(o, pcol + 8 * kk, b + 128u * kk, idesc_pv, (!first || kk > 0) ? 1u : 0u);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) tc::mma_ts_warp(o, pcol + 32 + 8 * kk, b + 128u * kk, idesc_pv, 1u);
      tc::mma_commit_warp(&bar.pv_done[m][buf]);
      if (c.u + 1 == c.subs) tc::mma_commit_warp(&bar.o_ready[m]);
      if (m == 1 && c.tile_ends()) tc::mma_commit_warp(&bar.v_empty[st]);
      if (s.live()) ok = issue_s(m, buf);  // over P of this sub-tile, in order behind its P V
    }
    if (!ok) break;
    if (s.live()) s.advance(p.iws, off_items);
    if (v_tail) cleared ^= 1u << st;
    c.advance(p.iws, off_items);
  }
  if (issued) {  // no product may still run when the CTA leaves the phase
    tc::mma_commit_warp(&bar.drain);
    if (lane == 0) mbar_wait_drain(&bar.drain, 0);
    __syncwarp();
  }
}

template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t packed) {
  return Elem<T>::to_float2(packed);
}

// The softmax warpgroup of map mt, and the end of the items.  At the end of an
// item warpgroup h takes dims 64 h .. 64 h + 63 of the difference for all 128
// rows (tensor-memory lanes are rows, and both warpgroups reach every column),
// so that only a row's normaliser and its sum of squares pass through shared
// memory (`stats`).
template <typename T, bool kMask>
__device__ void diff_pf_softmax(const DiffParams& dp, DiffPrefillBufs& pf, DiffPrefillBars& bar, float (*stats)[kTileM],
                                volatile int* abort, uint32_t tmem, int32_t b0, int32_t b1, int32_t off_items,
                                int causal, const Variant var) {
  const RunParams& p = dp.run;
  const int sw = (threadIdx.x >> 5) - kSoftmaxWarp0, mt = sw >> 2, lane = threadIdx.x & 31;
  const int r = 32 * (sw & 3) + lane;
  const uint32_t tl = tmem + (uint32_t(32 * (sw & 3)) << 16), o_cols = tl + kTmemO + mt * kHeadDim;
  const int G = p.group;
  const float sc = p.scale_log2;
  uint32_t n = 0, items = 0;  // sub-tiles and non-empty items so far
  for (int32_t i = b0; i < b1; ++i) {
    const Item item = load_item(p.iws, off_items, i);
    const Request& rq = item.rq;
    const int nrows = item.row1 - item.row0, subs = item_subs(item);
    const int row = item.row0 + r, tq = row / G, head = item.hk * G + (row - tq * G);
    const int pos = rq.kv_len - rq.qo_len + tq;
    // visible keys [lo, lim] and the sink (a padding row sees none)
    const int lim = r < nrows ? min(causal ? pos : rq.kv_len - 1, item.kv1 - 1) : -1;
    const int lo = kMask ? window_low(var, pos) : 0;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int u = 0; u < subs; ++u, ++n) {
      const int buf = n & 1;
      ok = ok && warp_wait(&bar.s_full[mt][buf], (n >> 1) & 1, abort);
      if (!ok) continue;
      tc::fence_after_sync();
      const uint32_t s_cols = tl + (2 * mt + buf) * kSubKeys;
      uint32_t sv[2][32];
      tc::tmem_ld32(s_cols, sv[0]);
      tc::tmem_ld32(s_cols + 32, sv[1]);
      tc::tmem_ld_wait();
      const int key0 = item.kv0 + u * kSubKeys;
      if (key0 + kSubKeys - 1 > lim || (kMask && key0 < lo)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int key = key0 + 32 * h + e;
            if (key > lim || (kMask && key < lo && key >= var.sink)) sv[h][e] = 0xff800000u;
          }
      }
      auto val = [&](int e) { return __uint_as_float(sv[e >> 5][e & 31]); };
      float mx[8];
#pragma unroll
      for (int a = 0; a < 8; ++a) mx[a] = max3(val(a), val(8 + a), val(16 + a));
#pragma unroll
      for (int e = 24; e < 56; e += 16)
#pragma unroll
        for (int a = 0; a < 8; ++a) mx[a] = max3(mx[a], val(e + a), val(e + 8 + a));
#pragma unroll
      for (int a = 0; a < 8; ++a) mx[a] = fmaxf(mx[a], val(56 + a));
      const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sc;
      const float m_new = top > m + kLazyRescale ? top : m;
      const bool rescale = m_new != m && u > 0;
      if (__any_sync(0xffffffffu, rescale)) {
        // O through the sub-tile before: its P V has to be complete.  (The
        // barrier is in that phase: the one before it on this buffer ended
        // before S of the sub-tile before was issued, and the next one needs
        // the P after this one.)
        ok = warp_wait(&bar.pv_done[mt][buf ^ 1], ((n - 1) >> 1) & 1, abort);
        if (!ok) continue;
        tc::fence_after_sync();
        const float alpha = rescale ? ex2(m - m_new) : 1.f;
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          uint32_t ov[32];
          tc::tmem_ld32(o_cols + 32 * h, ov);
          tc::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
          tc::tmem_st32(o_cols + 32 * h, ov);
        }
        tc::tmem_st_wait();
        l *= alpha;
      }
      m = m_new;
      const float ms = m == -INFINITY ? 0.f : m;
      const float2 cc = make_float2(sc, sc), nms = make_float2(-ms, -ms);
      float2 sum[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) sum[a] = make_float2(0.f, 0.f);
      uint32_t hi[32], low[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float2 x = fma2(make_float2(val(2 * e), val(2 * e + 1)), cc, nms);
        const float2 pe = make_float2(ex2(x.x), ex2(x.y));
        sum[e & 3] = add2(sum[e & 3], pe);
        hi[e] = tc::pack2<T>(pe.x, pe.y);
        const float2 hf = widen2<T>(hi[e]);
        const float2 d = add2(pe, make_float2(-hf.x, -hf.y));
        low[e] = tc::pack2<T>(d.x, d.y);
      }
      tc::tmem_st32(s_cols, hi);
      tc::tmem_st32(s_cols + 32, low);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[mt][buf]);
      const float2 t2 = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
      l += t2.x + t2.y;
    }

    // The end of the item.  The loads of O are not conditional (an item
    // without keys reads what the columns hold and drops it): as branches they
    // cost 900 bytes of spills.
    bool have_o = ok && subs > 0;
    have_o = have_o && warp_wait(&bar.o_ready[0], items & 1, abort);
    have_o = have_o && warp_wait(&bar.o_ready[1], items & 1, abort);
    tc::fence_after_sync();
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const float lse = l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
    const int64_t tok = int64_t(rq.qo_start) + tq;
    const bool write = r < nrows && !*abort;
    auto release_o = [&] {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0 && subs > 0) {
        mbar_arrive(&bar.o_free[0]);
        mbar_arrive(&bar.o_free[1]);
      }
    };
    if (item.part >= 0) {  // partial states: each warpgroup its own map
      const int64_t prw = int64_t(item.part) + mt * nrows + r;
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
        uint32_t ov[32];
        tc::tmem_ld32(o_cols + 32 * h, ov);
        tc::tmem_ld_wait();
        if (!write) continue;
        float4* dst = reinterpret_cast<float4*>(p.fws + p.partial_o_offset + prw * kHeadDim + 32 * h);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dst[e] = have_o ? make_float4(__uint_as_float(ov[4 * e]) * inv, __uint_as_float(ov[4 * e + 1]) * inv,
                                        __uint_as_float(ov[4 * e + 2]) * inv, __uint_as_float(ov[4 * e + 3]) * inv)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      release_o();
      if (write) p.fws[prw] = lse;
    } else {
      // `stats` of the item before has been read by now: its readers had to
      // release O before this item's last P V.  An item without keys has none.
      if (subs == 0) named_barrier_sync(kDiffBarrier, kSoftmaxThreads);
      stats[mt][r] = inv;
      if ((threadIdx.x & 127) == 0) tc::bulk_wait_read_all();  // the staging rows' last store has read them
      named_barrier_sync(kDiffBarrier, kSoftmaxThreads);
      const float i1 = stats[0][r], i2 = stats[1][r] * __ldg(dp.lambda + head);
      float y[64];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[32], b[32];
        tc::tmem_ld32(tl + kTmemO + 64 * mt + 32 * h, a);
        tc::tmem_ld32(tl + kTmemO + kHeadDim + 64 * mt + 32 * h, b);
        tc::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          y[32 * h + e] = have_o ? __uint_as_float(a[e]) * i1 - __uint_as_float(b[e]) * i2 : 0.f;
      }
      release_o();
      float f = dp.out_scale;
      if (dp.norm_w) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 64; ++e) ss += y[e] * y[e];
        stats[2 + mt][r] = ss;
        named_barrier_sync(kDiffBarrier, kSoftmaxThreads);
        f *= rsqrtf((stats[2][r] + stats[3][r]) * (1.f / kHeadDim) + dp.norm_eps);
#pragma unroll
        for (int e = 0; e < 64; ++e) y[e] *= __ldg(dp.norm_w + 64 * mt + e);
      }
      auto pack8 = [&](int e) {
        return make_uint4(tc::pack2<T>(y[e] * f, y[e + 1] * f), tc::pack2<T>(y[e + 2] * f, y[e + 3] * f),
                          tc::pack2<T>(y[e + 4] * f, y[e + 5] * f), tc::pack2<T>(y[e + 6] * f, y[e + 7] * f));
      };
      if (nrows == kTileM) {  // a whole tile: this half staged in the Q tile's layout, one TMA store
        uint16_t* stage = &pf.ostage[mt][0][0];
        uint4* my_row = reinterpret_cast<uint4*>(stage + r * 64);
#pragma unroll
        for (int c = 0; c < 8; ++c) my_row[c ^ (r & 7)] = pack8(8 * c);
        fence_proxy_async_smem();
        named_barrier_sync(kEpilogueBarrier0 + mt, 128);
        if ((threadIdx.x & 127) == 0 && !*abort) {
          tc::tma_store_3d(&p.tm_o, stage, 64 * mt, item.hk * G, rq.qo_start + item.row0 / G);
          tc::bulk_commit();
        }
      } else if (write) {
        uint4* dst = reinterpret_cast<uint4*>(p.o + tok * p.o_stride_tok + int64_t(head) * p.o_stride_head + 64 * mt);
#pragma unroll
        for (int c = 0; c < 8; ++c) dst[c] = pack8(8 * c);
      }
      if (p.lse && write) p.lse[(tok * p.num_qo_heads + head) * 2 + mt] = lse;
    }
    if (subs > 0) ++items;
  }
  if ((threadIdx.x & 127) == 0) tc::bulk_wait_all();  // output tiles written before the CTA moves on
  fence_proxy_async_smem();                           // the decode ring's copies land in this phase's buffers
}

}  // namespace fi
