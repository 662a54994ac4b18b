// kv4_kernel.cuh -- attention over the paged cache held in 4 bits: 16-row tiles.
//
// A value is s (n - z) (fi_kv4.h).  A code n in the low nibble of a 16-bit half
// is, as it lies there, the fp16 subnormal n 2^-24, and in the next nibble n
// 2^-20; the tensor cores take subnormals exactly.  So a word of eight codes
// becomes four operand registers with four ANDs and one shift, no conversion,
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
//
// Eight warps walk a chunk's keys in eight consecutive parts, each with a ring
// of its own: 32 keys a stage, brought by one bulk copy a block (keys, values
// and their words lie together), issued by the warp that consumed the stage
// before, kKv4Depth stages ahead and across items.  No producer warp, no barrier
// but the one that joins the eight states of an item.
#pragma once
#include "attention_kernel.cuh"
#include "kv4_layout.h"
#include "kv4_params.h"

namespace fi {

constexpr int kKv4Warps = 8;
constexpr int kKv4Threads = 32 * kKv4Warps;
constexpr int kKv4Stage = 32;          // keys of a stage
constexpr int kKv4Depth = 4;           // stages a warp has in flight
constexpr int kKv4StageBytes = 4608;   // 32 blocks of one slot, 144 bytes each
constexpr int kKv4Tile = 16;           // packed query rows of a pass
constexpr int kKv4CombRow = 132;       // floats from row to row of a warp's state (128 and 4 against bank conflicts)

struct alignas(128) Kv4Smem {
  uint8_t ring[kKv4Warps][kKv4Depth][kKv4StageBytes];
  float comb_o[kKv4Warps][kKv4Tile][kKv4CombRow];
  float comb_m[kKv4Warps][kKv4Tile];
  float comb_l[kKv4Warps][kKv4Tile];
  uint32_t seen[kKv4Warps][kKv4Depth];  // keys of a stage that are there, a bit each
  uint64_t full[kKv4Warps][kKv4Depth];
  volatile int abort;
  int merge_last;
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
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
constexpr uint32_t kNibble0 = 0x000F000Fu, kNibble1 = 0x00F000F0u;

// A word's two halves: the scale, and the zero point as n 2^-24 (the unit of the products).
__device__ __forceinline__ float word_scale(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w & 0xFFF0u))); }
__device__ __forceinline__ float word_zero(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w & 15u))); }

// ------------------------------------------------------------------- loads

// A warp's walk over the stages of its CTA's items, ahead of their use.
struct Kv4Loader {
  const Kv4Params& kp;
  Kv4Smem& sm;
  const int32_t off_items, end;
  const int warp, lane;
  int32_t i;                    // item being loaded
  int32_t pass, passes;         // of 16 rows
  int32_t st, st_begin, st_end; // this warp's stages of it
  int32_t kv0, kv1, npages, window;
  const int32_t* pages;
  const uint8_t* head;
  int32_t ids, ids_next;        // page ids 32 window + lane, and of the next window
  uint32_t issued;

  __device__ Kv4Loader(const Kv4Params& kp, Kv4Smem& sm, int32_t off_items, int32_t begin, int32_t end)
      : kp(kp), sm(sm), off_items(off_items), end(end), warp((threadIdx.x >> 5) % kKv4Warps), lane(threadIdx.x & 31),
        i(begin - 1), pass(0), passes(0), st(0), st_begin(0), st_end(0), window(-2), issued(0) {}

  __device__ __forceinline__ int32_t load_ids(int32_t w) const {
    const int32_t p = 32 * w + lane;
    return p < npages ? __ldg(pages + p) : -1;
  }
  // The next stage of this warp; false after the last.
  __device__ __forceinline__ bool more() {
    while (st == st_end) {
      if (++pass < passes) {
        st = st_begin;
        window = -2;
        continue;
      }
      if (++i >= end) {
        i = end;
        passes = 0;
        return false;
      }
      const Item it = load_item(kp.run.iws, off_items, i);
      const int nst = (it.kv1 - it.kv0 + kKv4Stage - 1) / kKv4Stage;
      st = st_begin = nst * warp / kKv4Warps;
      st_end = nst * (warp + 1) / kKv4Warps;
      pass = 0;
      passes = (it.row1 - it.row0 + kKv4Tile - 1) / kKv4Tile;
      kv0 = it.kv0;
      kv1 = it.kv1;
      const KvCache& kc = kp.run.kv[0];
      npages = (it.rq.kv_len + kc.page_size - 1) >> kc.log2_page;
      pages = kc.kv_indices + it.rq.page_start;
      head = kp.cache + it.hk * kp.head_stride;
      window = -2;
    }
    return true;
  }
  __device__ __forceinline__ void issue() {
    if (!more()) return;
    const KvCache& kc = kp.run.kv[0];
    const int32_t j0 = kv0 + kKv4Stage * st;
    const int32_t pg0 = j0 >> kc.log2_page;  // a stage's pages lie in one window of 32
    if (pg0 >> 5 != window) {
      ids = pg0 >> 5 == window + 1 ? ids_next : load_ids(pg0 >> 5);
      window = pg0 >> 5;
      ids_next = load_ids(window + 1);
    }
    const int32_t first = lane << kp.log2_block;  // of this lane's block in the stage
    const int32_t id = __shfl_sync(0xffffffffu, ids, (pg0 + lane) & 31);
    const bool mine = first < kKv4Stage && j0 + first < kv1 && id >= 0 && id < kc.num_pages;
    const uint32_t blocks = __ballot_sync(0xffffffffu, mine);
    const uint32_t keys = __ballot_sync(0xffffffffu, (blocks >> (lane >> kp.log2_block) & 1u) && j0 + lane < kv1);
    const int slot = issued % kKv4Depth;
    if (lane == 0) {
      sm.seen[warp][slot] = keys;
      mbar_arrive_expect_tx(&sm.full[warp][slot], __popc(blocks) * kp.block_bytes);
    }
    __syncwarp();
    if (mine)
      bulk_load(&sm.ring[warp][slot][lane * kp.block_bytes],
                head + id * kp.page_stride + ((j0 & (kc.page_size - 1)) >> kp.log2_block) * kp.block_bytes,
                kp.block_bytes, &sm.full[warp][slot]);
    ++st;
    ++issued;
  }
};

// ----------------------------------------------------------------- a stage

// Where this lane (g = lane / 4, t = lane % 4) reads a block of 16 keys.  Row r
// of the products is key r ^ (r >> 1 & 1): the rows that lanes t = 0 .. 3 of a
// half warp read of v then alternate between the two halves of the 128-byte
// lines (two ways instead of four).
struct Kv4Places {
  uint32_t k[2];        // rows of keys g and g + 8: 16 bytes, dims 32 t ..
  uint32_t kw[2];       // their words (those of v: v_words further)
  uint32_t v[4], vw[4]; // rows (8 bytes, dims 16 g ..) and words of keys 2t, 2t + 1, 2t + 8, 2t + 9
  uint32_t v_words;
  uint32_t next_rows, next_words;  // from the first 16 keys of a stage to the others

  __device__ explicit Kv4Places(const Kv4Params& kp) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, B = kp.block_slots;
    auto key = [](int r) { return r ^ ((r >> 1) & 1); };
    auto at = [&](int k, int row) { return (k >> kp.log2_block) * kp.block_bytes + (k & (B - 1)) * row; };
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      k[u] = at(key(g) + 8 * u, kKv4RowBytes) + 16 * t;
      kw[u] = at(key(g) + 8 * u, 2) + kv4_k_word(B, 0);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = key(2 * t + (u & 1)) + 8 * (u >> 1);
      v[u] = at(c, kKv4RowBytes) + kv4_v_row(B, 0) + 8 * g;
      vw[u] = at(c, 2) + kv4_v_word(B, 0);
    }
    v_words = 2 * B;
    next_rows = B == 32 ? 16 * kKv4RowBytes : (16 >> kp.log2_block) * kp.block_bytes;
    next_words = B == 32 ? 32 : next_rows;
  }
};

// Query rows 8 n + g as operand columns, and the states of rows 8 n + 2t, + 1.
template <int NT>
struct Kv4Rows16 {
  uint32_t q[NT][8][2];  // of the 16 dims of step k
  float c[NT][2];        // log2-domain factor of a row's products
  float qs[NT][2];       // sum of the row's operand values
  int lim[NT][2], lo[NT][2];
  float m[NT][2], l[NT][2];
  float o[NT][8][4];     // step i: dims 16 g + 8 (i / 4) + i % 4 (.., ..) and + 4
  float z[NT][4];
  float unit;            // the power of two that v's scales are multiplied by
};

template <typename T, int NT>
__device__ __forceinline__ void kv4_load_rows(const Kv4Params& kp, const Item& it, int pass, int causal,
                                              const Variant& var, Kv4Rows16<NT>& R) {
  const RunParams& p = kp.run;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, G = p.group;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = it.row0 + kKv4Tile * pass + 8 * n + g;
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = make_uint4(0u, 0u, 0u, 0u);
    if (row < it.row1) {
      const int tok = row / G;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t(it.rq.qo_start) + tok) * p.q_stride_tok +
                                                        int64_t(it.hk * G + row - tok * G) * p.q_stride_head + 32 * t);
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = __ldg(src + j);
    }
    float f[4][8], top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = Elem<T>::to_float2(w[e]);
        f[j][2 * e] = x.x;
        f[j][2 * e + 1] = x.y;
        top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the row times a power of two, its largest value in [2^14, 2^15): fp16 has
    // room for the dims in the upper nibbles, which enter with 2^-4
    int ex = int(__float_as_uint(top) >> 23) - 127;  // -127 for zero rows
    ex = min(max(ex, -100), 100);
    const float up = __int_as_float((127 + 14 - ex) << 23);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      auto put = [&](uint32_t& dst, float a, float b, float unit) {
        const __half2 h = __floats2half2_rn(a * (up * unit), b * (up * unit));
        dst = *reinterpret_cast<const uint32_t*>(&h);
        const float2 x = __half22float2(h);
        sum += (x.x + x.y) / unit;
      };
      put(R.q[n][2 * j][0], f[j][0], f[j][4], 1.f);
      put(R.q[n][2 * j][1], f[j][2], f[j][6], 1.f);
      put(R.q[n][2 * j + 1][0], f[j][1], f[j][5], 0.0625f);
      put(R.q[n][2 * j + 1][1], f[j][3], f[j][7], 0.0625f);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    const float c = p.scale_log2 * __int_as_float((127 + 10 + ex) << 23);  // 2^(ex - 14), and the products' 2^-24
#pragma unroll
    for (int u2 = 0; u2 < 2; ++u2) {
      R.qs[n][u2] = __shfl_sync(0xffffffffu, sum, 8 * t + 4 * u2);
      R.c[n][u2] = __shfl_sync(0xffffffffu, c, 8 * t + 4 * u2);
      const int r = it.row0 + kKv4Tile * pass + 8 * n + 2 * t + u2;
      const int pos = it.rq.kv_len - it.rq.qo_len + r / G;
      R.lim[n][u2] = r < it.row1 ? (causal ? pos : it.rq.kv_len - 1) : -1;
      R.lo[n][u2] = window_low(var, pos);
      R.m[n][u2] = -INFINITY;
      R.l[n][u2] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) R.o[n][i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) R.z[n][e] = 0.f;
  }
  R.unit = __int_as_float((127 + 100) << 23);
}

// The 32 keys of a stage from key j0 on.  inside: every key of the stage is
// there and visible to every row.
template <int NT>
__device__ __forceinline__ void kv4_stage(const uint8_t* stage, const Kv4Places& at, uint32_t seen, int j0, bool inside,
                                          const Variant& var, Kv4Rows16<NT>& R) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  float s[2][NT][4];
  float vs[2][2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint8_t* rows = stage + b * at.next_rows;
    const uint8_t* words = stage + b * at.next_words;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[b][n][e] = 0.f;
    const uint4 ka = *reinterpret_cast<const uint4*>(rows + at.k[0]);
    const uint4 kb = *reinterpret_cast<const uint4*>(rows + at.k[1]);
    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t ha = wa[j] >> 8, hb = wb[j] >> 8;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16(s[b][n], wa[j] & kNibble0, wb[j] & kNibble0, ha & kNibble0, hb & kNibble0, R.q[n][2 * j][0],
              R.q[n][2 * j][1]);
        mma16(s[b][n], wa[j] & kNibble1, wb[j] & kNibble1, ha & kNibble1, hb & kNibble1, R.q[n][2 * j + 1][0],
              R.q[n][2 * j + 1][1]);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t w = *reinterpret_cast<const uint16_t*>(words + at.kw[u]);
      const uint32_t x = *reinterpret_cast<const uint16_t*>(words + at.kw[u] + at.v_words);
      const float ks = word_scale(w), kz = word_zero(w);
      vs[b][u] = word_scale(x);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) s[b][n][2 * u + h] = fmaf(-kz, R.qs[n][h], s[b][n][2 * u + h]) * ks;
    }
  }
  if (!inside) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = 16 * b + 8 * u + (g ^ ((g >> 1) & 1)), key = j0 + k;
        const bool there = seen >> k & 1u;
        bool any = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool sees = there && key <= R.lim[n][h] && (key >= R.lo[n][h] || key < var.sink);
            if (!sees) s[b][n][2 * u + h] = -INFINITY;
            any |= sees;
          }
        if (!any) vs[b][u] = 0.f;  // a weight of 0 times any bytes, infinities included
      }
  }
  // The running maxima move when a row's grows by more than 2^8, the unit of
  // the weights when a value scale would pass twice it.
  float top[NT][2];
  bool move = fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1])) * R.unit >= 2.f;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[n][h] = fmaxf(fmaxf(s[0][n][h], s[0][n][2 + h]), fmaxf(s[1][n][h], s[1][n][2 + h])) * R.c[n][h];
      move |= top[n][h] > R.m[n][h] + kLazyRescale;
    }
  if (__any_sync(0xffffffffu, move)) {
    float v = fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1]));
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
    float back = 1.f;
    if (v * R.unit >= 2.f) {
      const float unit = __int_as_float((254 << 23) - int(__float_as_uint(v) & 0x7F800000u));  // 1 / the power of two below v
      back = unit / R.unit;
      R.unit = unit;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = top[n][h];
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
        f[h] = 1.f;
        if (x > R.m[n][h] + kLazyRescale) {
          f[h] = ex2(R.m[n][h] - x);
          R.m[n][h] = x;
        }
        R.l[n][h] *= f[h];
        f[h] *= back;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) R.o[n][i][e] *= f[e & 1];
#pragma unroll
      for (int e = 0; e < 4; ++e) R.z[n][e] *= f[e & 1];
    }
  }
  // weights p s_v as operand columns: keys 2t, 2t + 1 and 2t + 8, 2t + 9 of row g
  uint32_t w[2][NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float m0 = R.m[n][0] == -INFINITY ? 0.f : R.m[n][0], m1 = R.m[n][1] == -INFINITY ? 0.f : R.m[n][1];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float p0 = ex2(fmaf(s[b][n][2 * u], R.c[n][0], -m0)), p1 = ex2(fmaf(s[b][n][2 * u + 1], R.c[n][1], -m1));
        R.l[n][0] += p0;
        R.l[n][1] += p1;
        const float x = vs[b][u] * R.unit;
        w[b][n][u] = transpose8(tc::pack2<__half>(p0 * x, p1 * x));
      }
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint8_t* rows = stage + b * at.next_rows;
    const uint8_t* words = stage + b * at.next_words;
    uint32_t z[4];
    uint2 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      z[u] = *reinterpret_cast<const uint16_t*>(words + at.vw[u]);
      v[u] = *reinterpret_cast<const uint2*>(rows + at.v[u]);
    }
    const uint32_t z0 = (z[0] | z[1] << 16) & kNibble0, z1 = (z[2] | z[3] << 16) & kNibble0;
#pragma unroll
    for (int n = 0; n < NT; ++n) mma16(R.z[n], z0, z0, z1, z1, w[b][n][0], w[b][n][1]);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      auto word = [&](int u) { return half ? v[u].y : v[u].x; };
      const uint32_t a0 = __byte_perm(word(0), word(1), 0x5410), a1 = __byte_perm(word(0), word(1), 0x7632);
      const uint32_t a2 = __byte_perm(word(2), word(3), 0x5410), a3 = __byte_perm(word(2), word(3), 0x7632);
      const uint32_t h0 = a0 >> 8, h1 = a1 >> 8, h2 = a2 >> 8, h3 = a3 >> 8;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t b0 = w[b][n][0], b1 = w[b][n][1];
        mma16(R.o[n][4 * half], a0 & kNibble0, a1 & kNibble0, a2 & kNibble0, a3 & kNibble0, b0, b1);
        mma16(R.o[n][4 * half + 1], a0 & kNibble1, a1 & kNibble1, a2 & kNibble1, a3 & kNibble1, b0, b1);
        mma16(R.o[n][4 * half + 2], h0 & kNibble0, h1 & kNibble0, h2 & kNibble0, h3 & kNibble0, b0, b1);
        mma16(R.o[n][4 * half + 3], h0 & kNibble1, h1 & kNibble1, h2 & kNibble1, h3 & kNibble1, b0, b1);
      }
    }
  }
}

// This warp's state of the pass into shared memory: o (not yet divided), max, sum.
template <int NT>
__device__ __forceinline__ void kv4_put_state(Kv4Smem& sm, int warp, Kv4Rows16<NT>& R, bool any) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = R.l[n][h];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
      const int row = 8 * n + 2 * t + h;
      if (g == 0) {
        sm.comb_m[warp][row] = any ? R.m[n][h] : -INFINITY;
        sm.comb_l[warp][row] = l;
      }
      if (!any) continue;
      const float up = 16777216.f / R.unit;  // 2^24: codes and zero points came in as n 2^-24
      float* dst = &sm.comb_o[warp][row][16 * g];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = ((i & 1 ? 0.0625f : 1.f) * R.o[n][4 * half + i][2 * hi + h] - R.z[n][h]) * up;
          *reinterpret_cast<float4*>(dst + 8 * half + 4 * hi) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
}

template <typename T, int NT>
__device__ __forceinline__ void kv4_pass(const Kv4Params& kp, Kv4Smem& sm, Kv4Loader& load, const Kv4Places& at,
                                         const Item& it, int pass, int causal, const Variant& var, uint32_t& used) {
  const int warp = load.warp;
  Kv4Rows16<NT> R;
  kv4_load_rows<T, NT>(kp, it, pass, causal, var, R);
  // keys that every row of the pass sees
  const int r0 = it.row0 + kKv4Tile * pass, r1 = min(it.row1, r0 + kKv4Tile) - 1, G = kp.run.group;
  const int first = it.rq.kv_len - it.rq.qo_len + r0 / G, last = it.rq.kv_len - it.rq.qo_len + r1 / G;
  const int lim = causal ? first : it.rq.kv_len - 1, lo = window_low(var, last);
  const int nst = (it.kv1 - it.kv0 + kKv4Stage - 1) / kKv4Stage;
  const int s0 = nst * warp / kKv4Warps, s1 = nst * (warp + 1) / kKv4Warps;
  bool ok = !sm.abort;
  ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
  for (int st = s0; st < s1 && ok; ++st) {
    const int slot = used % kKv4Depth;
    ok = warp_wait(&sm.full[warp][slot], (used / kKv4Depth) & 1, &sm.abort);
    if (!ok) break;
    ++used;
    const int j0 = it.kv0 + kKv4Stage * st;
    const uint32_t seen = sm.seen[warp][slot];
    const bool inside = seen == 0xffffffffu && j0 + kKv4Stage - 1 <= lim && j0 >= lo;
    kv4_stage<NT>(sm.ring[warp][slot], at, seen, j0, inside, var, R);
    __syncwarp();
    load.issue();
  }
  kv4_put_state<NT>(sm, warp, R, s1 > s0);
}

// The items [begin, end) of a CTA; tid counts the kKv4Threads threads that run it.
template <typename T>
__device__ void kv4_consume(const Kv4Params& kp, Kv4Smem& sm, int tid, int32_t begin, int32_t end, int32_t off_items,
                            int32_t off_merge, int32_t off_cnt, int causal, const Variant& var) {
  const RunParams& p = kp.run;
  const int G = p.group;
  const Kv4Places at(kp);
  Kv4Loader load(kp, sm, off_items, begin, end);
  for (int d = 0; d < kKv4Depth; ++d) load.issue();
  uint32_t used = 0;
  for (int32_t i = begin; i < end; ++i) {
    const Item it = load_item(p.iws, off_items, i);
    const int nrows = it.row1 - it.row0;
    for (int pass = 0; kKv4Tile * pass < nrows; ++pass) {
      const int rows = min(kKv4Tile, nrows - kKv4Tile * pass);
      if (rows <= 8)
        kv4_pass<T, 1>(kp, sm, load, at, it, pass, causal, var, used);
      else
        kv4_pass<T, 2>(kp, sm, load, at, it, pass, causal, var, used);
      named_barrier_sync(1, kKv4Threads);
      if (!sm.abort) {
        for (int task = tid; task < rows * 32; task += kKv4Threads) {
          const int r = task >> 5, ch = task & 31;
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kKv4Warps; ++w) M = fmaxf(M, sm.comb_m[w][r]);
          float L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          if (M != -INFINITY) {
#pragma unroll
            for (int w = 0; w < kKv4Warps; ++w) {
              if (sm.comb_m[w][r] == -INFINITY) continue;  // no key, or no state at all
              const float f = ex2(sm.comb_m[w][r] - M);
              const float4 v = *reinterpret_cast<const float4*>(&sm.comb_o[w][r][4 * ch]);
              L += f * sm.comb_l[w][r];
              acc.x += f * v.x;
              acc.y += f * v.y;
              acc.z += f * v.z;
              acc.w += f * v.w;
            }
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
            *reinterpret_cast<uint2*>(p.o + tok * p.o_stride_tok + int64_t(head) * p.o_stride_head + 4 * ch) = packed;
            if (ch == 0 && p.lse) p.lse[tok * p.num_qo_heads + head] = lse;
          } else {
            const int64_t part = int64_t(it.part) + prow;
            *reinterpret_cast<float4*>(p.fws + p.partial_o_offset + part * kHeadDim + 4 * ch) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (ch == 0) p.fws[part] = lse;
          }
        }
      }
      named_barrier_sync(1, kKv4Threads);
    }
    if (it.merge >= 0)
      merge_split_unit<T>(p, it, it.rq, off_merge, off_cnt, tid, kKv4Threads, 2, &sm.merge_last, sm.abort);
  }
  // given up: the copies in flight have landed before the CTA leaves
  if (load.lane == 0)
    for (; used < load.issued; ++used) mbar_wait_drain(&sm.full[load.warp][used % kKv4Depth], (used / kKv4Depth) & 1);
  __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kKv4Threads, 1) kv4_attention_kernel(const __grid_constant__ Kv4Params kp) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Kv4Smem& sm = *reinterpret_cast<Kv4Smem*>(smem_raw);
  if (threadIdx.x == 0) let_dependents_start();
  const RunParams& p = kp.run;
  const int32_t* iws = p.iws;
  // The plan in the workspace has to be one over the 4-bit cache and fit this
  // launch: nothing is written otherwise.
  const int32_t n_items = ws_header(iws, FI_H_NUM_ITEMS), off_cta = ws_header(iws, FI_H_OFF_CTA);
  const int32_t h_rows = ws_header(iws, FI_H_PARTIAL_ROWS), h_qo = ws_header(iws, FI_H_TOTAL_QO);
  bool bad = ws_header(iws, FI_H_MAGIC) != FI_PLAN_MAGIC_KV4 || ws_header(iws, FI_H_NUM_CTAS) != int32_t(gridDim.x) ||
             h_rows < 0 || h_rows > p.max_partial_rows || h_qo < 0 || h_qo > p.q_num_tokens ||
             ws_header(iws, FI_H_NUM_QO_HEADS) != p.num_qo_heads ||
             ws_header(iws, FI_H_NUM_KV_HEADS) != p.num_kv_heads ||
             ws_header(iws, FI_H_PAGE_SIZE) != p.kv[0].page_size || (smem_u32(smem_raw) & 127u) != 0;
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
  const int32_t off_items = ws_header(iws, FI_H_OFF_ITEMS), off_merge = ws_header(iws, FI_H_OFF_MERGE);
  const int32_t off_cnt = ws_header(iws, FI_H_OFF_COUNTERS);
  const int causal = ws_header(iws, FI_H_CAUSAL);
  Variant var;
  var.window_left = ws_header(iws, FI_H_WINDOW_LEFT);
  var.sink = ws_header(iws, FI_H_SINK_TOKENS);
  var.cap_a = var.cap_b = 0.f;
  var.rope_table = nullptr;
  if (threadIdx.x == 0) {
    for (int w = 0; w < kKv4Warps; ++w)
      for (int s = 0; s < kKv4Depth; ++s) mbar_init(&sm.full[w][s], 1);
    sm.abort = 0;
    sm.merge_last = 0;
    fence_mbar_init();
  }
  __syncthreads();
  kv4_consume<T>(kp, sm, threadIdx.x, begin, end, off_items, off_merge, off_cnt, causal, var);
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort) atomicOr(p.iws + FI_H_STATUS, sm.abort);
}

}  // namespace fi
