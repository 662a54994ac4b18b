// kv4_append.cu -- the append to the 4-bit cache (norms, rotation and
// quantisation of a step's keys and values in one launch) and rows of that
// cache read back in 16 bits.
//
// The codes are defined to the bit (fi_kv4.h): a code next to a border goes by
// the last bit of an fp32 value, and a cache has to hold the same bytes
// whichever batch brought the token, so sums have one order and nothing is
// contracted to a fused multiply-add.  The lane layout follows from that order:
// eight lanes hold a head, lane p the chunks p and p + 8 of 8 dims each, so
// that the first sum (d and d + 64), like a pair of the half layout over the
// whole head, stays within a lane.
//
// Bound by the bytes of q (read and written), k and v (read, a quarter
// written).  A warp takes four heads at a time, q heads first, then k, then v,
// each kind's heads filled up to a multiple of four so that a warp does one
// thing; one warp per token, or per part of one when there are few tokens.  The
// next group's rows are in flight while one is turned and coded.  cos and sin
// stay in shared memory, read without bank conflicts, and no second group is held:
// 8192 tokens of 32 + 8 heads with norms and half pairs: 38.6 us (26.4 us of bytes at
// the copy rate), without norms 35.1, neighbouring pairs 40.1.  Half pairs over 64
// dims of a head 62: the other member of a pair is in another lane, 32 shuffles a
// group.  (With the rows read back by a launch behind it, 49 us, one or two groups
// ahead with 16 to 20 warps on an SM took 60 to 64, conflicts 6 more, clamps behind the
// rounding 1 and sums and products one at a time, or a lane's two angles one behind
// the other, 1 each.)
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "kv4_layout.h"
#include "rotary.h"

namespace fi {
namespace {

constexpr int kAppendWarps = 4;   // warps of a block
constexpr int kAppendBlocks = 6;  // blocks of an SM
constexpr float kFifteenth = 1.f / 15.f;

enum { kNoPairs = 0, kHalfPairs = 1, kNextPairs = 2, kPartHalfPairs = 3 };

struct Kv4Rows {
  const uint16_t* in;
  int64_t in_tok, in_head;
  int32_t heads;
};

struct Kv4AppendParams {
  Kv4Rows q, k, v;
  uint16_t* q_out;
  int64_t q_out_tok, q_out_head;
  const float *q_weight, *k_weight;
  int64_t q_weight_stride, k_weight_stride;
  const int32_t* positions;
  const int32_t* slots;
  uint8_t* cache;
  int64_t page_stride, head_stride, num_slots;
  int32_t num_tokens, parts;  // warps per token
  int32_t log2_page, block_slots, block_bytes;
  int32_t rot_chunks;  // chunks of 8 dims in the rotated part
  float amplitude, eps;
  uint64_t turns[FI_ROTARY_MAX_PAIRS / 2];
};

// rint(t) of |t| <= 15 by the spacing of the fp32 numbers above 2^23.
__device__ __forceinline__ int round_small(float t) {
  return __float_as_int(__fadd_rn(t, 12582912.f)) - 0x4B400000;
}

// Eight codes rint(x inv) + z, kept within 0 .. 15 before the rounding (the bounds
// are whole numbers; a NaN becomes 0), and summed modulo 2^32 with the rounded
// numbers' bits as they are.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float inv, int z) {
  const float lo = float(-z), hi = float(15 - z);
  uint32_t w = (uint32_t(z) - 0x4B400000u) * 0x11111111u;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 t = mul2(make_float2(x[e], x[e + 1]), make_float2(inv, inv));
    const float2 n = add2(make_float2(fminf(fmaxf(t.x, lo), hi), fminf(fmaxf(t.y, lo), hi)),
                          make_float2(12582912.f, 12582912.f));
    w += __float_as_uint(n.x) << (4 * e);
    w += __float_as_uint(n.y) << (4 * e + 4);
  }
  return w;
}

template <typename T, int kPairs>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendBlocks) kv4_append_kernel(const __grid_constant__ Kv4AppendParams a) {
  __shared__ alignas(16) float2 s_cs[kAppendWarps][FI_KV4_HEAD_DIM / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * kAppendWarps + warp;
  const int t = int(w / a.parts), part = int(w - int64_t(t) * a.parts);
  if (t >= a.num_tokens) return;
  const int64_t slot = __ldg(a.slots + t);
  const bool store_kv = slot >= 0 && slot < a.num_slots;
  const int p = lane & 7, sub = lane >> 3;  // this lane's chunks p and p + 8, of head `sub` of the four
  const int nq = (a.q.heads + 3) >> 2, nk = (a.k.heads + 3) >> 2;
  const int groups = store_kv ? nq + 2 * nk : nq;
  // group g of four heads: its operand, and this lane's head in it (-1: none)
  auto operand = [&](int g) -> const Kv4Rows& { return g < nq ? a.q : g < nq + nk ? a.k : a.v; };
  auto head_of = [&](int g) {
    const int h = 4 * (g < nq ? g : g < nq + nk ? g - nq : g - nq - nk) + sub;
    return h < operand(g).heads ? h : -1;
  };
  uint4 lo, hi;
  auto load = [&](int g) {
    lo = hi = make_uint4(0u, 0u, 0u, 0u);
    if (g >= groups) return;
    const int h = head_of(g);
    if (h < 0) return;
    const Kv4Rows& rows = operand(g);
    const uint16_t* src = rows.in + t * rows.in_tok + h * rows.in_head + 8 * p;
    lo = *reinterpret_cast<const uint4*>(src);
    hi = *reinterpret_cast<const uint4*>(src + 64);
  };
  load(part);

  // cos and sin of the token's pairs, the two pairs of a float4 next to those of the other lanes: read without bank
  // conflicts; of the half layout both cosines, then both sines
  constexpr int kMine = kPairs == kHalfPairs ? 8 : 4, kPlaces = kPairs == kHalfPairs ? 8 : 16;  // pairs of a chunk, chunks
  auto spot = [](int i) { return kPairs == kPartHalfPairs ? i : 2 * ((i % kMine >> 1) * kPlaces + i / kMine) + (i & 1); };
  float2* const cs = s_cs[warp];
  const float4* const cs2 = reinterpret_cast<const float4*>(s_cs[warp]);
  if (kPairs != kNoPairs) {
    const int32_t pos = __ldg(a.positions + t);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int i = lane + 32 * n;
      if (i >= a.rot_chunks * 4) break;
      const uint64_t turn = uint64_t(int64_t(pos)) * a.turns[i];  // modulo one turn
      // 2^-31: half turns in [-1, 1]; then the angle
      const float x = __fmul_rn(float(int32_t(turn >> 32)) * 4.6566128730773926e-10f, 3.14159265358979f);
      float c, sn;
      sincosf(x, &sn, &c);  // the same as sinf and cosf: once compared for every fp32 number up to pi
      c = __fmul_rn(c, a.amplitude);
      sn = __fmul_rn(sn, a.amplitude);
      if (kPairs == kHalfPairs) {
        float* const at = &s_cs[warp][spot(i & ~1)].x + (i & 1);
        at[0] = c;
        at[2] = sn;
      } else {
        cs[spot(i)] = make_float2(c, sn);
      }
    }
    __syncwarp();
  }
  auto turn_pair = [](float& x, float& y, const float2& c) {
    const float x0 = x;
    x = __fsub_rn(__fmul_rn(x0, c.x), __fmul_rn(y, c.y));
    y = __fadd_rn(__fmul_rn(y, c.x), __fmul_rn(x0, c.y));
  };

  const int64_t page = slot >> a.log2_page;
  const int in_page = int(slot) & ((1 << a.log2_page) - 1);
  const int block = in_page / a.block_slots, place = in_page - block * a.block_slots;
  uint8_t* const base = a.cache + page * a.page_stride + block * a.block_bytes;
  for (int g = part; g < groups; g += a.parts) {
    const int h = head_of(g);
    float x[8], y[8];
    unpack<T>(lo, x);
    unpack<T>(hi, y);
    load(g + a.parts);  // in flight while this group is turned
    const bool is_q = g < nq, is_v = g >= nq + nk;
    const float* weight = is_v ? nullptr : is_q ? a.q_weight : a.k_weight;
    if (weight) {
      float2 sq[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 u = make_float2(x[2 * e], x[2 * e + 1]), v = make_float2(y[2 * e], y[2 * e + 1]);
        sq[e] = add2(mul2(u, u), mul2(v, v));
      }
      const float2 four = add2(add2(sq[0], sq[2]), add2(sq[1], sq[3]));
      float sum = __fadd_rn(four.x, four.y);
#pragma unroll
      for (int m = 4; m > 0; m >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, m));
      const float f = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.f / 128.f), a.eps)));
      const float* mine = weight + max(h, 0) * (is_q ? a.q_weight_stride : a.k_weight_stride) + 8 * p;
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(mine)), w1 = __ldg(reinterpret_cast<const float4*>(mine + 4));
      const float4 w2 = __ldg(reinterpret_cast<const float4*>(mine + 64)), w3 = __ldg(reinterpret_cast<const float4*>(mine + 68));
      const float wx[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      const float wy[8] = {w2.x, w2.y, w2.z, w2.w, w3.x, w3.y, w3.z, w3.w};
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 ff = make_float2(f, f);
        const float2 u = mul2(mul2(make_float2(x[e], x[e + 1]), ff), make_float2(wx[e], wx[e + 1]));
        const float2 v = mul2(mul2(make_float2(y[e], y[e + 1]), ff), make_float2(wy[e], wy[e + 1]));
        x[e] = u.x;
        x[e + 1] = u.y;
        y[e] = v.x;
        y[e + 1] = v.y;
      }
    }
    if (!is_v) {
      if (kPairs == kHalfPairs) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 r = cs2[e / 2 * kPlaces + p];
          const float2 c = make_float2(r.x, r.y), sn = make_float2(r.z, r.w), less = make_float2(-r.z, -r.w);
          const float2 u = make_float2(x[e], x[e + 1]), v = make_float2(y[e], y[e + 1]);
          const float2 first = add2(mul2(u, c), mul2(v, less)), second = add2(mul2(v, c), mul2(u, sn));
          x[e] = first.x;
          x[e + 1] = first.y;
          y[e] = second.x;
          y[e + 1] = second.y;
        }
      } else if (kPairs == kNextPairs) {
        auto turn_chunk = [&](float (&f)[8], int c) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float4 r = cs2[e / 2 * kPlaces + c];
            turn_pair(f[2 * e], f[2 * e + 1], make_float2(r.x, r.y));
            turn_pair(f[2 * e + 2], f[2 * e + 3], make_float2(r.z, r.w));
          }
        };
        if (p < a.rot_chunks) turn_chunk(x, p);
        if (p + 8 < a.rot_chunks) turn_chunk(y, p + 8);
      } else if (kPairs == kPartHalfPairs) {
        // chunk c pairs with chunk c + half (c < half); the partner's values by shuffles
        const int half = a.rot_chunks >> 1;
        auto partner = [&](int c) { return c < half ? c + half : c < 2 * half ? c - half : c; };
        const int c0 = partner(p), c1 = partner(p + 8);
        const int from0 = (lane & 24) | (c0 & 7), from1 = (lane & 24) | (c1 & 7);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a0 = __shfl_sync(0xffffffffu, x[e], from0), b0 = __shfl_sync(0xffffffffu, y[e], from0);
          const float a1 = __shfl_sync(0xffffffffu, x[e], from1), b1 = __shfl_sync(0xffffffffu, y[e], from1);
          const float ox = c0 < 8 ? a0 : b0, oy = c1 < 8 ? a1 : b1;
          auto turned = [&](float mine, float other, int c) {
            if (c >= 2 * half) return mine;
            const float2 r = cs[8 * (c < half ? c : c - half) + e];
            return c < half ? __fsub_rn(__fmul_rn(mine, r.x), __fmul_rn(other, r.y))
                            : __fadd_rn(__fmul_rn(mine, r.x), __fmul_rn(other, r.y));
          };
          x[e] = turned(x[e], ox, p);
          y[e] = turned(y[e], oy, p + 8);
        }
      }
    }
    if (is_q) {
      if (h >= 0) {
        uint16_t* dst = a.q_out + t * a.q_out_tok + h * a.q_out_head + 8 * p;
        *reinterpret_cast<uint4*>(dst) = pack<T>(x);
        *reinterpret_cast<uint4*>(dst + 64) = pack<T>(y);
      }
      continue;
    }
    float least = 0.f, most = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      least = fminf(least, fminf(x[e], y[e]));
      most = fmaxf(most, fmaxf(x[e], y[e]));
    }
#pragma unroll
    for (int m = 4; m > 0; m >>= 1) {
      least = fminf(least, __shfl_xor_sync(0xffffffffu, least, m));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
    }
    const float range = __fmul_rn(__fsub_rn(most, least), kFifteenth);
    int bits = __half_as_ushort(__float2half_rn(range));
    bits = min((bits + 15) & ~15, kKv4MaxScaleBits);
    const float s = __half2float(__ushort_as_half(uint16_t(bits)));
    const float inv = bits ? __frcp_rn(s) : 0.f;
    const int z = round_small(fminf(__fmul_rn(-least, inv), 15.f));
    if (h < 0) continue;
    uint8_t* to = base + h * a.head_stride;
    uint32_t* row = reinterpret_cast<uint32_t*>(to + (is_v ? kv4_v_row(a.block_slots, place) : kv4_k_row(a.block_slots, place)));
    row[p] = codes8(x, inv, z);
    row[p + 8] = codes8(y, inv, z);
    if (p == 0)
      *reinterpret_cast<uint16_t*>(to + (is_v ? kv4_v_word(a.block_slots, place) : kv4_k_word(a.block_slots, place))) =
          uint16_t(bits | z);
  }
}

struct Kv4ReadParams {
  uint16_t* out[2];  // k, v (null: not written)
  int64_t out_tok[2], out_head[2];
  const int32_t* slots;
  const uint8_t* cache;
  int64_t page_stride, head_stride, num_slots, rows;  // rows: num_rows * heads
  int32_t heads, log2_page, block_slots, block_bytes;
};

constexpr int kReadThreads = 256;

// Eight lanes a row, each the words p and p + 8 of its codes: 128 contiguous
// bytes of output a step.  A lane has one row in flight, which waits for its slot,
// then for codes and word: 8384 slots of 8 heads 10.2 us (6.5 at the copy rate).
template <typename T>
__global__ void __launch_bounds__(kReadThreads) kv4_read_kernel(const __grid_constant__ Kv4ReadParams a) {
  const int p = threadIdx.x & 7;
  const int64_t step = int64_t(gridDim.x) * (kReadThreads / 8);
  for (int64_t i = int64_t(blockIdx.x) * (kReadThreads / 8) + (threadIdx.x >> 3); i < a.rows; i += step) {
    const int64_t row = i / a.heads;
    const int h = int(i - row * a.heads);
    const int64_t slot = __ldg(a.slots + row);
    const bool there = slot >= 0 && slot < a.num_slots;
    const int in_page = int(slot) & ((1 << a.log2_page) - 1);
    const int block = in_page / a.block_slots, place = in_page - block * a.block_slots;
    const uint8_t* base = a.cache + (slot >> a.log2_page) * a.page_stride + h * a.head_stride + block * a.block_bytes;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      if (!a.out[v]) continue;
      uint16_t* dst = a.out[v] + row * a.out_tok[v] + h * a.out_head[v] + 8 * p;
      uint32_t code[2] = {0u, 0u};
      int word = 0;
      if (there) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            base + (v ? kv4_v_row(a.block_slots, place) : kv4_k_row(a.block_slots, place)));
        code[0] = src[p];
        code[1] = src[p + 8];
        word = *reinterpret_cast<const uint16_t*>(
            base + (v ? kv4_v_word(a.block_slots, place) : kv4_k_word(a.block_slots, place)));
      }
      const float s = __half2float(__ushort_as_half(uint16_t(word & ~15)));
      const int z = word & 15;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = s * float(int((code[c] >> (4 * e)) & 15) - z);
        *reinterpret_cast<uint4*>(dst + 64 * c) = pack<T>(f);
      }
    }
  }
}

// Warps wanted on the card before a token is left to one warp: about one wave.
constexpr int kPartWarps = 152 * kAppendBlocks * kAppendWarps;

template <typename T>
void launch_append(const Kv4AppendParams& a, int pairs, unsigned blocks, cudaStream_t s) {
  const int threads = 32 * kAppendWarps;
  switch (pairs) {
    case kNoPairs: kv4_append_kernel<T, kNoPairs><<<blocks, threads, 0, s>>>(a); break;
    case kHalfPairs: kv4_append_kernel<T, kHalfPairs><<<blocks, threads, 0, s>>>(a); break;
    case kNextPairs: kv4_append_kernel<T, kNextPairs><<<blocks, threads, 0, s>>>(a); break;
    default: kv4_append_kernel<T, kPartHalfPairs><<<blocks, threads, 0, s>>>(a); break;
  }
}

// A 4-bit cache: sizes, pointer, strides.
fi_status check_kv4_cache(const void* cache, const int64_t strides[2], int64_t page_size, int64_t num_pages,
                          int64_t heads) {
  if (!cache || num_pages < 1 || num_pages > INT32_MAX || heads < 1) return FI_ERR_INVALID_ARG;
  if (heads > 65536) return FI_ERR_UNSUPPORTED;
  if (!aligned(cache, 16) || strides[0] % 16 || strides[1] % 16) return FI_ERR_ALIGNMENT;
  int64_t size[2] = {num_pages, heads}, stride[2] = {strides[0], strides[1]};
  return nested(size, stride, int64_t(fi_kv4_page_bytes(page_size))) ? FI_OK : FI_ERR_INVALID_ARG;
}

int log2_of(int64_t page_size) {
  int l = 0;
  while ((int64_t(1) << l) < page_size) ++l;
  return l;
}

}  // namespace
}  // namespace fi

using namespace fi;

extern "C" size_t fi_kv4_page_bytes(int64_t page_size) {
  if (page_size < 1 || page_size > 128 || (page_size & (page_size - 1))) return 0;
  const int slots = kv4_block_slots(int(page_size));
  return size_t(page_size / slots) * size_t(kv4_block_bytes(slots));
}

extern "C" fi_status fi_kv4_append(const fi_kv4_append_args* x, void* stream) {
  if (!x || x->num_tokens < 0 || x->num_tokens > INT32_MAX || x->num_q_heads < 0 || x->num_kv_heads < 0)
    return FI_ERR_INVALID_ARG;
  const fi_rotary* rot = x->rotary;
  if (rot) {
    const fi_status st = check_rotary(rot, x->num_tokens, x->num_q_heads, x->num_kv_heads, x->dtype);
    if (st != FI_OK) return st;
    if (rot->head_dim != FI_KV4_HEAD_DIM) return FI_ERR_UNSUPPORTED;
  }
  if ((x->dtype != FI_FP16 && x->dtype != FI_BF16) || x->num_q_heads > 65536 || x->num_kv_heads > 65536 ||
      fi_kv4_page_bytes(x->page_size) == 0)
    return FI_ERR_UNSUPPORTED;
  if (!eps_ok(x->eps)) return FI_ERR_INVALID_ARG;
  if (x->num_tokens == 0) return FI_OK;
  const bool q = x->num_q_heads > 0;
  if ((rot && !x->positions) || !x->slots || !x->k_in.data || !x->v_in.data || (q && (!x->q_in.data || !x->q_out.data)))
    return FI_ERR_INVALID_ARG;
  fi_status st = check_kv4_cache(x->cache, x->cache_strides, x->page_size, x->num_pages, x->num_kv_heads);
  if (st == FI_OK) st = check_weights(x->q_weight, x->q_weight_stride, FI_KV4_HEAD_DIM);
  if (st == FI_OK) st = check_weights(x->k_weight, x->k_weight_stride, FI_KV4_HEAD_DIM);
  if (st != FI_OK) return st;
  if ((rot && !aligned(x->positions, 4)) || !aligned(x->slots, 4) || !rows_ok(x->k_in) || !rows_ok(x->v_in) ||
      (q && (!rows_ok(x->q_in) || !rows_ok(x->q_out))))
    return FI_ERR_ALIGNMENT;
  if (q && !output_ok(x->q_in, x->q_out, x->num_tokens, x->num_q_heads, FI_KV4_HEAD_DIM)) return FI_ERR_INVALID_ARG;
  Kv4AppendParams a;
  std::memset(&a, 0, sizeof a);
  auto rows = [](const fi_rows& r, int64_t heads) {
    return Kv4Rows{static_cast<const uint16_t*>(r.data), r.stride_tok, r.stride_head, int32_t(heads)};
  };
  if (q) {
    a.q = rows(x->q_in, x->num_q_heads);
    a.q_out = static_cast<uint16_t*>(x->q_out.data);
    a.q_out_tok = x->q_out.stride_tok;
    a.q_out_head = x->q_out.stride_head;
  }
  a.k = rows(x->k_in, x->num_kv_heads);
  a.v = rows(x->v_in, x->num_kv_heads);
  a.q_weight = x->q_weight;
  a.k_weight = x->k_weight;
  a.q_weight_stride = x->q_weight_stride;
  a.k_weight_stride = x->k_weight_stride;
  a.positions = x->positions;
  a.slots = x->slots;
  a.cache = static_cast<uint8_t*>(x->cache);
  a.page_stride = x->cache_strides[0];
  a.head_stride = x->cache_strides[1];
  a.num_slots = x->num_pages * x->page_size;
  a.num_tokens = int32_t(x->num_tokens);
  a.log2_page = log2_of(x->page_size);
  a.block_slots = kv4_block_slots(int(x->page_size));
  a.block_bytes = kv4_block_bytes(a.block_slots);
  a.eps = float(x->eps);
  int pairs = kNoPairs;
  if (rot) {
    a.rot_chunks = rot->rot_dim / 8;
    a.amplitude = rot->amplitude;
    std::memcpy(a.turns, rot->turns, sizeof(uint64_t) * size_t(rot->rot_dim / 2));
    pairs = rot->interleaved ? kNextPairs : rot->rot_dim == FI_KV4_HEAD_DIM ? kHalfPairs : kPartHalfPairs;
  }
  const int groups = (a.q.heads + 3) / 4 + 2 * ((a.k.heads + 3) / 4);
  const int want = kPartWarps / a.num_tokens;
  a.parts = want < 1 ? 1 : want > groups ? groups : want;
  const int64_t warps = int64_t(a.num_tokens) * a.parts;
  const unsigned blocks = unsigned((warps + kAppendWarps - 1) / kAppendWarps);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x->dtype == FI_BF16)
    launch_append<__nv_bfloat16>(a, pairs, blocks, s);
  else
    launch_append<__half>(a, pairs, blocks, s);
  return cudaGetLastError() == cudaSuccess ? FI_OK : FI_ERR_CUDA;
}

extern "C" fi_status fi_kv4_read(const fi_kv4_read_args* x, void* stream) {
  if (!x || x->num_rows < 0 || x->num_rows > INT32_MAX) return FI_ERR_INVALID_ARG;
  if ((x->dtype != FI_FP16 && x->dtype != FI_BF16) || fi_kv4_page_bytes(x->page_size) == 0) return FI_ERR_UNSUPPORTED;
  if (x->num_rows == 0 || (!x->k_out.data && !x->v_out.data)) return FI_OK;
  if (!x->slots) return FI_ERR_INVALID_ARG;
  const fi_status st = check_kv4_cache(x->cache, x->cache_strides, x->page_size, x->num_pages, x->num_kv_heads);
  if (st != FI_OK) return st;
  if (!aligned(x->slots, 4)) return FI_ERR_ALIGNMENT;
  Kv4ReadParams a;
  std::memset(&a, 0, sizeof a);
  const fi_rows* outs[2] = {&x->k_out, &x->v_out};
  for (int v = 0; v < 2; ++v) {
    if (!outs[v]->data) continue;
    if (!rows_ok(*outs[v])) return FI_ERR_ALIGNMENT;
    int64_t size[2] = {x->num_rows, x->num_kv_heads}, stride[2] = {outs[v]->stride_tok, outs[v]->stride_head};
    if (!nested(size, stride, FI_KV4_HEAD_DIM)) return FI_ERR_INVALID_ARG;
    a.out[v] = static_cast<uint16_t*>(outs[v]->data);
    a.out_tok[v] = outs[v]->stride_tok;
    a.out_head[v] = outs[v]->stride_head;
  }
  if (a.out[0] && a.out[1] &&
      (a.out[0] == a.out[1] || !output_ok(x->k_out, x->v_out, x->num_rows, x->num_kv_heads, FI_KV4_HEAD_DIM)))
    return FI_ERR_INVALID_ARG;
  a.slots = x->slots;
  a.cache = static_cast<const uint8_t*>(x->cache);
  a.page_stride = x->cache_strides[0];
  a.head_stride = x->cache_strides[1];
  a.num_slots = x->num_pages * x->page_size;
  a.rows = x->num_rows * x->num_kv_heads;
  a.heads = int32_t(x->num_kv_heads);
  a.log2_page = log2_of(x->page_size);
  a.block_slots = kv4_block_slots(int(x->page_size));
  a.block_bytes = kv4_block_bytes(a.block_slots);
  const int64_t blocks = (a.rows + kReadThreads / 8 - 1) / (kReadThreads / 8);
  const unsigned grid = unsigned(blocks < (1 << 20) ? blocks : (1 << 20));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x->dtype == FI_BF16)
    kv4_read_kernel<__nv_bfloat16><<<grid, kReadThreads, 0, s>>>(a);
  else
    kv4_read_kernel<__half><<<grid, kReadThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FI_OK : FI_ERR_CUDA;
}
