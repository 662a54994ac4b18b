// norm_append.cu -- RMS norms of query and key heads, rotary positions and the
// append of keys and values to the paged cache, in one launch.
//
// y = x r w with r = 1 / sqrt(mean(x^2) + eps) over a head, then the rotation of
// rotary.cu.  A head has to be in registers whole before its first value can be
// written: the lanes that hold it take a place each (8 pairs, or 16 bytes), and
// the sum of squares goes over them by shuffles.
//
// Bound by the bytes of q, k and v, each read and written once: what counts is
// how many of them are in flight, so registers are few (cos and sin stay in
// shared memory, v's rows of the heads' size go through the heads' loop) and a
// head's successor is loaded before the head is turned.
// Measured: 16384 tokens of 32 + 8 heads of 128 in 71 us, 5.7 TB/s (60 us at the
// copy rate; 87 before the turns' reads met no bank twice and the sum took no more
// shuffles than a head has lanes for); 1111 tokens of 24 + 24 heads of 80 in 9.6 us,
// where four blocks on an SM with cos and sin in registers took 16.3; 64 tokens in
// 3.5 us, the launch and one chain of loads.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "rotary.h"

namespace fi {
namespace {

constexpr int kNormWarps = 4;   // warps of a block
constexpr int kNormBlocks = 8;  // blocks of an SM
constexpr int kValueAhead = 4;  // 16-byte pieces of v a lane has in flight

struct NormParams {
  RotaryRows q, k, v;
  const float *q_weight, *k_weight;  // null: not normed
  int64_t q_weight_stride, k_weight_stride;
  const int32_t* positions;
  const int32_t* slots;
  int64_t num_slots;
  int32_t num_tokens, parts;  // warps per token
  int32_t log2_page, half_places;  // half_places: the largest power of two below the places of a head (0: one place)
  int32_t v_like_heads;  // v's rows have the heads' size and go through their loop, as copies
  int32_t head_chunks, rot_chunks, v_chunks;  // 16-byte chunks of a head, of its rotated part, of a v row
  float amplitude, eps, inv_dim;
  uint64_t turns[FI_ROTARY_MAX_PAIRS];
};

__device__ __forceinline__ void load8(const float* w, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w)), b = __ldg(reinterpret_cast<const float4*>(w) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(32 * kNormWarps, kNormBlocks) norm_append_kernel(const __grid_constant__ NormParams a) {
  __shared__ alignas(16) float2 s_cs[kNormWarps][FI_ROTARY_MAX_PAIRS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * kNormWarps + warp;
  const int t = int(w / a.parts), part = int(w - int64_t(t) * a.parts);
  if (t >= a.num_tokens) return;
  const int32_t pos = __ldg(a.positions + t);
  const int64_t slot = __ldg(a.slots + t);
  const bool store_kv = slot >= 0 && slot < a.num_slots;

  // this lane's place and first head (q heads, then k heads, then v's)
  const int pair_places = kInterleaved ? a.rot_chunks : a.rot_chunks >> 1;
  const int places = pair_places + a.head_chunks - a.rot_chunks;
  const int at_once = 32 / places, h_off = lane / places, place = lane - h_off * places;
  const bool pairs = place < pair_places, active = h_off < at_once, two = !kInterleaved && pairs;
  const int off = 8 * (pairs ? place : place + a.rot_chunks - pair_places);
  const int other = 8 * pair_places;  // from the first members of 8 pairs to the second
  const int step = at_once * a.parts;
  const int nq = a.q.heads, nk = a.k.heads, turned = nq + nk, heads = turned + (a.v_like_heads ? a.v.heads : 0);
  uint4 lo, hi;
  auto load = [&](int h) {
    lo = hi = make_uint4(0u, 0u, 0u, 0u);
    if (!active || h >= heads || (h >= nq && !store_kv)) return;
    const RotaryRows& rows = h < nq ? a.q : h < turned ? a.k : a.v;
    const uint16_t* src = rows.in + t * rows.in_tok + (h < nq ? h : h < turned ? h - nq : h - turned) * rows.in_head + off;
    lo = *reinterpret_cast<const uint4*>(src);
    if (two) hi = *reinterpret_cast<const uint4*>(src + other);
  };
  const int first = part * at_once + h_off;
  load(first);

  // pairs 2 e and 2 e + 1 of place p together, next to those of the other places: lanes read without bank conflicts
  constexpr int kMine = kInterleaved ? 4 : 8;  // pairs of a place
  float2* cs = s_cs[warp];
#pragma unroll 2
  for (int i = lane; i < a.rot_chunks * 4; i += 32) {
    const uint64_t turn = uint64_t(int64_t(pos)) * a.turns[i];  // modulo one turn
    float sn, c;
    sincospif(float(int32_t(turn >> 32)) * 4.6566128730773926e-10f, &sn, &c);  // 2^-31: half turns in [-1, 1]
    cs[2 * ((i % kMine >> 1) * pair_places + i / kMine) + (i & 1)] = make_float2(c * a.amplitude, sn * a.amplitude);
  }
  __syncwarp();
  const float4* const mine = reinterpret_cast<const float4*>(cs) + (pairs ? place : 0);
  const int64_t page = slot >> a.log2_page, in_page = slot & ((int64_t(1) << a.log2_page) - 1);
  // the shuffles need every lane, so the loop runs while any head of the warp is left
  for (int h = first; h - h_off < heads; h += step) {
    const bool is_q = h < nq, is_v = h >= turned;
    float x[8], y[8];
    unpack<T>(lo, x);
    unpack<T>(hi, y);
    const uint4 raw_lo = lo, raw_hi = hi;
    load(h + step);  // in flight while this head is turned
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], fmaf(y[e], y[e], sum));
    // over the head's lanes, into its first, and back
#pragma unroll 1
    for (int m = a.half_places; m > 0; m >>= 1) {
      const float more = __shfl_down_sync(0xffffffffu, sum, m);
      if (place + m < places) sum += more;
    }
    sum = __shfl_sync(0xffffffffu, sum, lane - place);
    if (!active || h >= heads || (!is_q && !store_kv)) continue;
    const RotaryRows& rows = is_q ? a.q : is_v ? a.v : a.k;
    const int head = is_q ? h : is_v ? h - turned : h - nq;
    uint16_t* const dst = rows.out + (is_q ? t * rows.out_tok : page * rows.out_tok + in_page * rows.out_slot) +
                          head * rows.out_head + off;
    if (is_v) {
      *reinterpret_cast<uint4*>(dst) = raw_lo;
      if (two) *reinterpret_cast<uint4*>(dst + other) = raw_hi;
      continue;
    }
    const float* weight = is_q ? a.q_weight : a.k_weight;
    if (weight) {
      const float root = rsqrtf(fmaf(sum, a.inv_dim, a.eps));
      weight += head * (is_q ? a.q_weight_stride : a.k_weight_stride) + off;
      float g[8];
      load8(weight, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= root * g[e];
      if (two) {
        load8(weight + other, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= root * g[e];
      }
    }
    if (pairs) {
#pragma unroll
      for (int e = 0; e < kMine; e += 2) {
        const float4 r = mine[e / 2 * pair_places];
        if (kInterleaved) {
          const float x0 = x[2 * e], x1 = x[2 * e + 1], x2 = x[2 * e + 2], x3 = x[2 * e + 3];
          x[2 * e] = x0 * r.x - x1 * r.y;
          x[2 * e + 1] = x1 * r.x + x0 * r.y;
          x[2 * e + 2] = x2 * r.z - x3 * r.w;
          x[2 * e + 3] = x3 * r.z + x2 * r.w;
        } else {
          const float x0 = x[e % 8], x1 = y[e % 8], x2 = x[e % 8 + 1], x3 = y[e % 8 + 1];
          x[e % 8] = x0 * r.x - x1 * r.y;
          y[e % 8] = x1 * r.x + x0 * r.y;
          x[e % 8 + 1] = x2 * r.z - x3 * r.w;
          y[e % 8 + 1] = x3 * r.z + x2 * r.w;
        }
      }
      if (two) *reinterpret_cast<uint4*>(dst + other) = pack<T>(y);
    }
    *reinterpret_cast<uint4*>(dst) = pack<T>(x);
  }
  // v of rows of another size: 16-byte pieces, in order
  const int v_tasks = a.v_like_heads ? 0 : a.v.heads * a.v_chunks, v_step = 32 * a.parts;
  if (!store_kv || v_tasks == 0) return;
  auto piece = [&](int i, int64_t head, int64_t base) -> int64_t {
    const int h = i / a.v_chunks;
    return base + h * head + 8 * (i - h * a.v_chunks);
  };
  const int64_t v_base = page * a.v.out_tok + in_page * a.v.out_slot;
  for (int v0 = 32 * part + lane; v0 < v_tasks; v0 += kValueAhead * v_step) {
    uint4 vv[kValueAhead];
#pragma unroll
    for (int u = 0; u < kValueAhead; ++u)
      if (v0 + u * v_step < v_tasks)
        vv[u] = *reinterpret_cast<const uint4*>(a.v.in + t * a.v.in_tok + piece(v0 + u * v_step, a.v.in_head, 0));
#pragma unroll
    for (int u = 0; u < kValueAhead; ++u)
      if (v0 + u * v_step < v_tasks)
        *reinterpret_cast<uint4*>(a.v.out + piece(v0 + u * v_step, a.v.out_head, v_base)) = vv[u];
  }
}

// Warps wanted on the card before a token is left to one warp: about one wave.
constexpr int kPartWarps = 152 * kNormBlocks * kNormWarps;

}  // namespace
}  // namespace fi

using namespace fi;

extern "C" fi_status fi_norm_rotary_append(const fi_norm_rotary_append_args* n, void* stream) {
  if (!n) return FI_ERR_INVALID_ARG;
  const fi_rotary_append_args* x = &n->append;
  fi_status st = check_append(x);
  if (st != FI_OK) return st;
  if (!eps_ok(n->eps)) return FI_ERR_INVALID_ARG;
  if (x->num_tokens == 0) return FI_OK;
  const fi_rotary* rot = x->rotary;
  st = check_weights(n->q_weight, n->q_weight_stride, rot->head_dim);
  if (st == FI_OK) st = check_weights(n->k_weight, n->k_weight_stride, rot->head_dim);
  if (st != FI_OK) return st;
  NormParams a;
  std::memset(&a, 0, sizeof a);
  if (x->num_q_heads > 0) a.q = rows_of(x->q_in, x->q_out, x->num_q_heads);
  a.k = rows_to_cache(x->k_in, x->k_cache, x->k_strides, x->num_kv_heads);
  if (x->v_dim > 0) a.v = rows_to_cache(x->v_in, x->v_cache, x->v_strides, x->num_kv_heads);
  a.v_chunks = int32_t(x->v_dim / 8);
  a.q_weight = n->q_weight;
  a.k_weight = n->k_weight;
  a.q_weight_stride = n->q_weight_stride;
  a.k_weight_stride = n->k_weight_stride;
  a.positions = x->positions;
  a.slots = x->slots;
  a.num_slots = x->num_pages * x->page_size;
  while ((1 << a.log2_page) < x->page_size) ++a.log2_page;
  a.num_tokens = int32_t(x->num_tokens);
  a.head_chunks = rot->head_dim / 8;
  a.rot_chunks = rot->rot_dim / 8;
  a.amplitude = rot->amplitude;
  a.eps = float(n->eps);
  a.inv_dim = 1.f / float(rot->head_dim);
  std::memcpy(a.turns, rot->turns, sizeof(uint64_t) * size_t(rot->rot_dim / 2));
  const int places = (rot->interleaved ? a.rot_chunks : a.rot_chunks / 2) + a.head_chunks - a.rot_chunks;
  while ((1 << a.half_places) < places) ++a.half_places;
  a.half_places = (1 << a.half_places) >> 1;
  a.v_like_heads = x->v_dim == rot->head_dim ? 1 : 0;
  // Few tokens: a token's heads are spread over more warps, at least one head a lane
  const int at_once = 32 / places, heads = a.q.heads + a.k.heads + (a.v_like_heads ? a.v.heads : 0);
  const int rot_parts = (heads + at_once - 1) / at_once, v_parts = a.v_like_heads ? 0 : (a.v.heads * a.v_chunks + 31) / 32;
  const int most = rot_parts > v_parts ? rot_parts : v_parts;
  const int want = kPartWarps / a.num_tokens;
  a.parts = want < 1 ? 1 : want > most ? most : want;
  const int64_t warps = int64_t(a.num_tokens) * a.parts;
  const unsigned blocks = unsigned((warps + kNormWarps - 1) / kNormWarps);
  const int threads = 32 * kNormWarps;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x->dtype == FI_BF16) {
    if (rot->interleaved)
      norm_append_kernel<__nv_bfloat16, true><<<blocks, threads, 0, s>>>(a);
    else
      norm_append_kernel<__nv_bfloat16, false><<<blocks, threads, 0, s>>>(a);
  } else {
    if (rot->interleaved)
      norm_append_kernel<__half, true><<<blocks, threads, 0, s>>>(a);
    else
      norm_append_kernel<__half, false><<<blocks, threads, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FI_OK : FI_ERR_CUDA;
}
