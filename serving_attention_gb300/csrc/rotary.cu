// rotary.cu -- rotary positions of a step's new tokens, and the append of
// their keys and values to the paged cache.
//
// Pair i of a token at position n turns by the angle n f_i.  The rate is kept
// in turns per position as a 64-bit binary fraction F_i, so n F_i mod 2^64 is
// the exact fraction of a turn at any position: no table to read, no argument
// reduction, and the angle of position 10^6 is as exact as that of position
// 1 (an fp32 product of position and rate is off by 0.06 rad there).
//
// Bound by the bytes of q, k and v (each read and written once).  One warp per
// token, or per part of one when there are few tokens.  A lane keeps to one
// place of a head (8 pairs, or a 16-byte piece that is copied), so its cos and
// sin stay in registers while it goes from head to head; the values of the
// first heads and of v are loaded before the angles are computed.
// Measured: 16384 tokens of 32 + 8 + 8 heads of 128, 403 MB, 73.5 us (5.5 TB/s,
// 81 % of the copy rate); 64 tokens 3.9 us, a launch's latency.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "rotary.h"

namespace fi {
namespace {

constexpr int kRotaryWarps = 4;  // warps of a block (with 8: 75.4 against 73.4 us for 16384 tokens)
constexpr int kRotaryAhead = 2;  // heads a lane has in flight
constexpr int kValueAhead = 4;   // 16-byte pieces of v a lane has in flight

struct RotaryParams {
  RotaryRows q, k, v;
  const int32_t* positions;
  const int32_t* slots;  // null: k goes to row t of k.out
  int64_t num_slots;
  int32_t num_tokens, parts;  // warps per token
  int32_t log2_page;
  int32_t head_chunks, rot_chunks, v_chunks;  // 16-byte chunks of a head, of its rotated part, of a v row
  float amplitude;
  uint64_t turns[FI_ROTARY_MAX_PAIRS];
};

// The place of a lane: the two 16-byte pieces that hold 8 pairs (half layout),
// or one that holds 4 (interleaved), or one behind the rotated dims; 32 /
// places heads at a time.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(32 * kRotaryWarps, 6) rotary_kernel(const __grid_constant__ RotaryParams a) {
  __shared__ float2 s_cs[kRotaryWarps][FI_ROTARY_MAX_PAIRS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * kRotaryWarps + warp;
  const int t = int(w / a.parts), part = int(w - int64_t(t) * a.parts);
  if (t >= a.num_tokens) return;
  const int32_t pos = __ldg(a.positions + t);
  const int64_t slot = a.slots ? __ldg(a.slots + t) : t;

  // this lane's place and first head (q heads, then k heads)
  const int pair_places = kInterleaved ? a.rot_chunks : a.rot_chunks >> 1;
  const int places = pair_places + a.head_chunks - a.rot_chunks;
  const int at_once = 32 / places, h_off = lane / places, place = lane - h_off * places;
  const bool pairs = place < pair_places, active = h_off < at_once;
  const int off = 8 * (pairs ? place : place + a.rot_chunks - pair_places);
  const int other = 8 * pair_places;  // from the first members of 8 pairs to the second
  const int step = at_once * a.parts;
  const uint16_t *q_in = a.q.in + t * a.q.in_tok + off, *k_in = a.k.in + t * a.k.in_tok + off;
  const int heads = a.q.heads + a.k.heads;
  uint4 lo[kRotaryAhead], hi[kRotaryAhead];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kRotaryAhead; ++u) {
      const int h = h0 + u * step;
      if (!active || h >= heads) continue;
      const uint16_t* src = h < a.q.heads ? q_in + h * a.q.in_head : k_in + (h - a.q.heads) * a.k.in_head;
      lo[u] = *reinterpret_cast<const uint4*>(src);
      if (!kInterleaved && pairs) hi[u] = *reinterpret_cast<const uint4*>(src + other);
    }
  };
  int h0 = part * at_once + h_off;
  load(h0);
  // v: 16-byte pieces, in order
  const int v_tasks = a.v.heads * a.v_chunks, v_step = 32 * a.parts;
  const uint16_t* v_in = a.v.in + t * a.v.in_tok;
  uint4 vv[kValueAhead];
  auto v_at = [&](int i, int64_t head, int64_t base) -> int64_t {
    const int h = i / a.v_chunks;
    return base + h * head + 8 * (i - h * a.v_chunks);
  };
  auto load_v = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kValueAhead; ++u)
      if (i0 + u * v_step < v_tasks) vv[u] = *reinterpret_cast<const uint4*>(v_in + v_at(i0 + u * v_step, a.v.in_head, 0));
  };
  int v0 = 32 * part + lane;
  load_v(v0);

  float2* cs = s_cs[warp];
  for (int i = lane; i < a.rot_chunks * 4; i += 32) {
    const uint64_t turn = uint64_t(int64_t(pos)) * a.turns[i];  // modulo one turn
    float sn, c;
    sincospif(float(int32_t(turn >> 32)) * 4.6566128730773926e-10f, &sn, &c);  // 2^-31: half turns in [-1, 1]
    cs[i] = make_float2(c * a.amplitude, sn * a.amplitude);
  }
  __syncwarp();
  constexpr int kMine = kInterleaved ? 4 : 8;
  float2 r[kMine];
  if (pairs) {
    const float4* mine = reinterpret_cast<const float4*>(cs + kMine * place);
#pragma unroll
    for (int e = 0; e < kMine / 2; ++e) {
      const float4 x = mine[e];
      r[2 * e] = make_float2(x.x, x.y);
      r[2 * e + 1] = make_float2(x.z, x.w);
    }
  }
  const bool store_kv = !a.slots || (slot >= 0 && slot < a.num_slots);
  const int64_t page = a.slots ? slot >> a.log2_page : slot;
  const int64_t in_page = a.slots ? slot & ((int64_t(1) << a.log2_page) - 1) : 0;
  uint16_t* q_out = a.q.out + t * a.q.out_tok + off;
  uint16_t* k_out = a.k.out + page * a.k.out_tok + in_page * a.k.out_slot + off;
  for (; h0 < heads; h0 += kRotaryAhead * step) {
#pragma unroll
    for (int u = 0; u < kRotaryAhead; ++u) {
      const int h = h0 + u * step;
      if (!active || h >= heads || (h >= a.q.heads && !store_kv)) continue;
      uint16_t* dst = h < a.q.heads ? q_out + h * a.q.out_head : k_out + (h - a.q.heads) * a.k.out_head;
      if (pairs) {
        float x[8];
        unpack<T>(lo[u], x);
        if (kInterleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x0 = x[2 * e], x1 = x[2 * e + 1];
            x[2 * e] = x0 * r[e].x - x1 * r[e].y;
            x[2 * e + 1] = x1 * r[e].x + x0 * r[e].y;
          }
        } else {
          float y[8];
          unpack<T>(hi[u], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x0 = x[e], x1 = y[e];
            x[e] = x0 * r[e % kMine].x - x1 * r[e % kMine].y;
            y[e] = x1 * r[e % kMine].x + x0 * r[e % kMine].y;
          }
          *reinterpret_cast<uint4*>(dst + other) = pack<T>(y);
        }
        lo[u] = pack<T>(x);
      }
      *reinterpret_cast<uint4*>(dst) = lo[u];
    }
    load(h0 + kRotaryAhead * step);
  }
  if (!store_kv) return;
  const int64_t v_base = page * a.v.out_tok + in_page * a.v.out_slot;
  for (; v0 < v_tasks; v0 += kValueAhead * v_step) {
#pragma unroll
    for (int u = 0; u < kValueAhead; ++u)
      if (v0 + u * v_step < v_tasks)
        *reinterpret_cast<uint4*>(a.v.out + v_at(v0 + u * v_step, a.v.out_head, v_base)) = vv[u];
    load_v(v0 + kValueAhead * v_step);
  }
}

// Warps wanted on the card before a token is left to one warp: about what is
// resident.  With twice as many, 1111 tokens of 80 dims took 9.7 us for 5.8.
constexpr int kPartWarps = 4096;

cudaError_t launch_rotary(RotaryParams& a, const fi_rotary* rot, fi_dtype dtype, cudaStream_t s) {
  a.head_chunks = rot->head_dim / 8;
  a.rot_chunks = rot->rot_dim / 8;
  a.amplitude = rot->amplitude;
  std::memcpy(a.turns, rot->turns, sizeof(uint64_t) * size_t(rot->rot_dim / 2));
  // Few tokens: a token's heads are spread over more warps, at least one head a lane
  const int places = (rot->interleaved ? a.rot_chunks : a.rot_chunks / 2) + a.head_chunks - a.rot_chunks;
  const int at_once = 32 / places, heads = a.q.heads + a.k.heads;
  const int rot_parts = (heads + at_once - 1) / at_once, v_parts = (a.v.heads * a.v_chunks + 31) / 32;
  const int most = rot_parts > v_parts ? rot_parts : v_parts;
  const int want = kPartWarps / a.num_tokens;
  a.parts = want < 1 ? 1 : want > most ? most : want;
  const int64_t warps = int64_t(a.num_tokens) * a.parts;
  const unsigned blocks = unsigned((warps + kRotaryWarps - 1) / kRotaryWarps);
  const int threads = 32 * kRotaryWarps;
  if (dtype == FI_BF16) {
    if (rot->interleaved)
      rotary_kernel<__nv_bfloat16, true><<<blocks, threads, 0, s>>>(a);
    else
      rotary_kernel<__nv_bfloat16, false><<<blocks, threads, 0, s>>>(a);
  } else {
    if (rot->interleaved)
      rotary_kernel<__half, true><<<blocks, threads, 0, s>>>(a);
    else
      rotary_kernel<__half, false><<<blocks, threads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace fi

using namespace fi;

extern "C" fi_status fi_rotary_setup(const fi_rotary_config* cfg, fi_rotary* out) {
  if (!cfg || !out) return FI_ERR_INVALID_ARG;
  const int D = cfg->head_dim, R = cfg->rot_dim;
  if (D < 16 || D > 2 * FI_ROTARY_MAX_PAIRS || D % 8 || R < 16 || R > D || R % 16) return FI_ERR_UNSUPPORTED;
  if (cfg->interleaved != 0 && cfg->interleaved != 1) return FI_ERR_INVALID_ARG;
  if (cfg->scaling < FI_ROTARY_NONE || cfg->scaling > FI_ROTARY_YARN) return FI_ERR_INVALID_ARG;
  const double s = cfg->factor, two_pi = 6.283185307179586476925;
  double theta = cfg->theta;
  if (!(theta > 1.0 && std::isfinite(theta) && s >= 1.0 && std::isfinite(s))) return FI_ERR_INVALID_ARG;
  if (!(cfg->amplitude >= 0.f && std::isfinite(cfg->amplitude))) return FI_ERR_INVALID_ARG;
  const double L = cfg->original_positions, lo = cfg->low_turns, hi = cfg->high_turns;
  const bool parts = cfg->scaling == FI_ROTARY_BY_PARTS, yarn = cfg->scaling == FI_ROTARY_YARN;
  if ((parts || yarn) && !(L > 0 && lo > 0 && hi > lo && std::isfinite(hi))) return FI_ERR_INVALID_ARG;
  if (cfg->scaling == FI_ROTARY_NTK) theta *= std::pow(s, double(R) / double(R - 2));
  auto dim_of = [&](double turns) { return R * std::log(L / (turns * two_pi)) / (2.0 * std::log(theta)); };
  double d_lo = 0, d_hi = 0;
  if (yarn) {
    d_lo = std::fmax(0.0, std::floor(dim_of(hi)));
    d_hi = std::fmin(double(R - 1), std::ceil(dim_of(lo)));
  }
  std::memset(out, 0, sizeof *out);
  out->head_dim = D;
  out->rot_dim = R;
  out->interleaved = cfg->interleaved;
  out->amplitude = cfg->amplitude > 0.f ? cfg->amplitude : yarn ? float(0.1 * std::log(s) + 1.0) : 1.f;
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / R);
    double slow = 0.0;  // share of the slowed rate f / s
    if (cfg->scaling == FI_ROTARY_LINEAR) slow = 1.0;
    if (parts) slow = 1.0 - std::fmin(1.0, std::fmax(0.0, (L * f / two_pi - lo) / (hi - lo)));
    if (yarn) slow = std::fmin(1.0, std::fmax(0.0, (i - d_lo) / (d_hi > d_lo ? d_hi - d_lo : 1e-3)));
    f = f / s * slow + f * (1.0 - slow);
    out->turns[i] = uint64_t(std::ldexp(f / two_pi, 64) + 0.5);  // f <= 1, so under a turn
  }
  return FI_OK;
}

extern "C" fi_status fi_rotary_apply(const fi_rotary_apply_args* x, void* stream) {
  if (!x) return FI_ERR_INVALID_ARG;
  const fi_status st = check_rotary(x->rotary, x->num_tokens, x->num_q_heads, x->num_kv_heads, x->dtype);
  if (st != FI_OK) return st;
  const bool q = x->num_q_heads > 0, k = x->num_kv_heads > 0;
  if (x->num_tokens == 0 || (!q && !k)) return FI_OK;
  if (!x->positions || (q && (!x->q_in.data || !x->q_out.data)) || (k && (!x->k_in.data || !x->k_out.data)))
    return FI_ERR_INVALID_ARG;
  if (!aligned(x->positions, 4) || (q && (!rows_ok(x->q_in) || !rows_ok(x->q_out))) ||
      (k && (!rows_ok(x->k_in) || !rows_ok(x->k_out))))
    return FI_ERR_ALIGNMENT;
  if ((q && !output_ok(x->q_in, x->q_out, x->num_tokens, x->num_q_heads, x->rotary->head_dim)) ||
      (k && !output_ok(x->k_in, x->k_out, x->num_tokens, x->num_kv_heads, x->rotary->head_dim)))
    return FI_ERR_INVALID_ARG;
  RotaryParams a;
  std::memset(&a, 0, sizeof a);
  a.q = rows_of(x->q_in, x->q_out, x->num_q_heads);
  a.k = rows_of(x->k_in, x->k_out, x->num_kv_heads);
  a.positions = x->positions;
  a.num_tokens = int32_t(x->num_tokens);
  return launch_rotary(a, x->rotary, fi_dtype(x->dtype), static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FI_OK
             : FI_ERR_CUDA;
}

extern "C" fi_status fi_rotary_append(const fi_rotary_append_args* x, void* stream) {
  const fi_status st = check_append(x);
  if (st != FI_OK) return st;
  if (x->num_tokens == 0) return FI_OK;
  RotaryParams a;
  std::memset(&a, 0, sizeof a);
  if (x->num_q_heads > 0) a.q = rows_of(x->q_in, x->q_out, x->num_q_heads);
  a.k = rows_to_cache(x->k_in, x->k_cache, x->k_strides, x->num_kv_heads);
  if (x->v_dim > 0) a.v = rows_to_cache(x->v_in, x->v_cache, x->v_strides, x->num_kv_heads);
  a.v_chunks = int32_t(x->v_dim / 8);
  a.positions = x->positions;
  a.slots = x->slots;
  a.num_slots = x->num_pages * x->page_size;
  while ((1 << a.log2_page) < x->page_size) ++a.log2_page;
  a.num_tokens = int32_t(x->num_tokens);
  return launch_rotary(a, x->rotary, fi_dtype(x->dtype), static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FI_OK
             : FI_ERR_CUDA;
}
