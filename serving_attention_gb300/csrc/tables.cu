// tables.cu -- page tables and slot maps of a step, built on the GPU.
//
// Three prefix sums over the requests (query tokens, pages, pages taken from
// the free list), then every page-table entry and every token looked up in
// them.  One launch without any wait between blocks: each block scans all
// lengths itself (8 bytes a request, from L2 after the first block), keeps the
// sums in shared memory and takes its share of the entries.  Bound by
// latency: a step of 64 requests takes 4.7 us (the launch and the scans), one of
// 4096 requests with 1.5 million pages 12 us (launch 4.2, scans 3.4, entries 4.4;
// its 12.3 MB would take 1.8).
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "../../include/fi_step.h"
#include "launch.h"

namespace fi {
namespace {

// 256 threads: a step of 64 requests takes 4.6 us a call (5.2 with 512), one of
// 4096 requests 11.9 either way (19.2 with 128).
constexpr int kTableThreads = 256;
constexpr int kTableWarps = kTableThreads / 32;
constexpr int kTableAhead = 4;  // page-table entries a thread has in flight
constexpr size_t kPlainSmem = 47 * 1024;  // dynamic shared memory without an opt-in, beside the static arrays

struct TableParams {
  const int32_t *qo_lens, *kv_lens;
  int32_t batch, log2_page;
  int32_t* table;
  int64_t table_stride;
  int32_t table_width;
  const int32_t* free_pages;
  int32_t num_free;
  const int32_t* free_head;
  int32_t *qo_indptr, *kv_indptr, *last_page_len, *kv_indices;
  int32_t max_pages;
  int32_t *positions, *slots;
  int32_t max_tokens;
  int32_t* counts;
};

struct Sums {
  int64_t qo, pages, taken;
};

// Shared arrays by request have a gap after every 8 entries: the threads that
// sum 8 consecutive entries each would otherwise all meet in four banks.
__host__ __device__ __forceinline__ int gap(int i) { return i + (i >> 3); }

// The last entry of s[0 .. n] at or below x (s[0] <= x < s[n]).
__device__ __forceinline__ int find(const int32_t* s, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s[gap(mid)] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kTableThreads) step_tables_kernel(const __grid_constant__ TableParams a) {
  extern __shared__ int32_t smem[];
  const int B = a.batch, P = 1 << a.log2_page, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_smem = gap(B) + 1;
  int32_t *s_qo = smem, *s_kv = smem + n_smem, *s_new = smem + 2 * n_smem;
  __shared__ Sums s_warp[kTableWarps];
  __shared__ int s_bad;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int32_t head = a.free_head ? __ldg(a.free_head) : 0;
  auto pages_of = [&](int32_t len) { return int32_t((int64_t(len) + P - 1) >> a.log2_page); };

  // The requests' counts, loaded side by side; then thread t sums requests
  // [t * per, (t + 1) * per) and the threads are scanned.
  bool bad = false;
#pragma unroll 4
  for (int b = tid; b < B; b += kTableThreads) {
    int32_t q = __ldg(a.qo_lens + b), kv = __ldg(a.kv_lens + b);
    if (q < 0 || q > kv || int64_t(kv) > (int64_t(a.table_width) << a.log2_page)) {
      bad = true;
      q = kv = 0;
    }
    s_qo[gap(b)] = q;
    s_kv[gap(b)] = pages_of(kv);
    s_new[gap(b)] = pages_of(kv) - pages_of(kv - q);
  }
  if (bad) s_bad = 1;
  __syncthreads();
  const int per = (B + kTableThreads - 1) / kTableThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  Sums mine{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    mine.qo += s_qo[gap(b)];
    mine.pages += s_kv[gap(b)];
    mine.taken += s_new[gap(b)];
  }
  Sums inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, inc.qo, d), y = __shfl_up_sync(0xffffffffu, inc.pages, d),
                  z = __shfl_up_sync(0xffffffffu, inc.taken, d);
    if (lane >= d) {
      inc.qo += x;
      inc.pages += y;
      inc.taken += z;
    }
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  Sums before{0, 0, 0}, total{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kTableWarps; ++w) {
    const Sums x = s_warp[w];
    if (w < warp) {
      before.qo += x.qo;
      before.pages += x.pages;
      before.taken += x.taken;
    }
    total.qo += x.qo;
    total.pages += x.pages;
    total.taken += x.taken;
  }
  // Every block sees the same lengths and comes to the same verdict.
  int status = FI_OK;
  if (s_bad)
    status = FI_ERR_INVALID_ARG;
  else if (total.qo > a.max_tokens || total.pages > a.max_pages || head < 0 || head + total.taken > a.num_free)
    status = FI_ERR_CAPACITY;
  if (blockIdx.x == 0 && tid < FI_STEP_COUNTS) {
    auto cut = [](int64_t x) { return int32_t(x < INT_MAX ? x : INT_MAX); };
    a.counts[tid] = tid == 0   ? cut(total.qo)
                    : tid == 1 ? cut(total.pages)
                    : tid == 2 ? cut(total.taken)
                    : tid == 3 ? (status == FI_OK ? int32_t(head + total.taken) : head)
                    : tid == 4 ? status
                               : 0;
  }
  const int64_t threads = int64_t(gridDim.x) * kTableThreads, gtid = int64_t(blockIdx.x) * kTableThreads + tid;
  if (status != FI_OK) {
    // the last step's slots must not stand: the append behind this call would
    // write this step's keys and values over that step's
    for (int64_t t = gtid; t < a.max_tokens; t += threads) {
      a.positions[t] = 0;
      a.slots[t] = -1;
    }
    return;
  }
  {
    int32_t qo = int32_t(before.qo + inc.qo - mine.qo), kv = int32_t(before.pages + inc.pages - mine.pages),
            nw = int32_t(before.taken + inc.taken - mine.taken);
    for (int b = b0; b < b1; ++b) {
      const int i = gap(b);
      const int32_t q = s_qo[i], k = s_kv[i], n = s_new[i];
      s_qo[i] = qo;
      s_kv[i] = kv;
      s_new[i] = nw;
      qo += q;
      kv += k;
      nw += n;
    }
    if (tid == 0) {
      s_qo[gap(B)] = int32_t(total.qo);
      s_kv[gap(B)] = int32_t(total.pages);
      s_new[gap(B)] = int32_t(total.taken);
    }
  }
  __syncthreads();
  for (int64_t b = gtid; b <= B; b += threads) {
    a.qo_indptr[b] = s_qo[gap(int(b))];
    a.kv_indptr[b] = s_kv[gap(int(b))];
    if (b < B) {
      const int32_t len = __ldg(a.kv_lens + b);
      a.last_page_len[b] = len > 0 ? ((len - 1) & (P - 1)) + 1 : 0;
    }
  }
  // Page p of request b: in the table already, or the free list's (the blocks
  // that need a new page's id read the list, not one another's table writes).
  // had: the pages the request had before.
  auto had_of = [&](int b) {
    return (s_kv[gap(b + 1)] - s_kv[gap(b)]) - (s_new[gap(b + 1)] - s_new[gap(b)]);
  };
  auto page_id = [&](int b, int p, int had) {
    return p < had ? a.table[b * a.table_stride + p] : __ldg(a.free_pages + head + s_new[gap(b)] + (p - had));
  };
  // A warp takes a run of entries: one search for the first, a walk from there
  // (short, but for requests without pages in between).  It goes 32 *
  // kTableAhead entries at a time, whose loads go out before the first store.
  constexpr int kSpan = 32 * kTableAhead;
  const int64_t warps = threads >> 5, run = (total.pages + warps * kSpan - 1) / (warps * kSpan) * kSpan;
  const int64_t first = (gtid >> 5) * run, last = min(total.pages, first + run);
  int b = first < last ? find(s_kv, B, int(first)) : 0;
  for (int64_t w0 = first; w0 < last; w0 += kSpan) {
    int32_t id[kTableAhead];
    int32_t* slot[kTableAhead];  // of a new page in the table
#pragma unroll
    for (int u = 0; u < kTableAhead; ++u) {
      const int64_t e = w0 + 32 * u + lane;
      slot[u] = nullptr;
      if (e >= total.pages) continue;
      while (int(e) >= s_kv[gap(b + 1)]) ++b;
      const int p = int(e) - s_kv[gap(b)], had = had_of(b);
      id[u] = page_id(b, p, had);
      if (p >= had) slot[u] = a.table + b * a.table_stride + p;
    }
#pragma unroll
    for (int u = 0; u < kTableAhead; ++u) {
      const int64_t e = w0 + 32 * u + lane;
      if (e >= total.pages) continue;
      a.kv_indices[e] = id[u];
      if (slot[u]) *slot[u] = id[u];
    }
  }
  for (int64_t t = gtid; t < a.max_tokens; t += threads) {
    int32_t pos = 0, slot = -1;
    if (t < total.qo) {
      const int b = find(s_qo, B, int(t));
      const int32_t old = __ldg(a.kv_lens + b) - __ldg(a.qo_lens + b);
      pos = old + int32_t(t) - s_qo[gap(b)];
      const int64_t at = int64_t(page_id(b, pos >> a.log2_page, pages_of(old))) * P + (pos & (P - 1));
      slot = at >= 0 && at <= INT_MAX ? int32_t(at) : -1;
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
}

}  // namespace
}  // namespace fi

using namespace fi;

extern "C" fi_status fi_build_step_tables(const fi_step_tables_args* x, void* stream) {
  if (!x) return FI_ERR_INVALID_ARG;
  if (!x->qo_lens || !x->kv_lens || !x->block_table || !x->qo_indptr || !x->kv_indptr || !x->last_page_len ||
      !x->counts || x->batch < 1 || x->block_table_width < 1 || x->block_table_stride < x->block_table_width ||
      x->num_free < 0 || x->max_pages < 0 || x->max_tokens < 0)
    return FI_ERR_INVALID_ARG;
  if (x->block_table_width > INT32_MAX || x->num_free > INT32_MAX || x->max_pages > INT32_MAX ||
      x->max_tokens > INT32_MAX)
    return FI_ERR_INVALID_ARG;
  if ((x->num_free > 0 && (!x->free_pages || !x->free_head)) || (x->max_pages > 0 && !x->kv_indices) ||
      (x->max_tokens > 0 && (!x->positions || !x->slots)))
    return FI_ERR_INVALID_ARG;
  if (x->free_head && x->free_head >= x->counts && x->free_head < x->counts + FI_STEP_COUNTS)
    return FI_ERR_INVALID_ARG;
  const int64_t P = x->page_size;
  if (x->batch > FI_STEP_MAX_BATCH || P < 1 || P > 128 || (P & (P - 1))) return FI_ERR_UNSUPPORTED;
  uintptr_t all = 0;
  for (const int32_t* ptr : {x->qo_lens, x->kv_lens, static_cast<const int32_t*>(x->block_table), x->free_pages,
                             x->free_head, static_cast<const int32_t*>(x->qo_indptr),
                             static_cast<const int32_t*>(x->kv_indptr), static_cast<const int32_t*>(x->last_page_len),
                             static_cast<const int32_t*>(x->kv_indices), static_cast<const int32_t*>(x->positions),
                             static_cast<const int32_t*>(x->slots), static_cast<const int32_t*>(x->counts)})
    all |= reinterpret_cast<uintptr_t>(ptr);
  if (all & 3u) return FI_ERR_ALIGNMENT;
  TableParams a{x->qo_lens,       x->kv_lens,        int32_t(x->batch), 0,
                x->block_table,   x->block_table_stride, int32_t(x->block_table_width),
                x->free_pages,    int32_t(x->num_free), x->free_head,   x->qo_indptr,
                x->kv_indptr,     x->last_page_len,  x->kv_indices,     int32_t(x->max_pages),
                x->positions,     x->slots,          int32_t(x->max_tokens), x->counts};
  while ((1 << a.log2_page) < P) ++a.log2_page;
  const size_t smem = size_t(3) * (gap(a.batch) + 1) * 4;
  if (smem > kPlainSmem) {
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FI_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices || !configured[dev]) {
      if (cudaFuncSetAttribute(step_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               3 * (gap(FI_STEP_MAX_BATCH) + 1) * 4) != cudaSuccess)
        return FI_ERR_CUDA;
      if (dev >= 0 && dev < kMaxDevices) configured[dev] = true;
    }
  }
  // Enough blocks for four entries a thread, at most two per SM.
  const int64_t work = (int64_t(a.max_pages) + 3) / 4 + a.max_tokens;
  int64_t blocks = (work + kTableThreads - 1) / kTableThreads;
  blocks = blocks < 1 ? 1 : blocks > 304 ? 304 : blocks;
  step_tables_kernel<<<unsigned(blocks), kTableThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FI_OK : FI_ERR_CUDA;
}
