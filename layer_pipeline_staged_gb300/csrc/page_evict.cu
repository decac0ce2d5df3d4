// Eviction from a paged cache by accumulated attention weight. Per (sequence,
// kv head): of a sequence longer than the budget stay its last `recent` rows
// and, of the others, the heaviest (of equal ones the lowest row), `budget` in
// all and in order; they are copied, with their weights, to the rows 0, 1, ..
// of the new table's pages. The old pages are only read, so pages that several
// sequences share stay whole.
#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

constexpr int kSelect = 1024;  // threads of the selection
constexpr int kWarps = kSelect / 32;

// A weight as an unsigned number of the same order; NaN below everything.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix of x over the block and the block's sum.
__device__ __forceinline__ int block_prefix(int x, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = all;
    all += sums[w];
  }
  *total = all;
  return before + incl - x;
}

// Block = (kv head, sequence): the rows that stay, in order. The lightest weight
// that stays is found by its bits, eight at a time from the top: a histogram of
// the rows that agree so far, and the digit in which the count is reached.
__global__ void __launch_bounds__(kSelect) select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int hist[256], sums[kWarps];
  __shared__ int digit, above;
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x, g = blockIdx.x, b = blockIdx.y;
  const int n = p.lengths[b];
  const int* table = p.table + static_cast<long long>(b) * p.width;
  const int* fresh = p.fresh + static_cast<long long>(b) * p.fresh_width;
  int* rows = p.rows + (static_cast<long long>(b) * p.nkv + g) * p.budget;

  bool ok = n >= 0 && n <= static_cast<long long>(p.width) * p.page;
  const int kept = min(n, p.budget);
  if (ok) {
    for (int i = t; i < (n + p.page - 1) / p.page; i += kSelect) ok = ok && table[i] >= 0 && table[i] < p.n_pages;
    for (int i = t; i < (kept + p.page - 1) / p.page; i += kSelect) ok = ok && fresh[i] >= 0 && fresh[i] < p.n_pages;
  }
  ok = __syncthreads_and(ok);
  if (g == 0 && t == 0) p.new_lengths[b] = ok ? kept : -1;
  if (!ok) return;
  if (n <= p.budget) {
    for (int i = t; i < n; i += kSelect) rows[i] = i;
    return;
  }
  const int others = n - p.recent, want = p.budget - p.recent;  // 0 <= want < others
  auto key_of = [&](int row) {
    const int pi = row / p.page;
    return order_of(p.key_weights[(static_cast<long long>(table[pi]) * p.nkv + g) * p.page + (row - pi * p.page)]);
  };
  uint32_t least = 0;     // the weight of the last one that stays, and how many equal ones do
  int equal = want;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (t < 256) hist[t] = 0;
      __syncthreads();
      for (int i = t; i < others; i += kSelect) {
        const uint32_t k = key_of(i);
        if (shift == 24 || (k ^ least) >> (shift + 8) == 0) atomicAdd(&hist[k >> shift & 255], 1);
      }
      __syncthreads();
      // thread d: how many have a higher digit
      int x = t < 256 ? hist[255 - t] : 0, all;
      const int before = block_prefix(x, sums, &all);
      if (t < 256 && before < equal && before + x >= equal) digit = 255 - t, above = before;
      __syncthreads();
      least |= static_cast<uint32_t>(digit) << shift;
      equal -= above;
      __syncthreads();
    }
  }
  // in order: a row's place is the number that stay before it
  int done = 0, ties = 0;
  for (int i0 = 0; i0 < others; i0 += kSelect) {
    const int i = i0 + t;
    const uint32_t k = want > 0 && i < others ? key_of(i) : 0;
    const bool in = want > 0 && i < others, tie = in && k == least;
    int all_ties, all;
    const int tie_no = ties + block_prefix(tie, sums, &all_ties);
    const bool stays = in && (k > least || (tie && tie_no < equal));
    const int at = done + block_prefix(stays, sums, &all);
    if (stays) rows[at] = i;
    ties += all_ties;
    done += all;
  }
  for (int i = t; i < p.recent; i += kSelect) rows[want + i] = others + i;
}

// Thread = a 16-byte unit of a row of K and of V.
__global__ void __launch_bounds__(256) copy_kernel(const __grid_constant__ EvictParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int g = blockIdx.y, b = blockIdx.z;
  const int n = p.new_lengths[b];
  const int per = 256 / p.chunks, c = threadIdx.x % p.chunks;
  const int* table = p.table + static_cast<long long>(b) * p.width;
  const int* fresh = p.fresh + static_cast<long long>(b) * p.fresh_width;
  const int* rows = p.rows + (static_cast<long long>(b) * p.nkv + g) * p.budget;
  for (long long i = static_cast<long long>(blockIdx.x) * per + threadIdx.x / p.chunks; i < n; i += static_cast<long long>(gridDim.x) * per) {
    const int to = static_cast<int>(i), from = rows[to];
    const int pf = from / p.page, pt = to / p.page;
    const long long src = (static_cast<long long>(table[pf]) * p.nkv + g) * p.page + (from - pf * p.page);
    const long long dst = (static_cast<long long>(fresh[pt]) * p.nkv + g) * p.page + (to - pt * p.page);
    const uint4 k = p.k_pages[src * p.chunks + c], v = p.v_pages[src * p.chunks + c];
    p.k_pages[dst * p.chunks + c] = k;
    p.v_pages[dst * p.chunks + c] = v;
    if (c == 0) p.key_weights[dst] = p.key_weights[src];
  }
}

template <class Kern>
cudaError_t launch(Kern kern, dim3 grid, int threads, const EvictParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  cudaError_t e = launch(select_kernel, dim3(p.nkv, p.batch), kSelect, p, s);
  if (e != cudaSuccess) return e;
  const int per = 256 / p.chunks;
  const int blocks = (p.budget + per - 1) / per;
  return launch(copy_kernel, dim3(blocks < 4096 ? blocks : 4096, p.nkv, p.batch), 256, p, s);
}

}  // namespace lps
