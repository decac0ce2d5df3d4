// Eviction from a paged cache by accumulated attention weight. Per (sequence,
// kv head): of a sequence longer than the budget stay its last `recent` rows
// and, of the others, the heaviest (of equal ones the lowest row), `budget` in
// all and in order; they are copied, with their weights, to the rows 0, 1, ..
// of the new table's pages. The old pages are only read, so pages that several
// sequences share stay whole. One kernel finds the rows, a second one copies
// them. 8 sequences of up to 8192 rows, 8 heads of 128, brought to 4096: 48.0 us, of
// which the copy is 37 (6.5 TB/s) and the selection, bound by latency, the rest.
#include <cooperative_groups.h>

#include "launch.h"
#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelect = 1024;  // threads of the selection
constexpr int kWarps = kSelect / 32;
constexpr int kBins = 2048;
constexpr int kKeys = 32768;   // weights that a block of the selection keeps
constexpr int kCopy = 256;     // threads of a block that copies
constexpr int kRows = 64;      // its rows

// A weight as an unsigned number of the same order; NaN below everything.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A thread-block cluster per (kv head, sequence), a run of the rows per block: the rows
// that stay, in order. The lightest weight that stays is found by its bits from the
// top, 11, 11 and 10: a histogram of the rows that agree so far, summed over the
// cluster, and the digit in which the count is reached (counting the rows at or above
// candidates, two bits a round, takes 16 rounds of two barriers: 13 us instead of 6).
// Latency bounds it, and not least the instructions' own way from memory: its loops
// stay loops (unrolled, with the weights in registers, 1000 rows of 8 heads took 11.3 us
// with the copy, and 8.2 to 8.8 so).
__global__ void __launch_bounds__(kSelect) select_kernel(const __grid_constant__ EvictParams p, int held) {
  extern __shared__ uint4 held_keys[];  // [held / 4]: the orders of the block's first rows; those behind are read again
  uint32_t* keys = reinterpret_cast<uint32_t*>(held_keys);
  __shared__ __align__(16) int hist[3][kBins];
  __shared__ int sums[kWarps];
  __shared__ int2 block_counted;      // the block's heavier rows and equal ones
  __shared__ int digit, above;
  pdl_launch_dependents();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rank = cluster.block_rank(), blocks = cluster.num_blocks(), g = blockIdx.y, b = blockIdx.z;
  const int n = p.lengths[b];
  const int* table = p.table + static_cast<long long>(b) * p.width;
  const int* fresh = p.fresh + static_cast<long long>(b) * p.fresh_width;
  int* rows = p.rows + (static_cast<long long>(b) * p.nkv + g) * p.budget;
  auto meet = [&] {
    if (blocks > 1) cluster.sync();
    else __syncthreads();
  };
  for (int i = t; i < static_cast<int>(sizeof hist) / 16; i += kSelect) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);

  bool ok = n >= 0 && n <= static_cast<long long>(p.width) * p.page;
  const int kept = min(n, p.budget);
  const bool choose = ok && n > p.budget;
  const int others = choose ? n - p.recent : 0, want = p.budget - p.recent;  // 0 <= want < others
  // the block's run [b0, b0 + mine) of the rows
  const int share = (others + 8 * blocks - 1) / (8 * blocks) * 8, b0 = min(rank * share, others), mine = min(share, others - b0);
  // A page's rows come in eights, and so do the block's: a thread takes eight of one
  // page. A row on a page that is none is as light as can be, as is what fills an eight.
  const int in_smem = min(mine, held);
  // the first pages to be looked at are asked for before the weights
  const int pages = ok ? (n + p.page - 1) / p.page : 0, fresh_pages = ok ? (kept + p.page - 1) / p.page : 0;
  const int page0 = t < pages ? table[t] : 0, fresh0 = t < fresh_pages ? fresh[t] : 0;
  __syncthreads();
#pragma unroll 2
  for (int i = 8 * t; i < in_smem; i += 8 * kSelect) {
    const int pi = (b0 + i) / p.page, page = table[pi];
    float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), y = x;
    if (page >= 0 && page < p.n_pages) {
      const float4* w = reinterpret_cast<const float4*>(p.key_weights + (static_cast<long long>(page) * p.nkv + g) * p.page + (b0 + i - pi * p.page));
      x = w[0], y = w[1];
    }
    uint4 k = make_uint4(order_of(x.x), order_of(x.y), order_of(x.z), order_of(x.w));
    uint4 l = make_uint4(order_of(y.x), order_of(y.y), order_of(y.z), order_of(y.w));
    const int left = in_smem - i;
    if (left < 8) {
      l.w = 0, l.z = left > 6 ? l.z : 0, l.y = left > 5 ? l.y : 0, l.x = left > 4 ? l.x : 0;
      k.w = left > 3 ? k.w : 0, k.z = left > 2 ? k.z : 0, k.y = left > 1 ? k.y : 0;
    }
    held_keys[i / 4] = k, held_keys[i / 4 + 1] = l;
    // the first digit is counted on the way (what fills an eight goes to the lowest bin: above it are only rows)
    atomicAdd(&hist[0][k.x >> 21], 1), atomicAdd(&hist[0][k.y >> 21], 1), atomicAdd(&hist[0][k.z >> 21], 1), atomicAdd(&hist[0][k.w >> 21], 1);
    atomicAdd(&hist[0][l.x >> 21], 1), atomicAdd(&hist[0][l.y >> 21], 1), atomicAdd(&hist[0][l.z >> 21], 1), atomicAdd(&hist[0][l.w >> 21], 1);
  }
  auto read = [&](int i) {
    const int row = b0 + i, pi = row / p.page, page = table[pi];
    return order_of(p.key_weights[(static_cast<long long>(page) * p.nkv + g) * p.page + (row - pi * p.page)]);
  };
  // every block of the cluster looks at all pages, and finds the same
  ok = ok && page0 >= 0 && page0 < p.n_pages && fresh0 >= 0 && fresh0 < p.n_pages;
  for (int i = t + kSelect; i < pages; i += kSelect) ok = ok && table[i] >= 0 && table[i] < p.n_pages;
  for (int i = t + kSelect; i < fresh_pages; i += kSelect) ok = ok && fresh[i] >= 0 && fresh[i] < p.n_pages;
  ok = __syncthreads_and(ok);
  if (g == 0 && rank == 0 && t == 0) p.new_lengths[b] = ok ? kept : -1;
  if (!ok) return;
  const int first = rank * kSelect + t, step = blocks * kSelect;
  if (!choose) {
    for (int i = first; i < n; i += step) rows[i] = i;
    return;
  }
  for (int i = first; i < p.recent; i += step) rows[want + i] = others + i;
  if (want == 0) return;
  auto key_of = [&](int i) { return i < in_smem ? keys[i] : read(i); };

  uint32_t least = 0;  // the weight of the last one that stays, and how many equal ones do
  int equal = want;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = max(21 - 11 * pass, 0);
    const uint32_t bins = pass == 2 ? 1023 : kBins - 1, known = pass == 0 ? 0 : ~0u << (pass == 1 ? 21 : 10);  // bits that agree
    int* h = hist[pass];
    auto count = [&](uint32_t k) {
      if ((k & known) == least) atomicAdd(&h[k >> shift & bins], 1);
    };
#pragma unroll 1
    for (int i = pass ? t : in_smem; i < (in_smem + 3) / 4; i += kSelect) {
      const uint4 k = held_keys[i];
      count(k.x), count(k.y), count(k.z), count(k.w);
    }
#pragma unroll 1
    for (int i = held + t; i < mine; i += kSelect) count(read(i));
    meet();
    // thread: two bins, from the highest on
    int2 x = make_int2(0, 0);
    for (int r = 0; r < blocks; ++r) {
      const int2 v = reinterpret_cast<const int2*>(blocks > 1 ? cluster.map_shared_rank(h, r) : h)[kSelect - 1 - t];
      x.x += v.y, x.y += v.x;
    }
    int before = x.x + x.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    if (lane == 31) sums[warp] = before;
    __syncthreads();
    before += __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0) - x.x - x.y;
    if (before < equal && before + x.x >= equal) digit = kBins - 1 - 2 * t, above = before;
    before += x.x;
    if (before < equal && before + x.y >= equal) digit = kBins - 2 - 2 * t, above = before;
    __syncthreads();
    least |= static_cast<uint32_t>(digit) << shift;
    equal -= above;
  }

  // the heavier rows and the equal ones before the block's, for a block that is not the first
  int heavy = 0, tie = 0;
  if (blocks > 1) {
    int x = 0, y = 0;
#pragma unroll 1
    for (int i = t; i < mine; i += kSelect) {
      const uint32_t k = key_of(i);
      x += k > least, y += k == least;
    }
    x = __reduce_add_sync(0xffffffffu, x), y = __reduce_add_sync(0xffffffffu, y);
    if (t == 0) block_counted = make_int2(0, 0);
    __syncthreads();
    if (lane == 0) atomicAdd(&block_counted.x, x), atomicAdd(&block_counted.y, y);
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
      const int2 o = *cluster.map_shared_rank(&block_counted, r);
      heavy += o.x, tie += o.y;
    }
  }
  // Each row's place, a thread eight rows in turn: heavier rows in the lower half of a
  // sum and equal ones in the upper, at most 8192 of each
#pragma unroll 1
  for (int c0 = 0; c0 < mine; c0 += 8 * kSelect) {
    const int i0 = c0 + 8 * t;
    uint32_t more = 0, same = 0;  // a bit a row
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t k = i0 + e < mine ? key_of(i0 + e) : 0;
      more |= static_cast<uint32_t>(i0 + e < mine && k > least) << e;
      same |= static_cast<uint32_t>(i0 + e < mine && k == least) << e;
    }
    const int packed = __popc(more) | __popc(same) << 16;
    int before = packed;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    __syncthreads();  // the last sums have been read
    if (lane == 31) sums[warp] = before;
    __syncthreads();
    const int all = sums[lane];
    before += static_cast<int>(__reduce_add_sync(0xffffffffu, lane < warp ? all : 0)) - packed;
    int at_tie = tie + (before >> 16), at = heavy + (before & 0xffff) + min(at_tie, equal);  // of equal ones the first stay
    for (uint32_t left = more | same; left; left &= left - 1) {
      const int e = __ffs(left) - 1;
      if (more >> e & 1 || at_tie++ < equal) rows[at++] = b0 + i0 + e;
    }
    const int total = __reduce_add_sync(0xffffffffu, all);
    heavy += total & 0xffff, tie += total >> 16;
  }
  if (blocks > 1) cluster.sync();  // the counts are read before their block ends
}

// Block = kRows kept rows of (kv head, sequence): where they come from and go to,
// once a row; then a thread has all its 16-byte units of K and V on their way
// before it stores the first.
template <int CHUNKS>
__global__ void __launch_bounds__(kCopy) copy_kernel(const __grid_constant__ EvictParams p) {
  __shared__ long long src[kRows], dst[kRows];  // rows of the pools
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int n = p.new_lengths[b];
  constexpr int kEach = kRows * CHUNKS / kCopy;
  for (long long lot = static_cast<long long>(blockIdx.x) * kRows; lot < n; lot += static_cast<long long>(gridDim.x) * kRows) {
    const int row0 = static_cast<int>(lot), rows = min(kRows, n - row0);
    if (t < rows) {
      const int to = row0 + t, from = p.rows[(static_cast<long long>(b) * p.nkv + g) * p.budget + to];
      const int pf = from / p.page, pt = to / p.page;
      const long long s = (static_cast<long long>(p.table[static_cast<long long>(b) * p.width + pf]) * p.nkv + g) * p.page + (from - pf * p.page);
      const long long d = (static_cast<long long>(p.fresh[static_cast<long long>(b) * p.fresh_width + pt]) * p.nkv + g) * p.page + (to - pt * p.page);
      src[t] = s, dst[t] = d;
      p.key_weights[d] = p.key_weights[s];
    }
    __syncthreads();
    uint4 k[kEach], v[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int r = (i * kCopy + t) / CHUNKS, c = t % CHUNKS;
      if (r < rows) k[i] = p.k_pages[src[r] * CHUNKS + c], v[i] = p.v_pages[src[r] * CHUNKS + c];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int r = (i * kCopy + t) / CHUNKS, c = t % CHUNKS;
      if (r < rows) p.k_pages[dst[r] * CHUNKS + c] = k[i], p.v_pages[dst[r] * CHUNKS + c] = v[i];
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  static std::atomic<uint64_t> told;
  if (e == cudaSuccess) e = allow_smem(select_kernel, kKeys * 4, told);
  if (e != cudaSuccess) return e;
  // A head's rows are one block's, or shared out over two, four or eight. us for caches
  // just as long as their tables, brought to 1024 rows, heads of 128 (a block holds 32768):
  //                                 1      2      4      8
  //   8 heads, 16384 rows        13.7   14.5   14.6   17.9
  //   8 heads, 20000 rows        15.8   17.0   15.1   18.3
  //   8 heads, 28672 rows        18.9   17.6   15.8   18.6
  //   8 heads, 65536 rows               26.1   20.4   20.6
  //   8 heads, 131072 rows                     28.3   25.1
  //   32 heads, 24576 rows       19.5   19.9   18.8   51.8
  //   72 heads, 24576 rows       24.6   25.2   35.7   91.2
  //   72 heads, 32768 rows       28.6   26.8   37.6   93.1
  //   120 heads, 40000 rows             59.1   86.8  160.2
  // A larger cluster pays where every block has a place at once and the rows are many;
  // but no block has more rows than it holds, if eight are enough for that.
  const long long most = static_cast<long long>(p.width) * p.page, heads = static_cast<long long>(p.nkv) * p.batch;
  int blocks_of_head = 1;
  if (most >= 28672 && 2 * heads <= sms) blocks_of_head = 2;
  if (most >= 20000 && 4 * heads <= sms) blocks_of_head = 4;
  if (most >= 65536 && 8 * heads <= sms) blocks_of_head = 8;
  while (blocks_of_head < 8 && most > static_cast<long long>(kKeys) * blocks_of_head) blocks_of_head *= 2;
  const long long share = (most + blocks_of_head - 1) / blocks_of_head;
  const int held = static_cast<int>(share + 8 < kKeys ? (share + 15) / 8 * 8 : kKeys);  // a share is in eights
  e = launch_early_clusters(select_kernel, dim3(blocks_of_head, p.nkv, p.batch), kSelect, held * 4, blocks_of_head, s, p, held);
  if (e != cudaSuccess) return e;
  const int blocks = (p.budget + kRows - 1) / kRows;
  const dim3 grid(blocks < 4096 ? blocks : 4096, p.nkv, p.batch);
  return p.chunks == 16 ? launch_early(copy_kernel<16>, grid, kCopy, 0, s, p) : launch_early(copy_kernel<8>, grid, kCopy, 0, s, p);
}

}  // namespace lps
