// Eviction from a paged cache by accumulated attention weight. Per (sequence,
// kv head): of a sequence longer than the budget stay its last `recent` rows
// and, of the others, the heaviest (of equal ones the lowest row), `budget` in
// all and in order; they are copied, with their weights, to the rows 0, 1, ..
// of the new table's pages. The old pages are only read, so pages that several
// sequences share stay whole. One kernel finds the rows, a second one copies
// them; the copy is bound by HBM.
#include <cooperative_groups.h>

#include "launch.h"
#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelect = 1024;  // threads of the selection
constexpr int kWarps = kSelect / 32;
constexpr int kKeys = 49152;   // keys of a sequence that shared memory holds; those behind are read again
constexpr int kCopy = 256;     // threads of a block that copies
constexpr int kRows = 64;      // its rows

// A weight as an unsigned number of the same order; NaN below everything.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A thread-block cluster per (kv head, sequence), a run of the rows per block: the
// rows that stay, in order. The lightest weight that stays is found by its bits,
// eight at a time from the top: a histogram of the rows that agree so far, summed
// over the cluster, and the digit in which the count is reached.
__global__ void __launch_bounds__(kSelect) select_kernel(const __grid_constant__ EvictParams p, int held) {
  extern __shared__ uint32_t keys[];  // [held]
  __shared__ int hist[2][256];        // passes take turns: a block may be a pass ahead of those that read its sums
  __shared__ int all[256];
  __shared__ int2 counted[kWarps];    // heavier rows and equal ones of each warp's run
  __shared__ int2 block_counted;      // of the block
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

  // every block of the cluster finds the same
  bool ok = n >= 0 && n <= static_cast<long long>(p.width) * p.page;
  const int kept = min(n, p.budget);
  if (ok) {
    for (int i = t; i < (n + p.page - 1) / p.page; i += kSelect) ok = ok && table[i] >= 0 && table[i] < p.n_pages;
    for (int i = t; i < (kept + p.page - 1) / p.page; i += kSelect) ok = ok && fresh[i] >= 0 && fresh[i] < p.n_pages;
  }
  ok = __syncthreads_and(ok);
  if (g == 0 && rank == 0 && t == 0) p.new_lengths[b] = ok ? kept : -1;
  if (!ok) return;
  const int first = rank * kSelect + t, step = blocks * kSelect;
  if (n <= p.budget) {
    for (int i = first; i < n; i += step) rows[i] = i;
    return;
  }
  const int others = n - p.recent, want = p.budget - p.recent;  // 0 <= want < others
  for (int i = first; i < p.recent; i += step) rows[want + i] = others + i;
  if (want == 0) return;

  auto read = [&](int row) {
    const int pi = row / p.page;
    return order_of(p.key_weights[(static_cast<long long>(table[pi]) * p.nkv + g) * p.page + (row - pi * p.page)]);
  };
  // the block's run [b0, b0 + mine) of the rows
  const int share = (others + blocks - 1) / blocks, b0 = min(rank * share, others), mine = min(share, others - b0);
  const int in_smem = min(mine, held);
#pragma unroll 8
  for (int i = t; i < in_smem; i += kSelect) keys[i] = read(b0 + i);
  auto key_of = [&](int i) { return i < in_smem ? keys[i] : read(b0 + i); };

  uint32_t least = 0;  // the weight of the last one that stays, and how many equal ones do
  int equal = want, pass = 0;
  for (int shift = 24; shift >= 0; shift -= 8, ++pass) {
    int* h = hist[pass & 1];
    if (t < 256) h[t] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = t; i < mine; i += kSelect) {
      const uint32_t k = key_of(i);
      if (shift == 24 || (k ^ least) >> (shift + 8) == 0) atomicAdd(&h[k >> shift & 255], 1);
    }
    cluster.sync();
    if (t < 256) {
      int sum = 0;
      for (int r = 0; r < blocks; ++r) sum += cluster.map_shared_rank(h, r)[t];
      all[t] = sum;
    }
    __syncthreads();
    if (warp == 0) {  // lane: eight digits, from the highest on
      int x[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += x[j] = all[255 - 8 * lane - j];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      before -= sum;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (before < equal && before + x[j] >= equal) digit = 255 - 8 * lane - j, above = before;
        before += x[j];
      }
    }
    __syncthreads();
    least |= static_cast<uint32_t>(digit) << shift;
    equal -= above;
  }

  // a warp's run of the block's rows: how many stay before it, then each row's place
  const int run = (mine + kSelect - 1) / kSelect * 32, r0 = min(warp * run, mine), r1 = min(r0 + run, mine);
  int heavier = 0, ties = 0;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < r1 ? key_of(i) : 0;
    heavier += __popc(__ballot_sync(0xffffffffu, i < r1 && k > least));
    ties += __popc(__ballot_sync(0xffffffffu, i < r1 && k == least));
  }
  if (lane == 0) counted[warp] = make_int2(heavier, ties);
  __syncthreads();
  if (warp == 0) {
    int2 c = counted[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c.x += __shfl_xor_sync(0xffffffffu, c.x, o), c.y += __shfl_xor_sync(0xffffffffu, c.y, o);
    if (lane == 0) block_counted = c;
  }
  cluster.sync();
  int at = 0, tie = 0;
  auto pass_by = [&](int2 c) {
    at += c.x + max(0, min(c.y, equal - tie));
    tie += c.y;
  };
  for (int r = 0; r < rank; ++r) pass_by(*cluster.map_shared_rank(&block_counted, r));
  for (int w = 0; w < warp; ++w) pass_by(counted[w]);
  const unsigned below = (1u << lane) - 1;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < r1 ? key_of(i) : 0;
    const unsigned same = __ballot_sync(0xffffffffu, i < r1 && k == least);
    const bool stays = i < r1 && (k > least || (k == least && tie + __popc(same & below) < equal));
    const unsigned stay = __ballot_sync(0xffffffffu, stays);
    if (stays) rows[at + __popc(stay & below)] = b0 + i;
    at += __popc(stay);
    tie += __popc(same);
  }
  cluster.sync();  // the counts are read before their block ends
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
  static std::atomic<uint64_t> told;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess) e = allow_smem(select_kernel, kKeys * 4, told);
  if (e != cudaSuccess) return e;
  // a head's rows are shared out over as many blocks as the SMs have room for one by
  // one, while each has a few thousand rows
  const long long most = static_cast<long long>(p.width) * p.page, heads = static_cast<long long>(p.nkv) * p.batch;
  int blocks_of_head = 1;
  while (blocks_of_head < 8 && 2 * blocks_of_head * heads <= sms && most >= 2048ll * blocks_of_head) blocks_of_head *= 2;
  const long long share = (most + blocks_of_head - 1) / blocks_of_head;
  const int held = static_cast<int>(share < kKeys ? share : kKeys);
  e = launch_early_clusters(select_kernel, dim3(blocks_of_head, p.nkv, p.batch), kSelect, held * 4, blocks_of_head, s, p, held);
  if (e != cudaSuccess) return e;
  const int blocks = (p.budget + kRows - 1) / kRows;
  const dim3 grid(blocks < 4096 ? blocks : 4096, p.nkv, p.batch);
  return p.chunks == 16 ? launch_early(copy_kernel<16>, grid, kCopy, 0, s, p) : launch_early(copy_kernel<8>, grid, kCopy, 0, s, p);
}

}  // namespace lps
