// Row moves of a caller-owned cache: packed key and value rows to their cache
// rows (append), and the accepted path of a drafted tree to consecutive rows
// (accept). Both only move bytes, so both are bound by HBM when they are large
// and by the launch when they are small.
#include "cache_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

constexpr int kThreads = 256;

// Block = kTokens consecutive tokens and kThreads of a token's 16-byte units;
// thread = one unit (kv head, column) of its token, of K and of V, for every
// kWays-th of the block's tokens. All its loads are issued before its stores.
// 12185 tokens of 8 heads of 128 (100 MB read and written) take 16.0 us, 6.2
// TB/s; a thread a unit with a 64-bit division each took 17.8.
template <int UNITS>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  pdl_launch_dependents();
  constexpr int kLanes = UNITS < kThreads ? UNITS : kThreads;  // threads of one token
  constexpr int kWays = kThreads / kLanes, kEach = 4;
  const int units = p.nkv * p.chunks;
  const int u = blockIdx.y * kLanes + threadIdx.x % kLanes;
  if (u >= units) return;
  const int g = u / p.chunks, c = u - g * p.chunks;
  const int end = p.off[p.n_seqs];  // far enough below 2^31 for the last block's tokens
  const int tok0 = p.off[0] + static_cast<int>(blockIdx.x) * (kWays * kEach) + static_cast<int>(threadIdx.x) / kLanes;
  uint4 k[kEach], v[kEach];
  size_t dst[kEach];
  pdl_wait();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int tok = tok0 + i * kWays;
    if (tok < end) {
      k[i] = p.k[tok * p.k_tok + g * p.k_head + c];
      v[i] = p.v[tok * p.v_tok + g * p.v_head + c];
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int tok = tok0 + i * kWays;
    int lo = 0, hi = p.n_seqs - 1;  // the sequence that holds the token: the last s with off[s] <= tok
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.off[mid] <= tok) lo = mid; else hi = mid - 1;
    }
    dst[i] = ((static_cast<size_t>(lo) * p.nkv + g) * p.max_ctx + p.start[lo] + tok - p.off[lo]) * p.chunks + c;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (tok0 + i * kWays < end) {
      p.kc[dst[i]] = k[i];
      p.vc[dst[i]] = v[i];
    }
}

// Block = one (sequence, layer, K or V) and kThreads 16-byte columns of its
// rows; a thread walks its column down the path, kAhead rows read before they
// are written (one after the other, 16 rows took 5.3 us). The path is strictly
// ascending, so path[i] >= i: a row is read before any row at or after it is
// written, and the move is safe in place. A path that breaks its rules moves
// nothing.
constexpr int kAhead = 8;
__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ AcceptParams p) {
  __shared__ int path[kTreeMax];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x, l = blockIdx.y >> 1;
  const int t = threadIdx.x;
  const int n = p.accepted[b], pos = p.pos[b];
  // read without waiting for n: the path has width entries whatever n is
  const int x = t < p.width ? p.path[static_cast<size_t>(b) * p.width + t] : 0;
  const int before = t > 0 && t < p.width ? p.path[static_cast<size_t>(b) * p.width + t - 1] : -1;
  if (t < p.width) path[t] = x;
  const bool ok = n >= 0 && n <= p.width && (t >= n || (x > before && x < p.width && x < p.max_ctx - pos));
  if (!__syncthreads_and(ok)) return;
  uint4* cache = (blockIdx.y & 1 ? p.vc : p.kc) + (static_cast<size_t>(l) * p.batch + b) * p.nkv * p.max_ctx * p.chunks;
  const int u = blockIdx.z * kThreads + t;
  if (u >= p.nkv * p.chunks) return;
  const int g = u / p.chunks, c = u - g * p.chunks;
  uint4* col = cache + (static_cast<size_t>(g) * p.max_ctx + pos) * p.chunks + c;
  for (int i = 0; i < n; i += kAhead) {
    uint4 row[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (i + e < n) row[e] = col[static_cast<size_t>(path[i + e]) * p.chunks];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (i + e < n) col[static_cast<size_t>(i + e) * p.chunks] = row[e];
  }
}

// Launched so that its start runs under the stream's last kernel; the kernels
// touch global memory behind the dependency wait.
template <class Kern, class Params>
cudaError_t launch(Kern kern, dim3 grid, const Params& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int UNITS>
cudaError_t launch_append_t(const AppendParams& p, cudaStream_t s) {
  constexpr int kLanes = UNITS < kThreads ? UNITS : kThreads;
  constexpr int kTokens = kThreads / kLanes * 4;
  const int tokens = p.off[p.n_seqs] - p.off[0];
  const int units = p.nkv * p.chunks;
  return launch(append_kernel<UNITS>,
                dim3(static_cast<unsigned>((static_cast<long long>(tokens) + kTokens - 1) / kTokens), (units + kLanes - 1) / kLanes),
                p, s);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  if (p.off[p.n_seqs] == p.off[0]) return cudaSuccess;
  // the threads of a token: the smallest power of two that holds its units, so
  // that narrow rows do not leave lanes idle
  const int units = p.nkv * p.chunks;
  if (units <= 8) return launch_append_t<8>(p, s);
  if (units <= 16) return launch_append_t<16>(p, s);
  if (units <= 32) return launch_append_t<32>(p, s);
  if (units <= 64) return launch_append_t<64>(p, s);
  if (units <= 128) return launch_append_t<128>(p, s);
  return launch_append_t<256>(p, s);
}

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s) {
  const int units = p.nkv * p.chunks;
  return launch(accept_kernel, dim3(p.batch, 2 * p.layers, (units + kThreads - 1) / kThreads), p, s);
}

}  // namespace lps
