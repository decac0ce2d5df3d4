// Row moves of a caller-owned cache: packed key and value rows to their cache
// rows (append), and the accepted path of a drafted tree to consecutive rows
// (accept). Both only move bytes, so both are bound by HBM when they are large
// and by the launch when they are small.
#include "cache_ops.h"

namespace lps {
namespace {

constexpr int kThreads = 256;

// Thread = one 16-byte unit of one token's K row and of its V row.
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  const long long per_tok = static_cast<long long>(p.nkv) * p.chunks;
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long n = (p.off[p.n_seqs] - p.off[0]) * per_tok;
  if (i >= n) return;
  const int tok = p.off[0] + static_cast<int>(i / per_tok);
  const int r = static_cast<int>(i % per_tok);
  const int g = r / p.chunks, c = r - g * p.chunks;
  int lo = 0, hi = p.n_seqs - 1;  // the sequence that holds the token: the last s with off[s] <= tok
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.off[mid] <= tok) lo = mid; else hi = mid - 1;
  }
  const int row = p.start[lo] + tok - p.off[lo];
  const size_t dst = ((static_cast<size_t>(lo) * p.nkv + g) * p.max_ctx + row) * p.chunks + c;
  p.kc[dst] = p.k[tok * p.k_tok + g * p.k_head + c];
  p.vc[dst] = p.v[tok * p.v_tok + g * p.v_head + c];
}

// Block = one (sequence, layer, K or V); thread = one 16-byte column of one kv
// head, walked down the path in order. The path is strictly ascending, so
// path[i] >= i: a row is read before any row at or after it is written, and
// the move is safe in place. A path that breaks its rules moves nothing.
__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ AcceptParams p) {
  __shared__ int path[kTreeMax];
  const int b = blockIdx.x, l = blockIdx.y;
  const int n = p.accepted[b], pos = p.pos[b];
  bool ok = n >= 0 && n <= p.width;
  if (ok && static_cast<int>(threadIdx.x) < n) {
    const int t = threadIdx.x;
    const int x = p.path[static_cast<size_t>(b) * p.width + t];
    const int before = t ? p.path[static_cast<size_t>(b) * p.width + t - 1] : -1;
    ok = x > before && x < p.width && x < p.max_ctx - pos;
    path[t] = x;
  }
  if (!__syncthreads_and(ok)) return;
  uint4* cache = (blockIdx.z ? p.vc : p.kc) + (static_cast<size_t>(l) * p.batch + b) * p.nkv * p.max_ctx * p.chunks;
  for (int u = threadIdx.x; u < p.nkv * p.chunks; u += kThreads) {
    const int g = u / p.chunks, c = u - g * p.chunks;
    uint4* col = cache + (static_cast<size_t>(g) * p.max_ctx + pos) * p.chunks + c;
    for (int i = 0; i < n; ++i) col[static_cast<size_t>(i) * p.chunks] = col[static_cast<size_t>(path[i]) * p.chunks];
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  const long long n = static_cast<long long>(p.off[p.n_seqs] - p.off[0]) * p.nkv * p.chunks;
  if (n == 0) return cudaSuccess;
  append_kernel<<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s) {
  accept_kernel<<<dim3(p.batch, p.layers, 2), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace lps
