// Attention of packed prompts (causal) and of drafted trees over a cache.
// One warp per (token, query head): the lanes share the head dimension, keys
// are walked in order with the running maximum and sum of the softmax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* o) { *o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half* o) { *o = __float2half_rn(x); }

// The drafted rows that row t sees, as bits; 0 for a chain that leaves its
// range (a parent outside [-1, child)).
__device__ __forceinline__ unsigned long long tree_mask(const int* parents, int t) {
  unsigned long long m = 0;
  while (t >= 0) {
    m |= 1ull << t;
    const int up = parents[t];
    if (up < -1 || up >= t) return 0;
    t = up;
  }
  return m;
}

template <class T, int HD, bool TREE>
__global__ void __launch_bounds__(kWarps * 32) tile_attn_kernel(const __grid_constant__ TileAttnParams p) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.z, h = blockIdx.y, g = h / p.group;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.len[s]) return;
  const T* q = static_cast<const T*>(p.q) + s * p.q_seq + (p.tok0[s] + t) * p.q_tok + h * p.q_head + lane * E;
  const T* k = static_cast<const T*>(p.k) + s * p.k_seq + p.tok0[s] * p.k_row + g * p.k_head + lane * E;
  const T* v = static_cast<const T*>(p.v) + s * p.v_seq + p.tok0[s] * p.v_row + g * p.v_head + lane * E;
  T* o = static_cast<T*>(p.out) + s * p.o_seq + (p.tok0[s] + t) * p.o_tok + h * p.o_head + lane * E;
  const unsigned long long tm = TREE ? tree_mask(p.parents + static_cast<size_t>(s) * p.width, t) : 0;
  const int pos = TREE ? p.pos[s] : 0;
  const int nkeys = TREE ? (tm ? pos + t + 1 : 0) : t + 1;
  float qf[E], acc[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    qf[e] = to_f(q[e]) * p.scale;
    acc[e] = 0.f;
  }
  for (int j = 0; j < nkeys; ++j) {
    if (TREE && j >= pos && !((tm >> (j - pos)) & 1)) continue;
    float x = 0.f;
    for (int e = 0; e < E; ++e) x = fmaf(qf[e], to_f(k[j * p.k_row + e]), x);
    x = warp_sum(x);
    const float mn = fmaxf(m, x);
    const float a = m == mn ? 1.f : expf(m - mn), w = expf(x - mn);
    l = fmaf(l, a, w);
    for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], a, w * to_f(v[j * p.v_row + e]));
    m = mn;
  }
  const float inv = nkeys ? 1.0f / l : 0.f;
  for (int e = 0; e < E; ++e) from_f(acc[e] * inv, o + e);
}

template <class T, int HD, bool TREE>
cudaError_t launch_t(const TileAttnParams& p, cudaStream_t s) {
  int longest = 0;
  for (int i = 0; i < p.n_seqs; ++i) longest = p.len[i] > longest ? p.len[i] : longest;
  if (longest == 0) return cudaSuccess;
  tile_attn_kernel<T, HD, TREE><<<dim3((longest + kWarps - 1) / kWarps, p.nq, p.n_seqs), kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_hd(const TileAttnParams& p, int hd, bool tree, cudaStream_t s) {
  if (hd == 128) return tree ? launch_t<T, 128, true>(p, s) : launch_t<T, 128, false>(p, s);
  return tree ? launch_t<T, 64, true>(p, s) : launch_t<T, 64, false>(p, s);
}

}  // namespace

cudaError_t launch_tile_attn(const TileAttnParams& p, bool bf16, int hd, bool tree, cudaStream_t s) {
  return bf16 ? launch_hd<__nv_bfloat16>(p, hd, tree, s) : launch_hd<__half>(p, hd, tree, s);
}

}  // namespace lps
