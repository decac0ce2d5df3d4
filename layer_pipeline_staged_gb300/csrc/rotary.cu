// Rotary positions: pair i of a head's first `rot` elements is turned by the
// angle position * freqs[i],
//     a' = mag (a cos - b sin), b' = mag (b cos + a sin),
// with (a, b) = elements (i, i + rot / 2) or (2i, 2i + 1); the other elements
// pass. The append form also writes k' and v to their rows in the pages.
//
// Angles: only the angle's fraction of a turn matters, and at position 10^5 it
// is what is left of 10^4 turns. A frequency is held as f / (2 pi) in units of
// 2^-64 turns; the product with the position in 64-bit integers drops whole
// turns exactly, and its upper half, as a signed fraction of half a turn, is
// the argument of sincospi. The error is the frequency's own rounding (2^-53
// relative) times the position, and 2^-25 turns for the argument in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;

template <bool BF16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if constexpr (BF16) return make_float2(bf16lo(w), bf16hi(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack(float x, float y) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Block = TOK consecutive tokens: their angles' cosines and sines once into
// shared memory, then an item (token, head, 16 elements) per thread.
template <bool BF16, int HD, int TOK>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  __shared__ float2 turn[TOK][kMaxPairs];  // (cos, sin) times the magnitude
  __shared__ long long row[TOK];           // page * nkv * page rows + row in the page, or -1: not stored
  __shared__ int live[TOK];
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x, pairs = p.rot >> 1;
  const int tok0 = blockIdx.x * TOK;

  // where each token goes, and what turns it
  for (int i = t; i < TOK * kMaxPairs; i += kThreads) {
    const int ti = i / kMaxPairs, pair = i % kMaxPairs, tok = tok0 + ti;
    bool on = tok < p.tokens;
    int pos = 0;
    if (p.k_pages) {
      int s = tok, left = 1;
      if (on && p.offsets) {
        on = tok >= p.offsets[0] && tok < p.offsets[p.n_seqs];
        int lo = 0, hi = p.n_seqs - 1;  // the last s with offsets[s] <= tok
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (p.offsets[mid] <= tok) lo = mid; else hi = mid - 1;
        }
        s = lo;
        left = p.offsets[s + 1] - tok;
      }
      const long long r = on ? static_cast<long long>(p.lengths[s]) - left : -1;
      pos = static_cast<int>(r);
      if (pair == 0) {
        long long at = -1;
        if (r >= 0 && r < static_cast<long long>(p.width) * p.page) {
          const int ri = static_cast<int>(r), pi = ri / p.page;
          const int pg = p.table[static_cast<long long>(s) * p.width + pi];
          if (pg >= 0 && pg < p.n_pages) at = static_cast<long long>(pg) * p.nkv * p.page + (ri - pi * p.page);
        }
        row[ti] = at;
      }
    }
    if (on && p.positions) pos = p.positions[tok];
    if (pair == 0) live[ti] = on;
    if (pair < pairs) {
      const double f = p.freqs[pair] * 0.15915494309189533577;  // / (2 pi): turns a position
      const unsigned long long per = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
      const long long angle = static_cast<long long>(per * static_cast<unsigned long long>(static_cast<long long>(pos)));
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 4.6566128730773925781e-10f, &sn, &cs);  // * 2^-31
      turn[ti][pair] = make_float2(cs * p.magnitude, sn * p.magnitude);
    }
  }
  __syncthreads();

  constexpr int kUnits = HD / 16;  // a thread's item: two 16-byte chunks of a row
  const int heads = p.nq + p.nkv + (p.k_pages ? p.nkv : 0);
  const int per_tok = heads * kUnits, rot_units = p.rot / 16;
  for (int i = t; i < TOK * per_tok; i += kThreads) {
    const int ti = i / per_tok, j = i - ti * per_tok, h = j / kUnits, u = j % kUnits;
    if (!live[ti]) continue;
    const long long tok = tok0 + ti;
    const bool turned = u < rot_units && h < p.nq + p.nkv;
    // chunks of the row: a pair's partners lie rot / 2 elements apart, or side by side
    const int c0 = turned && !p.interleaved ? u : 2 * u, c1 = turned && !p.interleaved ? u + rot_units : 2 * u + 1;
    const char* src;
    if (h < p.nq) src = static_cast<const char*>(p.q) + 2 * (tok * p.q_tok + h * p.q_head);
    else if (h < p.nq + p.nkv) src = static_cast<const char*>(p.k) + 2 * (tok * p.k_tok + (h - p.nq) * p.k_head);
    else src = static_cast<const char*>(p.v) + 2 * (tok * p.v_tok + (h - p.nq - p.nkv) * p.v_head);
    uint4 a = reinterpret_cast<const uint4*>(src)[c0], b = reinterpret_cast<const uint4*>(src)[c1];
    if (turned) {
      uint32_t* aw = reinterpret_cast<uint32_t*>(&a);
      uint32_t* bw = reinterpret_cast<uint32_t*>(&b);
      const float2* cs = &turn[ti][8 * u];
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = unpack<BF16>(aw[e]), y = unpack<BF16>(bw[e]), m = cs[e], n = cs[4 + e];
          aw[e] = pack<BF16>(x.x * m.x - x.y * m.y, x.y * m.x + x.x * m.y);
          bw[e] = pack<BF16>(y.x * n.x - y.y * n.y, y.y * n.x + y.x * n.y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = unpack<BF16>(aw[e]), y = unpack<BF16>(bw[e]), m = cs[2 * e], n = cs[2 * e + 1];
          aw[e] = pack<BF16>(x.x * m.x - y.x * m.y, x.y * n.x - y.y * n.y);
          bw[e] = pack<BF16>(y.x * m.x + x.x * m.y, y.y * n.x + x.y * n.y);
        }
      }
    }
    if (h < p.nq) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(p.q_out) + 2 * (tok * p.qo_tok + h * p.qo_head));
      dst[c0] = a, dst[c1] = b;
    } else {
      const bool is_k = h < p.nq + p.nkv;
      const int g = h - p.nq - (is_k ? 0 : p.nkv);
      if (is_k && p.k_out) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(p.k_out) + 2 * (tok * p.ko_tok + g * p.ko_head));
        dst[c0] = a, dst[c1] = b;
      }
      if (p.k_pages && row[ti] >= 0) {
        const long long r = row[ti] + static_cast<long long>(g) * p.page;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(is_k ? p.k_pages : p.v_pages) + 2 * r * HD);
        dst[c0] = a, dst[c1] = b;
        if (is_k && u == 0 && p.key_weights) p.key_weights[r] = 0.f;
      }
    }
  }
}

template <bool BF16, int HD>
cudaError_t launch_t(const RotaryParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.tokens <= 256) {
    cfg.gridDim = dim3(p.tokens);
    return cudaLaunchKernelEx(&cfg, rotary_kernel<BF16, HD, 1>, p);
  }
  cfg.gridDim = dim3((p.tokens + 3) / 4);
  return cudaLaunchKernelEx(&cfg, rotary_kernel<BF16, HD, 4>, p);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, bool bf16, cudaStream_t s) {
  if (p.tokens == 0) return cudaSuccess;
  if (p.hd == 64) return bf16 ? launch_t<true, 64>(p, s) : launch_t<false, 64>(p, s);
  return bf16 ? launch_t<true, 128>(p, s) : launch_t<false, 128>(p, s);
}

}  // namespace lps
