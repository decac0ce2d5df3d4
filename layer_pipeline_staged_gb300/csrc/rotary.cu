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

#include "launch.h"
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

// Block = TOK consecutive tokens at a time, every grid's number of blocks again:
// their angles' cosines and sines once into shared memory, then an item (token,
// head, 16 elements) per thread, kBatch of which are on their way at once; the
// first ones while the angles are worked out.
template <bool BF16, int HD, int TOK>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  __shared__ unsigned long long per[kMaxPairs];  // turns a position, in units of 2^-64
  // (cos, sin) times the magnitude, of pair 8 u + e at [e][u]: lanes with other units read other banks
  __shared__ float2 turn[TOK][8][HD / 16];
  __shared__ long long row[TOK];                 // page * nkv * page rows + row in the page, or -1: not stored
  __shared__ int live[TOK], where[TOK];
  constexpr int kBatch = TOK == 1 ? 2 : 3;
  constexpr int kUnits = HD / 16;  // a thread's item: two 16-byte chunks of a row
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x, pairs = p.rot >> 1;
  if (t < pairs) {
    const double f = p.freqs[t] * 0.15915494309189533577;  // / (2 pi): turns a position
    per[t] = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
  }
  const int heads = p.nq + p.nkv + (p.k_pages ? p.nkv : 0);
  const int per_tok = heads * kUnits, rot_units = p.rot / 16, items = TOK * per_tok;

  for (int tok0 = blockIdx.x * TOK; tok0 < p.tokens; tok0 += gridDim.x * TOK) {
    // an item's place: its token, head and chunks of the row (a pair's partners lie
    // rot / 2 elements apart, or side by side)
    struct Item {
      int ti, h, u, c0, c1;
      bool on, turned;
    };
    auto item_of = [&](int i) {
      Item it;
      it.ti = 0;
#pragma unroll
      for (int k = 1; k < TOK; ++k) it.ti += i >= k * per_tok;
      const int j = i - it.ti * per_tok;
      it.h = j / kUnits, it.u = j % kUnits;
      it.on = i < items && tok0 + it.ti < p.tokens;
      it.turned = it.u < rot_units && it.h < p.nq + p.nkv;
      const bool apart = it.turned && !p.interleaved;
      it.c0 = apart ? it.u : 2 * it.u, it.c1 = apart ? it.u + rot_units : 2 * it.u + 1;
      return it;
    };
    auto fetch = [&](const Item& it, uint4& a, uint4& b) {
      if (!it.on) return;
      const long long tok = tok0 + it.ti;
      const char* src;
      if (it.h < p.nq) src = static_cast<const char*>(p.q) + 2 * (tok * p.q_tok + it.h * p.q_head);
      else if (it.h < p.nq + p.nkv) src = static_cast<const char*>(p.k) + 2 * (tok * p.k_tok + (it.h - p.nq) * p.k_head);
      else src = static_cast<const char*>(p.v) + 2 * (tok * p.v_tok + (it.h - p.nq - p.nkv) * p.v_head);
      a = reinterpret_cast<const uint4*>(src)[it.c0], b = reinterpret_cast<const uint4*>(src)[it.c1];
    };
    uint4 a[kBatch], b[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) fetch(item_of(t + e * kThreads), a[e], b[e]);

    __syncthreads();  // the last tokens' angles have been used
    if (t < TOK) {    // where each token goes, and what turns it
      const int tok = tok0 + t;
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
        long long at = -1;
        if (r >= 0 && r < static_cast<long long>(p.width) * p.page) {
          const int ri = static_cast<int>(r), pi = ri / p.page;
          const int pg = p.table[static_cast<long long>(s) * p.width + pi];
          if (pg >= 0 && pg < p.n_pages) at = static_cast<long long>(pg) * p.nkv * p.page + (ri - pi * p.page);
        }
        row[t] = at;
      }
      if (on && p.positions) pos = p.positions[tok];
      live[t] = on;
      where[t] = pos;
    }
    __syncthreads();
    for (int i = t; i < TOK * kMaxPairs; i += kThreads) {
      const int ti = i / kMaxPairs, pair = i % kMaxPairs;
      if (pair < pairs) {
        const long long angle = static_cast<long long>(per[pair] * static_cast<unsigned long long>(static_cast<long long>(where[ti])));
        float sn, cs;
        sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 4.6566128730773925781e-10f, &sn, &cs);  // * 2^-31
        turn[ti][pair & 7][pair >> 3] = make_float2(cs * p.magnitude, sn * p.magnitude);
      }
    }
    __syncthreads();

    for (int i0 = 0; i0 < items; i0 += kBatch * kThreads) {
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const Item it = item_of(i0 + t + e * kThreads);
        if (!it.on || !live[it.ti]) continue;
        if (it.turned) {
          uint32_t* aw = reinterpret_cast<uint32_t*>(&a[e]);
          uint32_t* bw = reinterpret_cast<uint32_t*>(&b[e]);
          const auto& cs = turn[it.ti];
          if (p.interleaved) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float2 x = unpack<BF16>(aw[w]), y = unpack<BF16>(bw[w]), m = cs[w][it.u], n = cs[4 + w][it.u];
              aw[w] = pack<BF16>(x.x * m.x - x.y * m.y, x.y * m.x + x.x * m.y);
              bw[w] = pack<BF16>(y.x * n.x - y.y * n.y, y.y * n.x + y.x * n.y);
            }
          } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float2 x = unpack<BF16>(aw[w]), y = unpack<BF16>(bw[w]), m = cs[2 * w][it.u], n = cs[2 * w + 1][it.u];
              aw[w] = pack<BF16>(x.x * m.x - y.x * m.y, x.y * n.x - y.y * n.y);
              bw[w] = pack<BF16>(y.x * m.x + x.x * m.y, y.y * n.x + x.y * n.y);
            }
          }
        }
        const long long tok = tok0 + it.ti;
        if (it.h < p.nq) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(p.q_out) + 2 * (tok * p.qo_tok + it.h * p.qo_head));
          dst[it.c0] = a[e], dst[it.c1] = b[e];
        } else {
          const bool is_k = it.h < p.nq + p.nkv;
          const int g = it.h - p.nq - (is_k ? 0 : p.nkv);
          if (is_k && p.k_out) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(p.k_out) + 2 * (tok * p.ko_tok + g * p.ko_head));
            dst[it.c0] = a[e], dst[it.c1] = b[e];
          }
          if (p.k_pages && row[it.ti] >= 0) {
            const long long r = row[it.ti] + static_cast<long long>(g) * p.page;
            uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(is_k ? p.k_pages : p.v_pages) + 2 * r * HD);
            dst[it.c0] = a[e], dst[it.c1] = b[e];
            if (is_k && it.u == 0 && p.key_weights) p.key_weights[r] = 0.f;
          }
        }
      }
      if (i0 + kBatch * kThreads < items) {
#pragma unroll
        for (int e = 0; e < kBatch; ++e) fetch(item_of(i0 + kBatch * kThreads + t + e * kThreads), a[e], b[e]);
      }
    }
  }
}

template <bool BF16, int HD>
cudaError_t launch_t(const RotaryParams& p, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // a token a block while that gives no SM more than two, else four
  if (p.tokens <= 2 * sms) return launch_early(rotary_kernel<BF16, HD, 1>, dim3(p.tokens), kThreads, 0, s, p);
  return launch_early(rotary_kernel<BF16, HD, 4>, dim3((p.tokens + 3) / 4), kThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, bool bf16, cudaStream_t s) {
  if (p.tokens == 0) return cudaSuccess;
  if (p.hd == 64) return bf16 ? launch_t<true, 64>(p, s) : launch_t<false, 64>(p, s);
  return bf16 ? launch_t<true, 128>(p, s) : launch_t<false, 128>(p, s);
}

}  // namespace lps
