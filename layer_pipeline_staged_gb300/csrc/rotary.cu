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
//
// Bound by HBM when it is large: 12185 tokens, 32/8 heads of 128 with the append in 48.1
// us, 6.2 TB/s. Cosines stored by pair cost 4-way bank conflicts (53), places worked out
// per item 200 instructions a 64 bytes (53), a block's angles per head twice the time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.h"
#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;
constexpr int kRows = 512;  // (token, head) rows whose places are held at once

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

// Block = TOK consecutive tokens: their angles' cosines and sines, and where each
// (token, head) comes from and goes to, once into shared memory; then an item (row,
// 16 elements) per thread, kBatch of which are on their way at once, the first ones
// while the angles are worked out.
template <bool BF16, int HD, int TOK>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int kBatch = 3, kUnits = HD / 16;  // an item: two 16-byte chunks of a row
  // (cos, sin) times the magnitude, of pair 8 u + e at [e][u]: lanes with other units read other banks
  __shared__ float2 turn[TOK][8][kUnits];
  __shared__ const char* src[kRows];  // of the (token, head) rows; bit 0: it turns, 1 and 2: its token
  __shared__ char* dst[kRows];        // NULL: not stored
  __shared__ long long row[TOK];      // page * nkv * page rows + row in the page, or -1: not stored
  __shared__ int where[TOK], live[TOK];
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x, pairs = p.rot >> 1, tok0 = blockIdx.x * TOK;
  const int heads = p.nq + p.nkv + (p.k_pages ? p.nkv : 0), all_rows = min(TOK, p.tokens - tok0) * heads;

  // A thread's units are one: its chunks of a row that turns (a pair's partners lie
  // rot / 2 elements apart, or side by side) and of one that does not
  const int u = t % kUnits, lane_row = t / kUnits;
  constexpr int kStep = kThreads / kUnits;  // rows of a step
  const bool in_rot = u < p.rot / 16, apart = in_rot && !p.interleaved;
  const int plain = 32 * u, t0 = apart ? 16 * u : plain, t1 = apart ? 16 * (u + p.rot / 16) : plain + 16;

  for (int r0 = 0; r0 < all_rows; r0 += kRows) {
    const int rows = min(kRows, all_rows - r0);
    for (int r = t; r < rows; r += kThreads) {
      const int ti = TOK == 1 ? 0 : (r0 + r) / heads, h = r0 + r - ti * heads;
      const long long tok = tok0 + ti;
      const void* from = h < p.nq ? p.q : h < p.nq + p.nkv ? p.k : p.v;
      const int g = h < p.nq ? h : h < p.nq + p.nkv ? h - p.nq : h - p.nq - p.nkv;
      const long long by_tok = h < p.nq ? p.q_tok : h < p.nq + p.nkv ? p.k_tok : p.v_tok;
      const long long by_head = h < p.nq ? p.q_head : h < p.nq + p.nkv ? p.k_head : p.v_head;
      src[r] = static_cast<const char*>(from) + 2 * (tok * by_tok + g * by_head) + (h < p.nq + p.nkv) + 2 * ti;
    }
    if (r0 == 0 && t < TOK) {  // where each token goes, and what turns it
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

    uint4 a[kBatch], b[kBatch];
    auto fetch = [&](int r, uint4& x, uint4& y) {
      if (r >= rows) return;
      const uintptr_t from = reinterpret_cast<uintptr_t>(src[r]);
      const char* at = reinterpret_cast<const char*>(from & ~static_cast<uintptr_t>(15));
      x = *reinterpret_cast<const uint4*>(at + (from & 1 ? t0 : plain));
      y = *reinterpret_cast<const uint4*>(at + (from & 1 ? t1 : plain + 16));
    };
#pragma unroll
    for (int e = 0; e < kBatch; ++e) fetch(lane_row + e * kStep, a[e], b[e]);

    if (r0 == 0) {
      for (int i = t; i < TOK * kMaxPairs; i += kThreads) {
        const int ti = i / kMaxPairs, pair = i % kMaxPairs;
        if (pair < pairs) {
          const double f = p.freqs[pair] * 0.15915494309189533577;  // / (2 pi): turns a position
          const unsigned long long per = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
          const long long angle = static_cast<long long>(per * static_cast<unsigned long long>(static_cast<long long>(where[ti])));
          float sn, cs;
          sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 4.6566128730773925781e-10f, &sn, &cs);  // * 2^-31
          turn[ti][pair & 7][pair >> 3] = make_float2(cs * p.magnitude, sn * p.magnitude);
        }
      }
    }
    for (int r = t; r < rows; r += kThreads) {
      const int ti = TOK == 1 ? 0 : (r0 + r) / heads, h = r0 + r - ti * heads;
      const long long tok = tok0 + ti;
      char* to = nullptr;
      if (h < p.nq) {
        to = static_cast<char*>(p.q_out) + 2 * (tok * p.qo_tok + h * p.qo_head);
      } else if (p.k_pages) {
        const bool is_k = h < p.nq + p.nkv;
        if (row[ti] >= 0) {
          const long long at = row[ti] + static_cast<long long>(h - p.nq - (is_k ? 0 : p.nkv)) * p.page;
          to = static_cast<char*>(is_k ? p.k_pages : p.v_pages) + 2 * at * HD;
          if (is_k && p.key_weights && live[ti]) p.key_weights[at] = 0.f;
        }
      } else {
        to = static_cast<char*>(p.k_out) + 2 * (tok * p.ko_tok + (h - p.nq) * p.ko_head);
      }
      dst[r] = live[ti] ? to : nullptr;
    }
    __syncthreads();

    for (int i0 = lane_row; i0 - lane_row < rows; i0 += kBatch * kStep) {
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int r = i0 + e * kStep;
        if (r >= rows) continue;
        char* to = dst[r];
        const uintptr_t from = reinterpret_cast<uintptr_t>(src[r]);
        if ((from & 1) && in_rot) {
          uint32_t* aw = reinterpret_cast<uint32_t*>(&a[e]);
          uint32_t* bw = reinterpret_cast<uint32_t*>(&b[e]);
          const auto& cs = turn[TOK == 1 ? 0 : from >> 1 & 3];
          if (p.interleaved) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float2 x = unpack<BF16>(aw[w]), y = unpack<BF16>(bw[w]), m = cs[w][u], n = cs[4 + w][u];
              aw[w] = pack<BF16>(x.x * m.x - x.y * m.y, x.y * m.x + x.x * m.y);
              bw[w] = pack<BF16>(y.x * n.x - y.y * n.y, y.y * n.x + y.x * n.y);
            }
          } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float2 x = unpack<BF16>(aw[w]), y = unpack<BF16>(bw[w]), m = cs[2 * w][u], n = cs[2 * w + 1][u];
              aw[w] = pack<BF16>(x.x * m.x - y.x * m.y, x.y * n.x - y.y * n.y);
              bw[w] = pack<BF16>(y.x * m.x + x.x * m.y, y.y * n.x + x.y * n.y);
            }
          }
        }
        if (to) {
          *reinterpret_cast<uint4*>(to + (from & 1 ? t0 : plain)) = a[e];
          *reinterpret_cast<uint4*>(to + (from & 1 ? t1 : plain + 16)) = b[e];
        }
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) fetch(i0 + (kBatch + e) * kStep, a[e], b[e]);
    }
    __syncthreads();  // the next rows' places
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
