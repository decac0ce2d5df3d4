// Logits before a token is chosen: penalties for repeated tokens, biases and a
// grammar's mask in one pass over the vocabulary. For token i of row b, with c
// its count in the row's output and s whether prompt or output hold it:
//     x = s ? (x > 0 ? x / repetition : x * repetition) : x
//     x = c > 0 ? x - frequency * c - presence : x
//     x = x + biases of i,  x = allowed ? x : -inf
// in fp32, rounded once. Bound by HBM: the logits in and out once. A block takes a
// run of the vocabulary and asks for its logits first; while they are on their
// way, it counts the row's history for its run in shared memory (every block of a
// row reads all of it, from L2; sharing the reading out over a thread-block cluster
// and counting in the owner's memory took longer: 64 rows of 128256 with up to 8192
// tokens 32.6 us instead of 25.2). No branch goes by a token's count: with a few
// percent of the tokens counted, nearly every warp would go both ways.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.h"
#include "lps.h"
#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

constexpr int kEach = 16;          // tokens of a thread
constexpr uint32_t kSeen = 1u << 31;

template <class T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);  // elements of a 16-byte vector
};
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float& y, float x) { y = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(__half& y, float x) { y = __float2half_rn(x); }

// Block = (run of THREADS * kEach tokens, row). Places are counted from the 16-byte
// boundary at or before the row's first logit, `shift` elements before it, so that
// a vector of the input is a vector of the counts, wherever the row begins.
template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1536 / THREADS) logits_kernel(const __grid_constant__ LogitsParams p) {
  constexpr int V = Vec<T>::n, kVecs = kEach / V, kRun = THREADS * kEach;
  extern __shared__ uint4 smem[];
  uint32_t* counts = reinterpret_cast<uint32_t*>(smem);                        // [kRun]: kSeen, and the count in the output
  float* extra = reinterpret_cast<float*>(counts + (p.tokens ? kRun : 0));     // [kRun]: biases
  int* held = reinterpret_cast<int*>(extra + (p.bias_ids ? kRun : 0));         // [THREADS]: a lot of bias ids
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x, b = blockIdx.y, run = blockIdx.x * kRun;
  const T* in = static_cast<const T*>(p.in) + b * p.in_row;
  T* out = static_cast<T*>(p.out) + b * p.out_row;
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(in) & 15) / sizeof(T));
  const bool aligned_out = static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T)) == shift;
  if (run - shift >= p.vocab) return;  // the grid has room for a row that begins behind a boundary

  uint4 raw[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int e = run + (i * THREADS + t) * V - shift;  // the vector's first token
    if (e >= 0 && e + V <= p.vocab) {
      raw[i] = *reinterpret_cast<const uint4*>(in + e);
    } else {
      T* x = reinterpret_cast<T*>(&raw[i]);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e + j >= 0 && e + j < p.vocab) x[j] = in[e + j];
        else from_float(x[j], 0.f);
    }
  }

  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kEach / 4; ++i) {
    if (p.tokens) reinterpret_cast<uint4*>(counts)[i * THREADS + t] = zero;
    if (p.bias_ids) reinterpret_cast<uint4*>(extra)[i * THREADS + t] = zero;
  }
  __syncthreads();
  if (p.tokens) {
    const int len = min(max(p.lengths[b], 0), p.width), prompt = p.prompts ? min(max(p.prompts[b], 0), len) : 0;
    const int* tokens = p.tokens + static_cast<long long>(b) * p.width;
    // A token's place, or past the run for those that are in another one, in none
    // or past the history. Those in the `shift` places before the row's first logit
    // are not used.
    const unsigned first = static_cast<unsigned>(run - shift), places = min(kRun, p.vocab - run + shift);  // at least 1
    auto each = [&](int from, int to, auto&& count) {
      constexpr int kAhead = 8;
      for (int i0 = from + t; i0 - t < to; i0 += THREADS * kAhead) {
        unsigned at[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) at[j] = (i0 + j * THREADS < to ? static_cast<unsigned>(tokens[i0 + j * THREADS]) : 0xffffffffu) - first;
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (at[j] < places) count(counts[at[j]]);
      }
    };
    each(0, prompt, [](uint32_t& c) { c = kSeen; });
    __syncthreads();
    each(prompt, len, [](uint32_t& c) { atomicAdd(&c, 1u); });  // a warp's equal ones are one addition in hardware
  }
  if (p.bias_ids) {
    const int* ids = p.bias_ids + static_cast<long long>(b) * p.n_bias;
    const float* bias = p.bias + static_cast<long long>(b) * p.n_bias;
    // a run's entries, one after another where a token has several: an entry that
    // follows an equal one is added by that one's thread
    for (int i0 = 0; i0 < p.n_bias; i0 += THREADS) {
      const int i = i0 + t, id = i < p.n_bias ? ids[i] : -1;
      __syncthreads();  // the last lot's ids have been compared
      held[t] = id;
      __syncthreads();
      const bool mine = id >= 0 && id < p.vocab && static_cast<unsigned>(id + shift - run) < static_cast<unsigned>(kRun);
      if (mine) {
        bool first = true;
        float sum = bias[i];
        for (int j = 0; j < THREADS && i0 + j < p.n_bias; j += 4) {
          const int4 h4 = *reinterpret_cast<const int4*>(held + j);
          if (h4.x != id && h4.y != id && h4.z != id && h4.w != id) continue;
          for (int k = j; k < j + 4; ++k)
            if (held[k] == id && k != t) {
              if (k < t) first = false;
              else sum += bias[i0 + k];
            }
        }
        if (first) extra[id + shift - run] += sum;  // after the lots before
      }
    }
  }
  __syncthreads();

  const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f, pres = p.presence ? p.presence[b] : 0.f;
  const float inv = 1.f / rep;
  const uint32_t* allowed = p.allowed ? p.allowed + static_cast<long long>(b) * p.words : nullptr;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int at = (i * THREADS + t) * V, e = run + at - shift;
    if (e + V <= 0 || e >= p.vocab) continue;
    T* x = reinterpret_cast<T*>(&raw[i]);
    uint32_t bits = 0xffffffffu;
    if (allowed) {
      const int e0 = max(e, 0), word = e0 >> 5;
      bits = __funnelshift_r(allowed[word], word + 1 < p.words ? allowed[word + 1] : 0u, e0 & 31);
      if (e < 0) bits <<= -e;
    }
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      uint4 c4 = zero;
      float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.tokens) c4 = *reinterpret_cast<const uint4*>(counts + at + j);
      if (p.bias_ids) add = *reinterpret_cast<const float4*>(extra + at + j);
      const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
      const float a[4] = {add.x, add.y, add.z, add.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float y = to_float(x[j + k]);
        if (p.tokens) {
          const uint32_t n = c[k] & ~kSeen;
          y *= c[k] ? (y > 0.f ? inv : rep) : 1.f;
          y -= n ? fmaf(freq, static_cast<float>(n), pres) : 0.f;
        }
        y += a[k];
        from_float(x[j + k], bits >> (j + k) & 1 ? y : -INFINITY);
      }
    }
    if (aligned_out && e >= 0 && e + V <= p.vocab) {
      *reinterpret_cast<uint4*>(out + e) = raw[i];
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e + j >= 0 && e + j < p.vocab) out[e + j] = x[j];
    }
  }
}

template <class T, int THREADS>
cudaError_t launch_t(const LogitsParams& p, cudaStream_t s) {
  constexpr int kRun = THREADS * kEach;
  static std::atomic<uint64_t> told;
  const size_t smem = (static_cast<size_t>(p.tokens != nullptr) + (p.bias_ids != nullptr)) * kRun * 4 + THREADS * 4;
  cudaError_t e = allow_smem(logits_kernel<T, THREADS>, 2 * kRun * 4 + THREADS * 4, told);
  if (e != cudaSuccess) return e;
  // a row may begin up to a vector's elements behind a boundary
  const long long runs = (static_cast<long long>(p.vocab) + Vec<T>::n - 1 + kRun - 1) / kRun;
  return launch_early(logits_kernel<T, THREADS>, dim3(static_cast<unsigned>(runs), p.batch), THREADS, smem, s, p);
}

template <class T>
cudaError_t launch_type(const LogitsParams& p, cudaStream_t s) {
  // runs of 8192 tokens where they fill the SMs (every block of a row reads all of
  // its history), else of 2048, for more SMs
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  return static_cast<double>(p.batch) * p.vocab > 8192.0 * sms ? launch_t<T, 512>(p, s) : launch_t<T, 128>(p, s);
}

}  // namespace

cudaError_t launch_logits(const LogitsParams& p, int type, cudaStream_t s) {
  if (type == LPS_TYPE_BF16) return launch_type<__nv_bfloat16>(p, s);
  if (type == LPS_TYPE_FP16) return launch_type<__half>(p, s);
  return launch_type<float>(p, s);
}

}  // namespace lps
