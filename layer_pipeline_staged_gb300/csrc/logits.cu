// Logits before a token is chosen: penalties for repeated tokens, biases and a
// grammar's mask in one pass over the vocabulary. For token i of row b, with c
// its count in the row's output and s whether prompt or output hold it:
//     x = s ? (x > 0 ? x / repetition : x * repetition) : x
//     x = c > 0 ? x - (frequency * c + presence) : x
//     x = x + biases of i,  x = allowed ? x : -inf
// in fp32, rounded once. Bound by HBM: the logits in and out once.
//
// Only the mask concerns every token. A block takes a run of the vocabulary; it
// counts the row's history for its run in shared memory and lists the tokens it
// meets for the first time; the listed ones are worked out by themselves, the run is
// streamed through with the mask alone, and the listed ones' results are written
// over it. Every block of a row reads all of its history, from L2, and that is what
// bounds long ones: 64 rows of 128256 in fp32 take 10 us without a history and 19.3 with
// up to 8192 tokens. Penalties worked out for every token took 26; the history's reading
// shared out over a cluster, with counts in the owner's memory, 33; runs of 16384 tokens
// 20.8, of 8192 with half the threads 23.7; the stream before the counting 21.7.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.h"
#include "lps.h"
#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

constexpr int kEach = 16;  // tokens of a thread
// a token's word: in the prompt or output, in bias_ids, count in the output
constexpr uint32_t kSeen = 1u << 31, kBiased = 1u << 30, kCount = kBiased - 1;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float& y, float x) { y = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(__half& y, float x) { y = __float2half_rn(x); }

// The bytes [p, p + n), both multiples of 16, on their way from HBM to L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t n) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(n) : "memory");
}

// Block = (run of THREADS * kEach tokens, row). Places are counted from the 16-byte
// boundary at or before the row's first logit, `shift` elements before it, so that
// vectors lie on their boundaries wherever the row begins.
template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS) logits_kernel(const __grid_constant__ LogitsParams p) {
  constexpr int V = 16 / sizeof(T), kVecs = kEach / V, kRun = THREADS * kEach, kAhead = 8;
  extern __shared__ uint32_t words[];                             // [kRun]: a token's word, then its result
  uint16_t* listed = reinterpret_cast<uint16_t*>(words + kRun);   // [kRun]: places of the tokens that have a word
  __shared__ int n_listed, twice;                                 // whether a token has several biases
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x, b = blockIdx.y, run = blockIdx.x * kRun;
  const T* in = static_cast<const T*>(p.in) + b * p.in_row;
  T* out = static_cast<T*>(p.out) + b * p.out_row;
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(in) & 15) / sizeof(T));
  const bool aligned_out = static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T)) == shift;
  if (run - shift >= p.vocab) return;  // the grid has room for a row that begins behind a boundary
  const uint32_t* allowed = p.allowed ? p.allowed + static_cast<long long>(b) * p.words : nullptr;

  const bool counted = p.tokens || p.bias_ids;
  const int* ids = p.bias_ids + static_cast<long long>(b) * p.n_bias;
  const float* bias = p.bias + static_cast<long long>(b) * p.n_bias;
  // A token's place, or past the run for those that are in another one or in none;
  // the places before the row's first logit are not used.
  const unsigned first = static_cast<unsigned>(run - shift), places = min(kRun, p.vocab - run + shift);  // at least 1 place
  const unsigned unused = run == 0 ? shift : 0;
  if (counted) {
    // the run comes to L2 while the history is read
    if (t == 0) {
      const uintptr_t from = (reinterpret_cast<uintptr_t>(in + (run - shift) + unused) + 15) & ~static_cast<uintptr_t>(15);
      const uintptr_t to = reinterpret_cast<uintptr_t>(in + (run - shift) + places) & ~static_cast<uintptr_t>(15);
      if (from < to) prefetch_l2(reinterpret_cast<const void*>(from), static_cast<uint32_t>(to - from));
    }
    // the history's first tokens are asked for before its length is known
    const int* tokens = p.tokens + static_cast<long long>(b) * p.width;
    int tok[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) tok[j] = p.tokens && j * THREADS + t < p.width ? tokens[j * THREADS + t] : -1;
    const int len = p.tokens ? min(max(p.lengths[b], 0), p.width) : 0, prompt = p.prompts ? p.prompts[b] : 0;
#pragma unroll
    for (int i = 0; i < kEach / 4; ++i) reinterpret_cast<uint4*>(words)[i * THREADS + t] = make_uint4(0, 0, 0, 0);
    if (t == 0) n_listed = twice = 0;
    __syncthreads();
    auto list = [&](unsigned at, uint32_t was) {
      if (was == 0) listed[atomicAdd(&n_listed, 1)] = static_cast<uint16_t>(at);
    };
    for (int i0 = t; i0 - t < len; i0 += THREADS * kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + j * THREADS;
        const unsigned at = static_cast<unsigned>(tok[j]) - first;
        if (at < places && at >= unused && i < len) list(at, i >= prompt ? atomicAdd(words + at, 1u) : atomicOr(words + at, kSeen));
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + (kAhead + j) * THREADS;
        tok[j] = i < len ? tokens[i] : -1;
      }
    }
    for (int i = t; i < p.n_bias; i += THREADS) {
      const unsigned at = static_cast<unsigned>(ids[i]) - first;
      if (at >= places || at < unused) continue;
      const uint32_t was = atomicOr(words + at, kBiased);
      list(at, was);
      if (was & kBiased) twice = 1;
    }
    __syncthreads();

    const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f, pres = p.presence ? p.presence[b] : 0.f;
    for (int i = t; i < n_listed; i += THREADS) {
      const int at = listed[i], e = run + at - shift;
      const uint32_t c = words[at], n = c & kCount;
      float x = to_float(in[e]);
      if (c & ~kBiased) x = x > 0.f ? x / rep : x * rep;
      if (n) x -= fmaf(freq, static_cast<float>(n), pres);
      if (twice && c & kBiased) {  // its entries, in order
#pragma unroll 8
        for (int k = 0; k < p.n_bias; ++k) x += ids[k] == e ? bias[k] : 0.f;
      }
      words[at] = __float_as_uint(x);
    }
    __syncthreads();  // the listed logits have been read, for those that write over them
    if (!twice) {
      for (int i = t; i < p.n_bias; i += THREADS) {
        const unsigned at = static_cast<unsigned>(ids[i]) - first;
        if (at < places && at >= unused) words[at] = __float_as_uint(__uint_as_float(words[at]) + bias[i]);
      }
    }
  }

  T low;
  from_float(low, -INFINITY);
#pragma unroll 4
  for (int i = 0; i < kVecs; ++i) {
    const int e = run + (i * THREADS + t) * V - shift;  // the vector's first token
    if (e + V <= 0 || e >= p.vocab) continue;
    const bool inside = e >= 0 && e + V <= p.vocab;
    uint4 raw;
    T* x = reinterpret_cast<T*>(&raw);
    if (inside) {
      raw = *reinterpret_cast<const uint4*>(in + e);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = e + j >= 0 && e + j < p.vocab ? in[e + j] : low;
    }
    if (allowed) {
      const int e0 = max(e, 0), word = e0 >> 5;
      uint32_t bits = __funnelshift_r(allowed[word], word + 1 < p.words ? allowed[word + 1] : 0u, e0 & 31);
      if (e < 0) bits <<= -e;
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = bits >> j & 1 ? x[j] : low;
    }
    if (inside && aligned_out) {
      *reinterpret_cast<uint4*>(out + e) = raw;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e + j >= 0 && e + j < p.vocab) out[e + j] = x[j];
    }
  }

  if (counted) {
    __syncthreads();
    for (int i = t; i < n_listed; i += THREADS) {
      const int at = listed[i], e = run + at - shift;
      from_float(out[e], !allowed || allowed[e >> 5] >> (e & 31) & 1 ? __uint_as_float(words[at]) : -INFINITY);
    }
  }
}

template <class T, int THREADS>
cudaError_t launch_t(const LogitsParams& p, cudaStream_t s) {
  constexpr int kRun = THREADS * kEach;
  static_assert(kRun <= 65536, "a place in 16 bits");
  static std::atomic<uint64_t> told;
  const cudaError_t e = allow_smem(logits_kernel<T, THREADS>, kRun * 6, told);
  if (e != cudaSuccess) return e;
  // a row may begin up to a vector's elements behind a boundary
  const long long runs = (static_cast<long long>(p.vocab) + 16 / sizeof(T) - 1 + kRun - 1) / kRun;
  return launch_early(logits_kernel<T, THREADS>, dim3(static_cast<unsigned>(runs), p.batch), THREADS,
                      p.tokens || p.bias_ids ? kRun * 6 : 0, s, p);
}

template <class T>
cudaError_t launch_type(const LogitsParams& p, cudaStream_t s) {
  // long runs where they fill the SMs (every block of a row reads all of its history),
  // else short ones, for more SMs
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
