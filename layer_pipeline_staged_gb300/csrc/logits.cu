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
// meets for the first time, while the run comes to L2; the run is streamed through with
// the mask alone, and the listed ones are then read again from the output, worked out
// and written over. Every block of a row reads all of its history, from L2, and that is
// what bounds long ones: 64 rows of 128256 in fp32 take 9.1 us without a history and 15.7
// with up to 8192 tokens. Penalties worked out for every token took 26; the history's
// reading shared out over a cluster, with counts in the owner's memory, 33; the stream
// before the counting 21.7; the listed ones worked out before the stream, with words of
// 32 bits that then held the results, 19.3.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.h"
#include "lps.h"
#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

// A token's word: whether prompt or output hold it, whether bias_ids do, and its count in
// the output. Two words share 32 bits where the history is shorter than 2^14 tokens, and
// so no count passes 14 bits: the blocks that an SM holds are bounded by shared memory.
template <bool WIDE>
struct Words {
  static constexpr uint32_t kSeen = WIDE ? 1u << 31 : 1u << 15, kBiased = kSeen >> 1, kCount = kBiased - 1;
  static constexpr int kBytes = WIDE ? 4 : 2;
  uint32_t* w;
  __device__ __forceinline__ uint32_t get(unsigned at) const {
    return WIDE ? w[at] : reinterpret_cast<const uint16_t*>(w)[at];
  }
  // the word as it was
  __device__ __forceinline__ uint32_t add_one(unsigned at) const {
    if (WIDE) return atomicAdd(w + at, 1u);
    const int by = (at & 1) * 16;
    return atomicAdd(w + (at >> 1), 1u << by) >> by & 0xffff;
  }
  __device__ __forceinline__ uint32_t set(unsigned at, uint32_t bit) const {
    if (WIDE) return atomicOr(w + at, bit);
    const int by = (at & 1) * 16;
    return atomicOr(w + (at >> 1), bit << by) >> by & 0xffff;
  }
};

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

// Block = (run of THREADS * EACH tokens, row). Places are counted from the 16-byte
// boundary at or before the row's first logit, `shift` elements before it, so that
// vectors lie on their boundaries wherever the row begins.
template <class T, int THREADS, int EACH, bool WIDE>
__global__ void __launch_bounds__(THREADS) logits_kernel(const __grid_constant__ LogitsParams p) {
  constexpr int V = 16 / sizeof(T), kVecs = EACH / V, kRun = THREADS * EACH, kAhead = 8;
  using W = Words<WIDE>;
  extern __shared__ uint4 space[];
  const W words{reinterpret_cast<uint32_t*>(space)};                                // [kRun]
  uint16_t* listed = reinterpret_cast<uint16_t*>(space + kRun * W::kBytes / 16);    // places of the tokens that have a word
  __shared__ int n_listed, twice;                                                   // whether a token has several biases
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
    for (int i = 0; i < EACH * W::kBytes / 16; ++i) space[i * THREADS + t] = make_uint4(0, 0, 0, 0);
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
        if (at < places && at >= unused && i < len) list(at, i >= prompt ? words.add_one(at) : words.set(at, W::kSeen));
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
      const uint32_t was = words.set(at, W::kBiased);
      list(at, was);
      if (was & W::kBiased) twice = 1;
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

  // The stream has left a listed token's own logit in `out`, or -inf for good.
  if (counted) {
    __syncthreads();
    const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f, pres = p.presence ? p.presence[b] : 0.f;
    auto is_allowed = [&](int e) { return !allowed || allowed[e >> 5] >> (e & 31) & 1; };
    auto penalized = [&](float x, uint32_t c) {
      if (c & ~W::kBiased) x = x > 0.f ? x / rep : x * rep;
      if (c & W::kCount) x -= fmaf(freq, static_cast<float>(c & W::kCount), pres);
      return x;
    };
#pragma unroll 2
    for (int i = t; i < n_listed; i += THREADS) {
      const int at = listed[i], e = run + at - shift;
      const uint32_t c = words.get(at);
      if (c & W::kBiased && !twice) continue;
      const float was = to_float(out[e]);
      if (!is_allowed(e)) continue;
      float x = penalized(was, c);
      if (c & W::kBiased) {  // its entries, in order
#pragma unroll 8
        for (int k = 0; k < p.n_bias; ++k) x += ids[k] == e ? bias[k] : 0.f;
      }
      from_float(out[e], x);
    }
    if (!twice) {
      for (int i = t; i < p.n_bias; i += THREADS) {
        const unsigned at = static_cast<unsigned>(ids[i]) - first;
        if (at < places && at >= unused && is_allowed(ids[i])) from_float(out[ids[i]], penalized(to_float(out[ids[i]]), words.get(at)) + bias[i]);
      }
    }
  }
}

long long history(const LogitsParams& p) { return static_cast<long long>(p.tokens ? p.width : 0) + (p.bias_ids ? p.n_bias : 0); }

template <class T, int THREADS, int EACH, bool WIDE>
cudaError_t launch_t(const LogitsParams& p, cudaStream_t s) {
  constexpr int kRun = THREADS * EACH;
  static_assert(kRun <= 65536, "a place in 16 bits");
  static std::atomic<uint64_t> told;
  const cudaError_t e = allow_smem(logits_kernel<T, THREADS, EACH, WIDE>, kRun * (Words<WIDE>::kBytes + 2), told);
  if (e != cudaSuccess) return e;
  // a row may begin up to a vector's elements behind a boundary
  const long long runs = (static_cast<long long>(p.vocab) + 16 / sizeof(T) - 1 + kRun - 1) / kRun;
  const long long entries = history(p);
  const int list = static_cast<int>(entries < kRun ? entries : kRun);
  return launch_early(logits_kernel<T, THREADS, EACH, WIDE>, dim3(static_cast<unsigned>(runs), p.batch), THREADS,
                      list ? kRun * Words<WIDE>::kBytes + 2 * list : 0, s, p);
}

// Threads of a block and tokens of a thread. Every block of a row reads all of its
// history, so a long one wants long runs, of many threads; short runs use more SMs and
// leave less to wait for at the end. us, rows of 128256, histories of up to so many tokens:
//                        128 x 16   512 x 16   512 x 32   1024 x 32
//   8 rows, fp32, 300          4.8        5.7        6.0
//   6 rows, fp32, 4000         7.3        5.5        6.5        7.4
//   12 rows, fp32, 300         5.1        6.3        6.8
//   12 rows, fp32, 20000      25.1       13.8       12.8       11.4
//   64 rows, fp32, 300        11.9       12.9       13.1       13.5
//   64 rows, fp32, 1000       12.7       13.3       13.4
//   32 rows, fp32, 2000       10.5        9.0       11.0       11.4
//   64 rows, fp32, 8192                  19.2       17.6       15.7
//   24 rows, bf16, 300         6.5        6.9        6.9        7.9
//   32 rows, bf16, 1000        7.9        7.3        8.3        8.7
//   40 rows, bf16, 300         7.3        7.9        8.5        9.4
//   44 rows, bf16, 2000       10.2        8.8        9.6        9.7
//   64 rows, bf16, 300         9.9       10.2        9.4        9.7
//   64 rows, bf16, 8000       28.3       15.8       13.6       11.3
// Short runs suit fp32 up to 1024 entries whatever the rows (1 to 128 of them); of 16-bit
// logits, where the stream takes half as long, up to 20480 tokens an SM (fp16 as bf16;
// around 35000 they would gain a tenth). Four blocks of 512 x 16 lie on an SM; with more
// tokens than 40960 an SM, a thread of 16-bit logits takes as many bytes as one of fp32.
template <class T>
cudaError_t launch_type(const LogitsParams& p, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const double of_sm = static_cast<double>(p.batch) * p.vocab / sms;
  const long long entries = history(p);
  const bool wide = p.tokens && p.width >= 1 << 14;
  if ((sizeof(T) == 4 || of_sm <= 20480) && entries <= 1024) return launch_t<T, 128, 16, false>(p, s);
  if ((of_sm > 8192 && entries > 8192) || (of_sm > 32768 && entries > 4096))
    return wide ? launch_t<T, 1024, 32, true>(p, s) : launch_t<T, 1024, 32, false>(p, s);
  if constexpr (sizeof(T) == 2)
    if (of_sm > 40960) return launch_t<T, 512, 32, false>(p, s);
  return wide ? launch_t<T, 512, 16, true>(p, s) : launch_t<T, 512, 16, false>(p, s);
}

}  // namespace

cudaError_t launch_logits(const LogitsParams& p, int type, cudaStream_t s) {
  if (type == LPS_TYPE_BF16) return launch_type<__nv_bfloat16>(p, s);
  if (type == LPS_TYPE_FP16) return launch_type<__half>(p, s);
  return launch_type<float>(p, s);
}

}  // namespace lps
