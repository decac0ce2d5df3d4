// Logits before a token is chosen: penalties for repeated tokens, biases and a
// grammar's mask in one pass over the vocabulary. For token i of row b, with c
// its count in the row's output and s whether prompt or output hold it:
//     x = s ? (x > 0 ? x / repetition : x * repetition) : x
//     x = x - frequency * c - presence * (c > 0) + biases of i
//     x = allowed ? x : -inf
// in fp32, rounded once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lps.h"
#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

constexpr int kThreads = 512;
constexpr int kChunk = 8192;       // tokens of a block
constexpr uint32_t kSeen = 1u << 31;

template <class T>
__device__ __forceinline__ float load(const T* p);
template <>
__device__ __forceinline__ float load(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store(__half* p, float x) { *p = __float2half_rn(x); }

// Block = (chunk of the vocabulary, row): the row's history is counted for the
// chunk in shared memory (count of the output in the lower 31 bits, kSeen for
// the prompt), biases are added up there, and the chunk's logits pass once.
template <class T>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitsParams p) {
  extern __shared__ uint32_t counts[];  // [kChunk], then with biases float [kChunk]
  float* extra = reinterpret_cast<float*>(counts + (p.tokens ? kChunk : 0));
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x, b = blockIdx.y, lo = blockIdx.x * kChunk;
  const int n = min(kChunk, p.vocab - lo);
  for (int i = t; i < n; i += kThreads) {
    if (p.tokens) counts[i] = 0;
    if (p.bias_ids) extra[i] = 0.f;
  }
  __syncthreads();
  if (p.tokens) {
    const int len = min(max(p.lengths[b], 0), p.width), prompt = p.prompts ? p.prompts[b] : 0;
    const int* tokens = p.tokens + static_cast<long long>(b) * p.width;
    for (int i = t; i < len; i += kThreads) {
      const unsigned at = static_cast<unsigned>(tokens[i]) - static_cast<unsigned>(lo);
      if (at >= static_cast<unsigned>(n)) continue;
      if (i >= prompt) atomicAdd(&counts[at], 1u);
      else atomicOr(&counts[at], kSeen);
    }
  }
  if (p.bias_ids) {
    const int* ids = p.bias_ids + static_cast<long long>(b) * p.n_bias;
    const float* bias = p.bias + static_cast<long long>(b) * p.n_bias;
    for (int i = t; i < p.n_bias; i += kThreads) {
      const int id = ids[i];
      const unsigned at = static_cast<unsigned>(id) - static_cast<unsigned>(lo);
      if (at >= static_cast<unsigned>(n)) continue;
      // the first entry of a token adds up all of its entries, in order
      bool first = true;
      for (int j = 0; j < i && first; ++j) first = ids[j] != id;
      if (!first) continue;
      float sum = bias[i];
      for (int j = i + 1; j < p.n_bias; ++j)
        if (ids[j] == id) sum += bias[j];
      extra[at] = sum;
    }
  }
  __syncthreads();
  const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f, pres = p.presence ? p.presence[b] : 0.f;
  const T* in = static_cast<const T*>(p.in) + b * p.in_row + lo;
  T* out = static_cast<T*>(p.out) + b * p.out_row + lo;
  const uint32_t* allowed = p.allowed ? p.allowed + static_cast<long long>(b) * p.words + lo / 32 : nullptr;
  for (int i = t; i < n; i += kThreads) {
    float x = load(in + i);
    if (p.tokens) {
      const uint32_t w = counts[i];
      if (w) {
        x = x > 0.f ? x / rep : x * rep;
        const float c = static_cast<float>(w & ~kSeen);
        if (c > 0.f) x = x - freq * c - pres;
      }
    }
    if (p.bias_ids) x += extra[i];
    if (allowed && !(allowed[i >> 5] >> (i & 31) & 1)) x = -INFINITY;
    store(out + i, x);
  }
}

template <class T>
cudaError_t launch_t(const LogitsParams& p, cudaStream_t s) {
  const size_t smem = (static_cast<size_t>(p.tokens != nullptr) + (p.bias_ids != nullptr)) * kChunk * 4;
  cudaError_t e = cudaFuncSetAttribute(logits_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kChunk * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.vocab + kChunk - 1) / kChunk, p.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logits_kernel<T>, p);
}

}  // namespace

cudaError_t launch_logits(const LogitsParams& p, int type, cudaStream_t s) {
  if (type == LPS_TYPE_BF16) return launch_t<__nv_bfloat16>(p, s);
  if (type == LPS_TYPE_FP16) return launch_t<__half>(p, s);
  return launch_t<float>(p, s);
}

}  // namespace lps
