// What the operators' entry points share on the host: the C boundary, checks of
// heads, scale, overlap and alignment, and the tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <exception>
#include <string>

#include "cache_ops.h"
#include "lps.h"

namespace lps {

int host_fail(int code, const char* fn, const std::string& why);
// The wait limit that cache_ops_set_wait_limit has set for the calling thread (0: the default).
long long op_wait_limit();

constexpr float kLog2e = 1.44269504088896340736f;

// Runs the body of an entry point; no exception leaves the C boundary.
template <class F>
int guarded(const char* fn, F&& body) {
  try {
    return body();
  } catch (const std::exception& e) {
    try {
      return host_fail(LPS_ENOMEM, fn, e.what());
    } catch (...) {
      return LPS_ENOMEM;
    }
  } catch (...) {
    return LPS_ENOMEM;
  }
}

// Whether two caches of so many rows of hd elements share memory.
inline bool overlap(const void* a, const void* b, double rows, int hd) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return static_cast<double>(x < y ? y - x : x - y) < rows * hd * 2;
}

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

inline int check_heads(const char* fn, int type, int nq, int nkv, int hd) {
  if (type != LPS_TYPE_BF16 && type != LPS_TYPE_FP16) return host_fail(LPS_EINVAL, fn, "type must be LPS_TYPE_BF16 or LPS_TYPE_FP16");
  if (hd != 64 && hd != 128) return host_fail(LPS_EINVAL, fn, "head_dim must be 64 or 128");
  if (nkv < 1 || nkv > 65535 || nq < 1 || nq % nkv || nq / nkv > kMaxGroup || nq > 65535)
    return host_fail(LPS_EINVAL, fn, "n_q_heads must be 1 to 16 times n_kv_heads (each at most 65535)");
  return LPS_OK;
}

inline int check_scale(const char* fn, float scale) {
  if (!(scale >= 0.f) || std::isinf(scale)) return host_fail(LPS_EINVAL, fn, "scale must be finite and >= 0 (0: 1/sqrt(head_dim))");
  if (std::isinf(scale * kLog2e)) return host_fail(LPS_EINVAL, fn, "scale must be below 2.3e38 (its product with log2(e) is what the kernels use)");
  return LPS_OK;
}

// Element strides of a tensor's outer axes: whole 16-byte units, at least one
// row apart, and inside what a tensor map can hold.
inline int check_strides(const char* fn, const int64_t* st, int n, int hd) {
  for (int i = 0; i < n; ++i)
    if (st[i] < hd || st[i] % 8 || st[i] >= (1ll << 38))
      return host_fail(LPS_EINVAL, fn, "strides must be multiples of 8 elements, at least head_dim and below 2^38");
  return LPS_OK;
}

// The driver's tensor-map encoder, looked up once per process.
inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// [n3][n2][n1][hd] of 2-byte elements with element strides s1..s3, in boxes of
// 64 elements x b1 x b2 with the 128-byte swizzle. The stride of an axis of one
// entry is never used and set to one row.
inline bool encode4(CUtensorMap* map, bool bf16, const void* base, int hd, const long long (&n)[3], const long long (&st)[3],
             int b1, int b2) {
  if (!encoder()) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(n[0]), static_cast<cuuint64_t>(n[1]),
                        static_cast<cuuint64_t>(n[2])};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) strides[i] = static_cast<cuuint64_t>(n[i] > 1 ? st[i] : hd) * 2;
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  auto encode = [&] {
    return encoder()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                     const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return true;
  // The driver's call wants a current context, which a host thread has from its
  // first runtime call on the device, and this may be it.
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

// Pages [n_pages][nkv][page][hd], dense, in boxes of `box` rows of both halves of
// the head, which lie one after the other: [half][row][64 elements].
inline bool encode_pages(CUtensorMap* map, bool bf16, const void* base, int hd, int page, int nkv, int n_pages, int box) {
  if (!encoder()) return false;
  cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(hd / 64), static_cast<cuuint64_t>(nkv),
                        static_cast<cuuint64_t>(n_pages)};
  const cuuint64_t row = static_cast<cuuint64_t>(hd) * 2;
  cuuint64_t strides[4] = {row, 128, row * page, row * page * nkv};
  cuuint32_t size[5] = {64, static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(hd / 64), 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  auto encode = [&] {
    return encoder()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                     const_cast<void*>(base), dims, strides, size, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return true;
  // as in encode4: a host thread's first call has no context yet
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

// The same map for another address: 0.3 to 0.5 us less of a call's 7 to 8 on the host than encoding it again.
inline bool encode_beside(CUtensorMap* map, const CUtensorMap& like, const void* base) {
  static const PFN_cuTensorMapReplaceAddress_v12000 replace = []() -> PFN_cuTensorMapReplaceAddress_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapReplaceAddress", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapReplaceAddress_v12000>(f);
  }();
  *map = like;
  return replace && replace(map, const_cast<void*>(base)) == CUDA_SUCCESS;
}

// Rows and tokens are counted in 32 bits, a block of keys past the last one included.
constexpr int32_t kMaxRows = 0x7fff0000;

}  // namespace lps
