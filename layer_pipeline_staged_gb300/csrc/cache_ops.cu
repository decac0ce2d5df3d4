// Entry points of the operators over a caller-owned cache: argument checks,
// tensor maps and launches. Nothing here synchronises, allocates device memory
// or keeps anything between calls (a test's wait limit apart). Lengths, offsets and positions are host
// arrays that travel in the kernel parameters (so a captured launch keeps the
// values it was captured with); a tree's parents and an accepted path are
// device arrays, as a drafter and a sampler on the GPU leave them, and the
// kernels check them.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <string>

#include "cache_ops.h"
#include "kernels.h"
#include "lps.h"
#include "ptx.cuh"

namespace lps {
int host_fail(int code, const char* fn, const std::string& why);
}  // namespace lps

namespace {

using namespace lps;

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

// Whether every row of an output starts on 32 bytes.
bool wide(const void* p, std::initializer_list<int64_t> strides) {
  if (reinterpret_cast<uintptr_t>(p) & 31) return false;
  for (int64_t s : strides)
    if (s % 16) return false;
  return true;
}

// Whether two caches of so many rows of hd elements share memory.
bool overlap(const void* a, const void* b, double rows, int hd) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return static_cast<double>(x < y ? y - x : x - y) < rows * hd * 2;
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

int check_heads(const char* fn, int type, int nq, int nkv, int hd) {
  if (type != LPS_TYPE_BF16 && type != LPS_TYPE_FP16) return host_fail(LPS_EINVAL, fn, "type must be LPS_TYPE_BF16 or LPS_TYPE_FP16");
  if (hd != 64 && hd != 128) return host_fail(LPS_EINVAL, fn, "head_dim must be 64 or 128");
  if (nkv < 1 || nkv > 65535 || nq < 1 || nq % nkv || nq / nkv > kMaxGroup || nq > 65535)
    return host_fail(LPS_EINVAL, fn, "n_q_heads must be 1 to 16 times n_kv_heads (each at most 65535)");
  return LPS_OK;
}

int check_scale(const char* fn, float scale) {
  if (!(scale >= 0.f) || std::isinf(scale)) return host_fail(LPS_EINVAL, fn, "scale must be finite and >= 0 (0: 1/sqrt(head_dim))");
  if (std::isinf(scale * kLog2e)) return host_fail(LPS_EINVAL, fn, "scale must be below 2.3e38 (its product with log2(e) is what the kernels use)");
  return LPS_OK;
}

// Element strides of a tensor's outer axes: whole 16-byte units, at least one
// row apart, and inside what a tensor map can hold.
int check_strides(const char* fn, const int64_t* st, int n, int hd) {
  for (int i = 0; i < n; ++i)
    if (st[i] < hd || st[i] % 8 || st[i] >= (1ll << 38))
      return host_fail(LPS_EINVAL, fn, "strides must be multiples of 8 elements, at least head_dim and below 2^38");
  return LPS_OK;
}

// The driver's tensor-map encoder, looked up once per process.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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
bool encode4(CUtensorMap* map, bool bf16, const void* base, int hd, const long long (&n)[3], const long long (&st)[3],
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

// Test hook: the wait limit of the calling thread's later calls.
thread_local long long g_wait_limit = 0;

// Rows and tokens are counted in 32 bits, a block of keys past the last one included.
constexpr int32_t kMaxRows = 0x7fff0000;

int check_offsets(const char* fn, int n_seqs, const int32_t* offsets) {
  if (offsets[0] < 0 || offsets[n_seqs] > kMaxRows) return host_fail(LPS_EINVAL, fn, "offsets must lie in [0, 2^31 - 2^16]");
  for (int s = 0; s < n_seqs; ++s)
    if (offsets[s + 1] < offsets[s]) return host_fail(LPS_EINVAL, fn, "offsets must not descend");
  return LPS_OK;
}

}  // namespace

extern "C" int attention_prompt_packed(const void* q, const void* k, const void* v, void* out, int type, int n_seqs,
                                       const int32_t* offsets, int n_q_heads, int n_kv_heads, int head_dim,
                                       const int64_t* strides, float scale, void* stream) {
  static const char* FN = "attention_prompt_packed";
  return guarded(FN, [&]() -> int {
    if (!q || !k || !v || !out || !offsets) return host_fail(LPS_EINVAL, FN, "q, k, v, out and offsets are required");
    if (n_seqs < 1) return host_fail(LPS_EINVAL, FN, "n_seqs must be >= 1");
    int rc = check_heads(FN, type, n_q_heads, n_kv_heads, head_dim);
    if (rc) return rc;
    if ((rc = check_scale(FN, scale)) || (rc = check_offsets(FN, n_seqs, offsets))) return rc;
    const int64_t q_dense = static_cast<int64_t>(n_q_heads) * head_dim, k_dense = static_cast<int64_t>(n_kv_heads) * head_dim;
    const int64_t dense[8] = {q_dense, head_dim, k_dense, head_dim, k_dense, head_dim, q_dense, head_dim};
    const int64_t* st = strides ? strides : dense;
    if ((rc = check_strides(FN, st, 8, head_dim))) return rc;
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(out))
      return host_fail(LPS_EINVAL, FN, "q, k, v and out must be 16-byte aligned");

    for (int s0 = 0; s0 < n_seqs; s0 += kOpSeqs) {
      TileAttnParams p{};
      p.n_seqs = n_seqs - s0 < kOpSeqs ? n_seqs - s0 : kOpSeqs;
      p.k = k, p.v = v, p.out = out;
      p.k_row = st[2], p.k_head = st[3];
      p.v_row = st[4], p.v_head = st[5], p.o_tok = st[6], p.o_head = st[7];
      p.nkv = n_kv_heads, p.group = n_q_heads / n_kv_heads;
      p.wide_out = wide(out, {st[6], st[7]});
      p.wait_limit = wait_cycles(g_wait_limit);
      p.scale_log2 = kLog2e * (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(head_dim)));
      for (int s = 0; s < p.n_seqs; ++s) {
        p.tok0[s] = offsets[s0 + s];
        p.len[s] = offsets[s0 + s + 1] - offsets[s0 + s];
      }
      const long long ctas = tile_prompt_plan(p);
      if (ctas == 0) continue;
      if (ctas > 0x7fffffffll) return host_fail(LPS_EINVAL, FN, "too many tokens for one launch");
      const bool bf16 = type == LPS_TYPE_BF16;
      const long long tokens = offsets[n_seqs];
      if (!encode4(&p.tmap_q, bf16, q, head_dim, {n_q_heads, tokens, 1}, {st[1], st[0], 0}, p.group, p.tpt) ||
          !encode4(&p.tmap_k, bf16, k, head_dim, {tokens, n_kv_heads, 1}, {st[2], st[3], 0}, 128, 1) ||
          !encode4(&p.tmap_v, bf16, v, head_dim, {tokens, n_kv_heads, 1}, {st[4], st[5], 0}, 128, 1))
        return host_fail(LPS_ECUDA, FN, "cuTensorMapEncodeTiled failed");
      const cudaError_t e = launch_tile_prompt(p, ctas, bf16, head_dim, static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return host_fail(LPS_ECUDA, FN, std::string("launch: ") + cudaGetErrorString(e));
    }
    return LPS_OK;
  });
}

namespace {
int check_tree(const char* fn, int batch, int width, const int32_t* pos, const int32_t* rows, int max_ctx) {
  if (batch < 1 || batch > kOpSeqs) return host_fail(LPS_EINVAL, fn, "batch must be in 1..256");
  if (width < 1 || width > kTreeMax) return host_fail(LPS_EINVAL, fn, "width must be in 1..64");
  if (max_ctx < 1 || max_ctx > kMaxRows) return host_fail(LPS_EINVAL, fn, "max_ctx must be in [1, 2^31 - 2^16]");
  for (int b = 0; b < batch; ++b) {
    if (pos[b] < 0 || rows[b] < 0 || rows[b] > width) return host_fail(LPS_EINVAL, fn, "need pos >= 0 and 0 <= rows <= width");
    if (pos[b] > max_ctx - rows[b]) return host_fail(LPS_EINVAL, fn, "pos + rows must stay within max_ctx");
  }
  return LPS_OK;
}
}  // namespace

extern "C" int attention_tree_verify(const void* q, const void* k_cache, const void* v_cache, void* out, int type,
                                     int batch, int width, const int32_t* pos, const int32_t* rows,
                                     const int32_t* parents, int n_q_heads, int n_kv_heads, int head_dim, int max_ctx,
                                     const int64_t* strides, float scale, void* stream) {
  static const char* FN = "attention_tree_verify";
  return guarded(FN, [&]() -> int {
    if (!q || !k_cache || !v_cache || !out || !pos || !rows || !parents)
      return host_fail(LPS_EINVAL, FN, "q, the caches, out, pos, rows and parents are required");
    int rc = check_heads(FN, type, n_q_heads, n_kv_heads, head_dim);
    if (rc) return rc;
    if ((rc = check_tree(FN, batch, width, pos, rows, max_ctx)) || (rc = check_scale(FN, scale))) return rc;
    const int64_t tok = static_cast<int64_t>(n_q_heads) * head_dim;
    const int64_t dense[6] = {width * tok, tok, head_dim, width * tok, tok, head_dim};
    const int64_t* st = strides ? strides : dense;
    if ((rc = check_strides(FN, st, 6, head_dim))) return rc;
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(out))
      return host_fail(LPS_EINVAL, FN, "q, the caches and out must be 16-byte aligned");
    const bool bf16 = type == LPS_TYPE_BF16;
    TileAttnParams p{};
    p.n_seqs = batch;
    p.width = width;
    p.nkv = n_kv_heads, p.group = n_q_heads / n_kv_heads;
    for (int b = 0; b < batch; ++b) p.pos[b] = pos[b], p.len[b] = rows[b];
    long long ctas = 0;
    cudaError_t e = tile_tree_plan(p, bf16, head_dim, &ctas);
    if (e != cudaSuccess) return host_fail(LPS_ECUDA, FN, std::string("plan: ") + cudaGetErrorString(e));
    if (ctas == 0) return LPS_OK;
    if (ctas > 0x7fffffffll) return host_fail(LPS_EINVAL, FN, "too many rows for one launch");
    p.k = k_cache, p.v = v_cache, p.out = out;
    p.o_seq = st[3], p.o_tok = st[4], p.o_head = st[5];
    p.k_row = p.v_row = head_dim;
    p.k_head = p.v_head = static_cast<long long>(max_ctx) * head_dim;
    p.k_seq = p.v_seq = p.k_head * n_kv_heads;
    p.parents = parents;
    p.wide_out = wide(out, {st[3], st[4], st[5]});
    p.wait_limit = wait_cycles(g_wait_limit);
    p.scale_log2 = kLog2e * (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(head_dim)));
    const long long kv_n[3] = {max_ctx, n_kv_heads, batch}, kv_st[3] = {p.k_row, p.k_head, p.k_seq};
    if (!encode4(&p.tmap_q, bf16, q, head_dim, {n_q_heads, width, batch}, {st[2], st[1], st[0]}, p.group, p.tpt) ||
        !encode4(&p.tmap_k, bf16, k_cache, head_dim, kv_n, kv_st, 128, 1) ||
        !encode4(&p.tmap_v, bf16, v_cache, head_dim, kv_n, kv_st, 128, 1))
      return host_fail(LPS_ECUDA, FN, "cuTensorMapEncodeTiled failed");
    e = launch_tile_tree(p, ctas, bf16, head_dim, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return host_fail(LPS_ECUDA, FN, std::string("launch: ") + cudaGetErrorString(e));
    return LPS_OK;
  });
}

extern "C" int kv_rows_append(const void* k, const void* v, int n_seqs, const int32_t* offsets, void* k_cache,
                              void* v_cache, const int32_t* start, int n_kv_heads, int head_dim, int max_ctx,
                              const int64_t* strides, void* stream) {
  static const char* FN = "kv_rows_append";
  return guarded(FN, [&]() -> int {
    if (!k || !v || !offsets || !k_cache || !v_cache || !start)
      return host_fail(LPS_EINVAL, FN, "k, v, offsets, the caches and start are required");
    if (n_seqs < 1) return host_fail(LPS_EINVAL, FN, "n_seqs must be >= 1");
    int rc = check_heads(FN, LPS_TYPE_BF16, n_kv_heads, n_kv_heads, head_dim);
    if (rc || (rc = check_offsets(FN, n_seqs, offsets))) return rc;
    if (max_ctx < 1 || max_ctx > kMaxRows) return host_fail(LPS_EINVAL, FN, "max_ctx must be in [1, 2^31 - 2^16]");
    if (k_cache == v_cache) return host_fail(LPS_EINVAL, FN, "the two caches must differ");
    for (int s = 0; s < n_seqs; ++s)
      if (start[s] < 0 || start[s] > max_ctx || offsets[s + 1] - offsets[s] > max_ctx - start[s])
        return host_fail(LPS_EINVAL, FN, "start + the sequence's length must stay within [0, max_ctx]");
    const int64_t kd = static_cast<int64_t>(n_kv_heads) * head_dim;
    const int64_t dense[4] = {kd, head_dim, kd, head_dim};
    const int64_t* st = strides ? strides : dense;
    if ((rc = check_strides(FN, st, 4, head_dim))) return rc;
    if (misaligned(k) || misaligned(v) || misaligned(k_cache) || misaligned(v_cache))
      return host_fail(LPS_EINVAL, FN, "k, v and the caches must be 16-byte aligned");
    if (overlap(k_cache, v_cache, static_cast<double>(n_seqs) * n_kv_heads * max_ctx, head_dim))
      return host_fail(LPS_EINVAL, FN, "the two caches must not overlap");
    const long long seq_units = static_cast<long long>(n_kv_heads) * max_ctx * (head_dim / 8);
    for (int s0 = 0; s0 < n_seqs; s0 += kOpSeqs) {
      AppendParams p{};
      p.n_seqs = n_seqs - s0 < kOpSeqs ? n_seqs - s0 : kOpSeqs;
      p.k = static_cast<const uint4*>(k), p.v = static_cast<const uint4*>(v);
      p.kc = static_cast<uint4*>(k_cache) + s0 * seq_units, p.vc = static_cast<uint4*>(v_cache) + s0 * seq_units;
      p.k_tok = st[0] / 8, p.k_head = st[1] / 8, p.v_tok = st[2] / 8, p.v_head = st[3] / 8;
      p.nkv = n_kv_heads, p.chunks = head_dim / 8, p.max_ctx = max_ctx;
      for (int s = 0; s < p.n_seqs; ++s) p.off[s] = offsets[s0 + s], p.start[s] = start[s0 + s];
      p.off[p.n_seqs] = offsets[s0 + p.n_seqs];
      const cudaError_t e = launch_append(p, static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return host_fail(LPS_ECUDA, FN, std::string("launch: ") + cudaGetErrorString(e));
    }
    return LPS_OK;
  });
}

extern "C" int kv_rows_accept(void* k_cache, void* v_cache, int n_layers, int batch, int n_kv_heads, int head_dim,
                              int max_ctx, const int32_t* pos, int width, const int32_t* path,
                              const int32_t* accepted, void* stream) {
  static const char* FN = "kv_rows_accept";
  return guarded(FN, [&]() -> int {
    if (!k_cache || !v_cache || !pos || !path || !accepted)
      return host_fail(LPS_EINVAL, FN, "the caches, pos, path and accepted are required");
    if (n_layers < 1 || n_layers > 32767) return host_fail(LPS_EINVAL, FN, "n_layers must be in 1..32767");
    if (batch < 1 || batch > kOpSeqs) return host_fail(LPS_EINVAL, FN, "batch must be in 1..256");
    if (width < 1 || width > kTreeMax) return host_fail(LPS_EINVAL, FN, "width must be in 1..64");
    const int rc = check_heads(FN, LPS_TYPE_BF16, n_kv_heads, n_kv_heads, head_dim);
    if (rc) return rc;
    if (max_ctx < 1 || max_ctx > kMaxRows) return host_fail(LPS_EINVAL, FN, "max_ctx must be in [1, 2^31 - 2^16]");
    if (k_cache == v_cache) return host_fail(LPS_EINVAL, FN, "the two caches must differ");
    for (int b = 0; b < batch; ++b)
      if (pos[b] < 0 || pos[b] > max_ctx) return host_fail(LPS_EINVAL, FN, "pos out of [0, max_ctx]");
    if (misaligned(k_cache) || misaligned(v_cache)) return host_fail(LPS_EINVAL, FN, "the caches must be 16-byte aligned");
    if (overlap(k_cache, v_cache, static_cast<double>(n_layers) * batch * n_kv_heads * max_ctx, head_dim))
      return host_fail(LPS_EINVAL, FN, "the two caches must not overlap");
    AcceptParams p{};
    p.kc = static_cast<uint4*>(k_cache), p.vc = static_cast<uint4*>(v_cache);
    p.path = path, p.accepted = accepted;
    p.layers = n_layers, p.batch = batch, p.nkv = n_kv_heads, p.max_ctx = max_ctx, p.chunks = head_dim / 8, p.width = width;
    for (int b = 0; b < batch; ++b) p.pos[b] = pos[b];
    const cudaError_t e = launch_accept(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return host_fail(LPS_ECUDA, FN, std::string("launch: ") + cudaGetErrorString(e));
    return LPS_OK;
  });
}

extern "C" int cache_ops_set_wait_limit(long long cycles) {
  if (cycles < 0) return host_fail(LPS_EINVAL, "cache_ops_set_wait_limit", "cycles must be >= 0");
  g_wait_limit = cycles;
  return LPS_OK;
}

extern "C" int cache_ops_status(void* stream) {
  static const char* FN = "cache_ops_status";
  return guarded(FN, [&]() -> int {
    int st[2] = {0, 0};
    const cudaError_t e = tile_attn_status(st, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return host_fail(LPS_ECUDA, FN, cudaGetErrorString(e));
    if (!st[0] && !st[1]) return LPS_OK;
    return host_fail(LPS_ECUDA, FN, "an earlier call's output is invalid: " + describe_status(st[0], st[1]));
  });
}
