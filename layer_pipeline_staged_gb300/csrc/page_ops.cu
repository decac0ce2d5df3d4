// Entry points of the operators over a paged cache and of the logits'
// adjustment: argument checks, tensor maps and launches. Nothing here
// synchronises, allocates device memory or keeps anything between calls;
// lengths, tables, offsets and positions are device arrays that the kernels
// check, so a captured launch replays with what they hold then.
#include "kernels.h"
#include "op_host.h"
#include "page_ops.h"
#include "ptx.cuh"

namespace {

using namespace lps;

int check_pages(const char* fn, int n_pages, int page_size, int width) {
  if (n_pages < 1) return host_fail(LPS_EINVAL, fn, "n_pages must be >= 1");
  if (page_size < 8 || page_size % 8 || page_size > 65536)
    return host_fail(LPS_EINVAL, fn, "page_size must be a multiple of 8 in 8..65536");
  if (width < 1 || static_cast<long long>(width) * page_size > kMaxRows)
    return host_fail(LPS_EINVAL, fn, "table_width must be >= 1, and table_width * page_size at most 2^31 - 2^16");
  return LPS_OK;
}

int check_pools(const char* fn, const void* k, const void* v, int n_pages, int page_size, int nkv, int hd) {
  if (misaligned(k) || misaligned(v)) return host_fail(LPS_EINVAL, fn, "the pages must be 16-byte aligned");
  if (overlap(k, v, static_cast<double>(n_pages) * page_size * nkv, hd))
    return host_fail(LPS_EINVAL, fn, "the pages of keys and of values must not overlap");
  return LPS_OK;
}

int check_turn(const char* fn, const double* freqs, int rot, int hd, float magnitude) {
  if (rot < 0 || rot > hd || rot % 16) return host_fail(LPS_EINVAL, fn, "rot_dim must be a multiple of 16 in 0..head_dim");
  if (rot && !freqs) return host_fail(LPS_EINVAL, fn, "freqs is required");
  if (!std::isfinite(magnitude)) return host_fail(LPS_EINVAL, fn, "magnitude must be finite");
  return LPS_OK;
}

int launched(const char* fn, cudaError_t e) {
  return e == cudaSuccess ? LPS_OK : host_fail(LPS_ECUDA, fn, std::string("launch: ") + cudaGetErrorString(e));
}

int check_plain_heads(const char* fn, int type, int nq, int nkv, int hd) {
  if (nq < 1 || nq > 65535 || nkv < 1 || nkv > 65535) return host_fail(LPS_EINVAL, fn, "n_q_heads and n_kv_heads must be in 1..65535");
  return check_heads(fn, type, nkv, nkv, hd);
}

}  // namespace

extern "C" int rotary_rows(const void* q, const void* k, void* q_out, void* k_out, int type, int n_tokens,
                           const int32_t* positions, const double* freqs, int rot_dim, int interleaved, float magnitude,
                           int n_q_heads, int n_kv_heads, int head_dim, const int64_t* strides, void* stream) {
  static const char* FN = "rotary_rows";
  return guarded(FN, [&]() -> int {
    if (!q || !k || !q_out || !k_out || !positions) return host_fail(LPS_EINVAL, FN, "q, k, their outputs and positions are required");
    if (n_tokens < 0 || n_tokens > kMaxRows) return host_fail(LPS_EINVAL, FN, "n_tokens must be in [0, 2^31 - 2^16]");
    int rc = check_plain_heads(FN, type, n_q_heads, n_kv_heads, head_dim);
    if (rc || (rc = check_turn(FN, freqs, rot_dim, head_dim, magnitude))) return rc;
    const int64_t qd = static_cast<int64_t>(n_q_heads) * head_dim, kd = static_cast<int64_t>(n_kv_heads) * head_dim;
    const int64_t dense[8] = {qd, head_dim, kd, head_dim, qd, head_dim, kd, head_dim};
    const int64_t* st = strides ? strides : dense;
    if ((rc = check_strides(FN, st, 8, head_dim))) return rc;
    if (misaligned(q) || misaligned(k) || misaligned(q_out) || misaligned(k_out))
      return host_fail(LPS_EINVAL, FN, "q, k and their outputs must be 16-byte aligned");
    RotaryParams p{};
    p.q = q, p.k = k, p.q_out = q_out, p.k_out = k_out;
    p.q_tok = st[0], p.q_head = st[1], p.k_tok = st[2], p.k_head = st[3];
    p.qo_tok = st[4], p.qo_head = st[5], p.ko_tok = st[6], p.ko_head = st[7];
    p.freqs = freqs, p.positions = positions;
    p.tokens = n_tokens;
    p.nq = n_q_heads, p.nkv = n_kv_heads, p.hd = head_dim, p.rot = rot_dim, p.interleaved = interleaved != 0;
    p.magnitude = magnitude;
    return launched(FN, launch_rotary(p, type == LPS_TYPE_BF16, static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int rotary_append_paged(const void* q, const void* k, const void* v, void* q_out, int type, int n_tokens,
                                   int n_seqs, const int32_t* offsets, const int32_t* lengths, const int32_t* table,
                                   int table_width, void* k_pages, void* v_pages, int n_pages, int page_size,
                                   const int32_t* positions, const double* freqs, int rot_dim, int interleaved,
                                   float magnitude, float* key_weights, int n_q_heads, int n_kv_heads, int head_dim,
                                   const int64_t* strides, void* stream) {
  static const char* FN = "rotary_append_paged";
  return guarded(FN, [&]() -> int {
    if (!q || !k || !v || !q_out || !lengths || !table || !k_pages || !v_pages)
      return host_fail(LPS_EINVAL, FN, "q, k, v, q_out, lengths, table and the pages are required");
    if (n_tokens < 0 || n_tokens > kMaxRows || n_seqs < 1) return host_fail(LPS_EINVAL, FN, "n_tokens must be in [0, 2^31 - 2^16] and n_seqs >= 1");
    if (!offsets && n_tokens != n_seqs) return host_fail(LPS_EINVAL, FN, "without offsets there is one token a sequence");
    int rc = check_plain_heads(FN, type, n_q_heads, n_kv_heads, head_dim);
    if (rc || (rc = check_turn(FN, freqs, rot_dim, head_dim, magnitude)) || (rc = check_pages(FN, n_pages, page_size, table_width)))
      return rc;
    const int64_t qd = static_cast<int64_t>(n_q_heads) * head_dim, kd = static_cast<int64_t>(n_kv_heads) * head_dim;
    const int64_t dense[8] = {qd, head_dim, kd, head_dim, kd, head_dim, qd, head_dim};
    const int64_t* st = strides ? strides : dense;
    if ((rc = check_strides(FN, st, 8, head_dim)) || (rc = check_pools(FN, k_pages, v_pages, n_pages, page_size, n_kv_heads, head_dim)))
      return rc;
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(q_out))
      return host_fail(LPS_EINVAL, FN, "q, k, v and q_out must be 16-byte aligned");
    RotaryParams p{};
    p.q = q, p.k = k, p.v = v, p.q_out = q_out;
    p.q_tok = st[0], p.q_head = st[1], p.k_tok = st[2], p.k_head = st[3], p.v_tok = st[4], p.v_head = st[5];
    p.qo_tok = st[6], p.qo_head = st[7];
    p.freqs = freqs, p.positions = positions, p.offsets = offsets, p.lengths = lengths, p.table = table;
    p.k_pages = k_pages, p.v_pages = v_pages, p.key_weights = key_weights;
    p.tokens = n_tokens, p.n_seqs = n_seqs, p.width = table_width, p.n_pages = n_pages, p.page = page_size;
    p.nq = n_q_heads, p.nkv = n_kv_heads, p.hd = head_dim, p.rot = rot_dim, p.interleaved = interleaved != 0;
    p.magnitude = magnitude;
    return launched(FN, launch_rotary(p, type == LPS_TYPE_BF16, static_cast<cudaStream_t>(stream)));
  });
}

namespace {

// The shape of a decode call, checked; the CTAs of the current device.
int paged_shape(const char* fn, PagedAttnParams& p, int batch, int nq, int nkv, int hd, int page_size, int width) {
  if (batch < 1 || batch > kPagedBatch) return host_fail(LPS_EINVAL, fn, "batch must be in 1..1024");
  int rc = check_heads(fn, LPS_TYPE_BF16, nq, nkv, hd);
  if (rc || (rc = check_pages(fn, 1, page_size, width))) return rc;
  const long long rows = static_cast<long long>(width) * page_size;
  if (((rows + 63) / 64 + 1) * nkv > 0x7fffffffll / batch) return host_fail(LPS_EINVAL, fn, "too many rows, kv heads and sequences for one launch");
  p.batch = batch, p.nq = nq, p.nkv = nkv, p.group = nq / nkv, p.page = page_size, p.width = width;
  const cudaError_t e = paged_attn_ctas(&p.ctas);
  return e == cudaSuccess ? LPS_OK : host_fail(LPS_ECUDA, fn, cudaGetErrorString(e));
}

}  // namespace

extern "C" long long attention_paged_decode_workspace(int batch, int n_q_heads, int n_kv_heads, int head_dim, int page_size,
                                                      int table_width, int weights) {
  static const char* FN = "attention_paged_decode_workspace";
  long long bytes = 0;
  const int rc = guarded(FN, [&]() -> int {
    PagedAttnParams p{};
    const int bad = paged_shape(FN, p, batch, n_q_heads, n_kv_heads, head_dim, page_size, table_width);
    if (!bad) bytes = paged_attn_workspace(p, head_dim, weights != 0);
    return bad;
  });
  return rc ? rc : bytes;
}

extern "C" int attention_paged_decode(const void* q, const void* k_pages, const void* v_pages, void* out, int type, int batch,
                                      const int32_t* lengths, const int32_t* table, int table_width, int n_pages,
                                      int page_size, int n_q_heads, int n_kv_heads, int head_dim, const int64_t* strides,
                                      float scale, float* key_weights, float decay, void* workspace,
                                      long long workspace_bytes, void* stream) {
  static const char* FN = "attention_paged_decode";
  return guarded(FN, [&]() -> int {
    if (!q || !k_pages || !v_pages || !out || !lengths || !table || !workspace)
      return host_fail(LPS_EINVAL, FN, "q, the pages, out, lengths, table and workspace are required");
    int rc = check_heads(FN, type, n_q_heads, n_kv_heads, head_dim);
    if (rc || (rc = check_scale(FN, scale)) || (rc = check_pages(FN, n_pages, page_size, table_width))) return rc;
    if (!(decay >= 0.f && decay <= 1.f)) return host_fail(LPS_EINVAL, FN, "decay must be in [0, 1]");
    const int64_t seq = static_cast<int64_t>(n_q_heads) * head_dim;
    const int64_t dense[4] = {seq, head_dim, seq, head_dim};
    const int64_t* st = strides ? strides : dense;
    if ((rc = check_strides(FN, st, 4, head_dim))) return rc;
    if (misaligned(q) || misaligned(k_pages) || misaligned(v_pages) || misaligned(out) || misaligned(workspace))
      return host_fail(LPS_EINVAL, FN, "q, the pages, out and workspace must be 16-byte aligned");
    if (out == q) return host_fail(LPS_EINVAL, FN, "out must not be q: several blocks read a head's q");
    PagedAttnParams p{};
    if ((rc = paged_shape(FN, p, batch, n_q_heads, n_kv_heads, head_dim, page_size, table_width))) return rc;
    if (workspace_bytes < paged_attn_workspace(p, head_dim, key_weights != nullptr))
      return host_fail(LPS_EINVAL, FN, "workspace_bytes is less than attention_paged_decode_workspace asks for");
    paged_attn_place(p, head_dim, key_weights != nullptr, workspace);
    p.q = q, p.out = out;
    p.q_seq = st[0], p.q_head = st[1], p.o_seq = st[2], p.o_head = st[3];
    p.table = table, p.lengths = lengths, p.key_weights = key_weights;
    p.n_pages = n_pages;
    p.box = page_size & -page_size;  // the most rows of a power of two that lie in one page wherever they begin
    if (p.box > 64) p.box = 64;
    p.wait_limit = wait_cycles(op_wait_limit());
    p.decay = decay;
    p.scale_log2 = kLog2e * (scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(head_dim)));
    const bool bf16 = type == LPS_TYPE_BF16;
    if (!encode_pages(&p.tmap_k, bf16, k_pages, head_dim, page_size, n_kv_heads, n_pages, p.box) ||
        !encode_beside(&p.tmap_v, p.tmap_k, v_pages))
      return host_fail(LPS_ECUDA, FN, "cuTensorMapEncodeTiled failed");
    return launched(FN, launch_paged_attn(p, bf16, head_dim, static_cast<cudaStream_t>(stream)));
  });
}

namespace {
int check_evict(const char* fn, int batch, int nkv, int budget) {
  if (batch < 1 || batch > 65535) return host_fail(LPS_EINVAL, fn, "batch must be in 1..65535");
  if (nkv < 1 || nkv > 65535) return host_fail(LPS_EINVAL, fn, "n_kv_heads must be in 1..65535");
  if (budget < 1 || budget > kMaxRows) return host_fail(LPS_EINVAL, fn, "budget must be in [1, 2^31 - 2^16]");
  return LPS_OK;
}
}  // namespace

extern "C" long long kv_pages_evict_workspace(int batch, int n_kv_heads, int budget) {
  static const char* FN = "kv_pages_evict_workspace";
  long long bytes = 0;
  const int rc = guarded(FN, [&]() -> int {
    const int bad = check_evict(FN, batch, n_kv_heads, budget);
    if (!bad) bytes = 4ll * batch * n_kv_heads * budget;
    return bad;
  });
  return rc ? rc : bytes;
}

extern "C" int kv_pages_evict(void* k_pages, void* v_pages, float* key_weights, int n_pages, int page_size, int n_kv_heads,
                              int head_dim, int batch, const int32_t* lengths, const int32_t* table, int table_width,
                              const int32_t* new_table, int new_width, int32_t* new_lengths, int budget, int recent,
                              void* workspace, long long workspace_bytes, void* stream) {
  static const char* FN = "kv_pages_evict";
  return guarded(FN, [&]() -> int {
    if (!k_pages || !v_pages || !key_weights || !lengths || !table || !new_table || !new_lengths || !workspace)
      return host_fail(LPS_EINVAL, FN, "the pages, key_weights, lengths, the tables, new_lengths and workspace are required");
    int rc = check_heads(FN, LPS_TYPE_BF16, n_kv_heads, n_kv_heads, head_dim);
    if (rc || (rc = check_evict(FN, batch, n_kv_heads, budget)) || (rc = check_pages(FN, n_pages, page_size, table_width)) ||
        (rc = check_pages(FN, n_pages, page_size, new_width)) ||
        (rc = check_pools(FN, k_pages, v_pages, n_pages, page_size, n_kv_heads, head_dim)))
      return rc;
    if (recent < 0 || recent > budget) return host_fail(LPS_EINVAL, FN, "recent must be in 0..budget");
    if (static_cast<long long>(new_width) * page_size < budget) return host_fail(LPS_EINVAL, FN, "the new table must have room for budget rows");
    if (lengths == new_lengths || table == new_table) return host_fail(LPS_EINVAL, FN, "the new lengths and table must not be the old ones");
    if (misaligned(key_weights)) return host_fail(LPS_EINVAL, FN, "key_weights must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(workspace) & 3 || workspace_bytes < 4ll * batch * n_kv_heads * budget)
      return host_fail(LPS_EINVAL, FN, "workspace must be 4-byte aligned and hold what kv_pages_evict_workspace asks for");
    EvictParams p{};
    p.k_pages = static_cast<uint4*>(k_pages), p.v_pages = static_cast<uint4*>(v_pages), p.key_weights = key_weights;
    p.table = table, p.fresh = new_table, p.lengths = lengths, p.new_lengths = new_lengths, p.rows = static_cast<int*>(workspace);
    p.batch = batch, p.width = table_width, p.fresh_width = new_width, p.n_pages = n_pages, p.nkv = n_kv_heads, p.page = page_size;
    p.chunks = head_dim / 8, p.budget = budget, p.recent = recent;
    return launched(FN, launch_evict(p, static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int logits_adjust(const void* logits, void* out, int type, int batch, int vocab, const int64_t* strides,
                             const int32_t* tokens, int width, const int32_t* lengths, const int32_t* prompt_lengths,
                             const float* repetition, const float* frequency, const float* presence,
                             const int32_t* bias_ids, const float* bias, int n_bias, const uint32_t* allowed,
                             void* stream) {
  static const char* FN = "logits_adjust";
  return guarded(FN, [&]() -> int {
    if (!logits || !out) return host_fail(LPS_EINVAL, FN, "logits and out are required");
    if (type != LPS_TYPE_BF16 && type != LPS_TYPE_FP16 && type != LPS_TYPE_FP32)
      return host_fail(LPS_EINVAL, FN, "type must be LPS_TYPE_BF16, LPS_TYPE_FP16 or LPS_TYPE_FP32");
    if (batch < 1 || batch > 65535) return host_fail(LPS_EINVAL, FN, "batch must be in 1..65535");
    if (vocab < 1 || vocab > kMaxRows) return host_fail(LPS_EINVAL, FN, "vocab must be in [1, 2^31 - 2^16]");
    if (width < 0 || width >= (1 << 30) || n_bias < 0 || n_bias >= (1 << 30))
      return host_fail(LPS_EINVAL, FN, "width and n_bias must be in [0, 2^30)");
    if (width > 0 && (!tokens || !lengths)) return host_fail(LPS_EINVAL, FN, "a history needs tokens and lengths");
    if (width == 0 && (repetition || frequency || presence)) return host_fail(LPS_EINVAL, FN, "penalties need a history");
    if (n_bias > 0 && (!bias_ids || !bias)) return host_fail(LPS_EINVAL, FN, "biases need bias_ids and bias");
    const int64_t dense[2] = {vocab, vocab};
    const int64_t* st = strides ? strides : dense;
    for (int i = 0; i < 2; ++i)
      if (st[i] < vocab || st[i] >= (1ll << 38)) return host_fail(LPS_EINVAL, FN, "row strides must be at least vocab and below 2^38");
    const uintptr_t size = type == LPS_TYPE_FP32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) % size || reinterpret_cast<uintptr_t>(out) % size)
      return host_fail(LPS_EINVAL, FN, "logits and out must be aligned to their elements");
    LogitsParams p{};
    p.in = logits, p.out = out, p.in_row = st[0], p.out_row = st[1];
    if (width > 0) p.tokens = tokens, p.lengths = lengths, p.prompts = prompt_lengths, p.width = width;
    p.repetition = repetition, p.frequency = frequency, p.presence = presence;
    if (n_bias > 0) p.bias_ids = bias_ids, p.bias = bias, p.n_bias = n_bias;
    p.allowed = allowed;
    p.batch = batch, p.vocab = vocab, p.words = (vocab - 1) / 32 + 1;
    return launched(FN, launch_logits(p, type, static_cast<cudaStream_t>(stream)));
  });
}
