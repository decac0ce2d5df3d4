// Parameter blocks and launchers of the operators over a paged cache: rotary
// positions with the append to pages (rotary.cu), decode attention
// (paged_attn.cu), eviction (page_evict.cu), and the logits' adjustment
// (logits.cu). Lengths, tables, offsets and positions are device arrays, which
// the kernels check; everything else is checked by the entry points
// (page_ops.cu) before any launcher is called.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache_ops.h"

namespace lps {

constexpr int kPagedBatch = 1024;  // sequences of one attention call (their lengths are kept in shared memory)

// Rows (token, head) of q and k turned by their token's position; with pages,
// k and v also go to row lengths[s] - (offsets[s + 1] - token) of sequence s.
struct RotaryParams {
  const void* q;               // element (t, h): q + t * q_tok + h * q_head
  const void* k;
  const void* v;               // append only
  void* q_out;
  void* k_out;                 // NULL: k goes to the pages only
  long long q_tok, q_head, k_tok, k_head, v_tok, v_head, qo_tok, qo_head, ko_tok, ko_head;
  const double* freqs;         // [rot / 2] radians a position
  const int* positions;        // [tokens], or NULL: the cache row
  const int* offsets;          // append: [n_seqs + 1], or NULL: token t is sequence t's
  const int* lengths;          // append: [n_seqs], rows of the cache after the append
  const int* table;            // append: [n_seqs][width]
  void* k_pages;               // append: [n_pages][nkv][page][hd], or NULL: no append
  void* v_pages;
  float* key_weights;          // [n_pages][nkv][page], set to 0 for the new rows; or NULL
  int tokens, n_seqs, width, n_pages, page;
  int nq, nkv, hd, rot, interleaved;
  float magnitude;
};
cudaError_t launch_rotary(const RotaryParams& p, bool bf16, cudaStream_t s);

// One query row a sequence against its pages. A CTA takes an equal, contiguous
// share of all the tiles (sequence, kv head, 64 keys); what it computes of a
// head that others share goes to the workspace, and a second kernel joins it. Or,
// where the tables have room for few rows of few heads, a head is a cluster's, which
// joins it in the same launch; the second kernel then only sums key weights, if any.
struct PagedAttnParams {
  CUtensorMap tmap_k;          // [n_pages][nkv][page][hd], boxes of `box` rows
  CUtensorMap tmap_v;
  const void* q;               // element (b, h): q + b * q_seq + h * q_head
  void* out;
  long long q_seq, q_head, o_seq, o_head;
  const int* table;            // [batch][width]
  const int* lengths;          // [batch]
  float* key_weights;          // [n_pages][nkv][page], or NULL
  float* part_o;               // workspace: [ctas][2][group][hd]
  float2* part_ml;             // [ctas][2][group]: base, and sum (-1: no key was seen); then,
                               // with key_weights, of heads that one CTA (or cluster) has whole: [batch][nkv][group]
  int4* border;                // [ctas]: the head that begins in the CTA's share and ends in another's: sequence,
                               // kv head, its parts (0: there is none), whether the share begins before it
  int* first_unit;             // key_weights: [batch + 1]: of each sequence, then their number
  float* scores;               // key_weights: [batch][nq][width * page], times log2(e)
  long long wait_limit;
  int batch, width, n_pages, page, box;
  int nq, nkv, group;
  int ctas;
  float scale_log2, decay;
  int cluster;  // the members of a head's cluster, where it is one's
};
// CTAs of the current device's launch, and the workspace's bytes (weights: with key_weights).
cudaError_t paged_attn_ctas(int* ctas);
long long paged_attn_workspace(const PagedAttnParams& p, int hd, bool weights);
// Set the workspace's pointers.
void paged_attn_place(PagedAttnParams& p, int hd, bool weights, void* workspace);
cudaError_t launch_paged_attn(const PagedAttnParams& p, bool bf16, int hd, cudaStream_t s);
cudaError_t paged_attn_status(int* status, cudaStream_t s);

// Per (sequence, kv head): the last `recent` rows and the heaviest of the
// others, `budget` in all, in order, to the rows of the new table.
struct EvictParams {
  uint4* k_pages;              // [n_pages][nkv][page][hd]
  uint4* v_pages;
  float* key_weights;          // [n_pages][nkv][page]
  const int* table;            // [batch][width]
  const int* fresh;            // [batch][fresh_width]
  const int* lengths;          // [batch]
  int* new_lengths;            // [batch]; -1: a sequence whose length or table breaks the rules
  int* rows;                   // workspace: [batch][nkv][budget], the rows taken
  int batch, width, fresh_width, n_pages, nkv, page, chunks;  // chunks: 16-byte units of a row
  int budget, recent;
};
cudaError_t launch_evict(const EvictParams& p, cudaStream_t s);

struct LogitsParams {
  const void* in;              // row b: in + b * in_row elements
  void* out;
  long long in_row, out_row;
  const int* tokens;           // [batch][width], or NULL
  const int* lengths;          // [batch]
  const int* prompts;          // [batch], or NULL: 0
  const float* repetition;     // [batch], or NULL: 1
  const float* frequency;      // [batch], or NULL: 0
  const float* presence;       // [batch], or NULL: 0
  const int* bias_ids;         // [batch][n_bias], or NULL
  const float* bias;
  const uint32_t* allowed;     // [batch][words], or NULL
  int batch, vocab, width, n_bias, words;
};
cudaError_t launch_logits(const LogitsParams& p, int type, cudaStream_t s);

}  // namespace lps
