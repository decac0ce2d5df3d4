// Parameter blocks and launchers of the operators over a caller-owned cache:
// attention of packed prompts and of drafted trees (tile_attn.cu), and the
// cache's row moves (cache_rows.cu). Arguments are checked by the entry points
// (cache_ops.cu) before any launcher is called.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lps {

constexpr int kOpSeqs = 256;   // sequences per launch (kernel-parameter arrays)
constexpr int kTreeMax = 64;   // drafted rows per sequence (one 64-bit ancestor mask)
constexpr int kMaxGroup = 16;  // query heads per kv head

// Attention of rows (token, query head) against keys of the same sequence.
// prompt: sequence s holds len[s] packed tokens from tok0[s], and token t sees
// the tokens [0, t] of its sequence. tree: sequence s has len[s] drafted rows
// whose keys lie in cache rows pos[s] .., and row t sees the rows [0, pos[s])
// and its own chain of parents.
struct TileAttnParams {
  CUtensorMap tmap_q;  // [batch][token][head][hd], boxes of one tile's rows
  CUtensorMap tmap_k;  // [batch][head][row][hd]
  CUtensorMap tmap_v;
  const void* k;       // element (s, j, g): k + s * k_seq + (tok0 + j) * k_row + g * k_head
  const void* v;
  void* out;           // element (s, t, h): out + s * o_seq + (tok0 + t) * o_tok + h * o_head
  long long k_seq, k_row, k_head;
  long long v_seq, v_row, v_head;
  long long o_seq, o_tok, o_head;
  const int* parents;  // tree: device [n_seqs][width]
  int width;
  int nkv, group, n_seqs;
  float scale_log2;    // scale * log2(e)
  int wide_out;        // out's rows are 32-byte aligned
  long long wait_limit;  // cycles a wait may take before it reports an error
  int tok0[kOpSeqs], len[kOpSeqs], pos[kOpSeqs];
  // set by the plan
  int tpt;             // tokens of a tile: 128 / group
  int solo;            // tree: one tile, its key blocks dealt to the two slots
  int cluster;         // tree: CTAs that share a sequence's keys
  int item0[kOpSeqs];  // first work item of each sequence; an item is nkv CTAs (tree: clusters)
};
// Set the plan (which puts the longest sequences first) and the launch's CTAs
// (0: nothing to do). A tree's tok0 becomes the sequences' places in the batch.
long long tile_prompt_plan(TileAttnParams& p);
cudaError_t tile_tree_plan(TileAttnParams& p, bool bf16, int hd, long long* ctas);
cudaError_t launch_tile_prompt(const TileAttnParams& p, long long ctas, bool bf16, int hd, cudaStream_t s);
cudaError_t launch_tile_tree(const TileAttnParams& p, long long ctas, bool bf16, int hd, cudaStream_t s);
// Synchronize the stream, then read and clear the kernels' status words.
cudaError_t tile_attn_status(int* status, cudaStream_t s);

// Packed rows of sequence s, tokens [off[s], off[s + 1]), to the cache rows
// start[s] .. of sequence s; elements of 2 bytes, moved 16 bytes at a time.
struct AppendParams {
  const uint4* k;
  const uint4* v;
  uint4* kc;           // [n_seqs][nkv][max_ctx][hd]
  uint4* vc;
  long long k_tok, k_head, v_tok, v_head;  // in 16-byte units
  int nkv, chunks, max_ctx, n_seqs;        // chunks: 16-byte units per row
  int off[kOpSeqs + 1], start[kOpSeqs];
};
cudaError_t launch_append(const AppendParams& p, cudaStream_t s);

// Row pos[b] + path[b][i] to row pos[b] + i, i < accepted[b], in place.
struct AcceptParams {
  uint4* kc;           // [layers][batch][nkv][max_ctx][hd]
  uint4* vc;
  const int* path;     // device [batch][width], strictly ascending
  const int* accepted; // device [batch]
  int layers, batch, nkv, max_ctx, chunks, width;
  int pos[kOpSeqs];
};
cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s);

}  // namespace lps
