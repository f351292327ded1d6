// Argument blocks and launchers of the paged-cache serving kernels: step
// tables, rotary embedding with the page store, attention of drafted trees
// over the pages, and the rules on logits.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace tpk {

constexpr int kMaxStepSeqs = 8192;   // the step tables keep three words a sequence in shared memory
constexpr int kMaxTreeTokens = 256;  // new tokens a sequence with tree masks, and in tree attention
constexpr int kMaxTreeWords = kMaxTreeTokens / 64;
constexpr int kMaxLength = 1 << 30;  // tokens of a sequence, rows of a step
constexpr int kMaxVocab = 1 << 30;   // logits of a row
constexpr size_t kStepTicketBytes = 256;  // the step tables' part of the workspace

struct StepTablesArgs {
  int n_pages, ld_table;
  int page_size;
  FastDiv div_page;
  int32_t* table;
  int32_t* free_ring;
  const int32_t* free_state;
  int32_t* free_next;
  int n_seqs, n_tokens, max_new, cap;  // cap: no length is larger
  int tree_words;
  const int32_t *old_lens, *new_lens, *parents;
  int32_t *q_start, *slots, *positions, *token_seq;
  uint64_t* tree_mask;
  int* ticket;  // zero on entry and exit
  int* status;
};
cudaError_t launch_step_tables(const StepTablesArgs& a, cudaStream_t st);

struct CacheAppendArgs {
  const uint16_t* qkv;
  int64_t rank_stride;
  int n_r;                    // columns of one rank's qkv row
  int M;
  const int32_t *positions, *slots;
  int n_pages, page_size;
  FastDiv div_page;
  uint16_t *k, *v, *q;        // q may be null
  int64_t ld_q;
  int n_heads, n_kv, head_dim, q_per_rank, kv_r, kv_replicas;
  FastDiv div_q, div_kv;      // by q_per_rank, kv_r
  const float2* rope;
  int max_positions;
  int* status;
};
cudaError_t launch_cache_append(const CacheAppendArgs& a, int num_sms, cudaStream_t st);

struct TreeAttnArgs {
  CUtensorMap tmK, tmV;       // (d, page_size, copies * n_pages * kv_r), box (64, box_rows, 1)
  CUtensorMap tmQ;            // (d, n_heads, n_tokens), box (64, group, tile_toks)
  int tile_toks, tile_rows;   // tokens of a query tile (128 / group), its rows
  int box_rows;               // keys a box brings: a power of two that divides page_size
  int slices;                 // the third extent: coordinates from here on read zeros
  uint16_t* o;
  int64_t ld_o;
  const uint16_t* v;
  int n_pages, page_size, ld_table;
  FastDiv div_page;
  const int32_t* table;
  int n_seqs, n_tokens, max_new, cap;  // cap: no sequence's old + new tokens are more
  const int32_t *old_lens, *q_start;
  const uint64_t* tree_mask;  // null: chains
  int tree_words;
  int n_heads, n_kv, kv_r, group, head_dim;
  FastDiv div_group;
  float scale_log2;           // log2(e) / sqrt(d)
  int kv_once;                // 1: no sequence has more than one query tile, K and V are read once
  int grid;
  float* partials;            // [grid][2][d / 4][128][4]
  float2* ml;                 // [grid][2][128]
  int* tickets;               // [n_seqs][n_kv][q_tiles_max], zero on entry and exit
  int q_tiles_max;            // query tiles of max_new tokens
  int* status;
};
constexpr int kTreeRows = 128;  // query rows (tokens x Q heads of a KV head) of a tile
constexpr int kTreeKeys = 64;   // keys of a tile
constexpr int kTreeLoaders = 4;
cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t st);

struct LogitsArgs {
  const uint16_t* logits;
  int64_t ld;
  int S, vocab;
  void* out;
  int64_t ld_out;
  int out_fp32;
  int n_reqs;
  const int32_t* row_req;
  const int32_t* history;
  int64_t ld_history;
  const int32_t *history_lens, *prompt_lens;
  const float *repetition, *frequency, *presence;
  const int32_t* draft_tokens;
  const uint64_t* tree_mask;
  const int32_t* q_start;
  int tree_words;
  int n_biases;
  const int32_t *bias_start, *bias_ids;
  const float* bias_values;
  int n_allowed;
  int64_t ld_allowed;
  const uint32_t* allowed;
  const int32_t* allowed_row;
  int* status;
};
cudaError_t launch_process_logits(const LogitsArgs& a, int num_sms, cudaStream_t st);

}  // namespace tpk
