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
  const int32_t* holders;     // null: no page is shared
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

constexpr int kMaxBeams = 32;      // of a request
constexpr int kMaxBeamCands = 64;  // of a request
constexpr int kMaxEnds = 8;

// The K best logits of a part of a row, and some others: (ordered value << 32) | ~token, 0
// behind the last; its largest logit; and its sum of exponentials, of 2^power, times 2^32
// (from the largest logit on where that is far from 0: beam.cu).
struct BeamPart {
  unsigned long long sum;
  float top;
  int power;
};
struct BeamSelectArgs {
  const void* logits;
  int64_t ld;
  int fp32, vocab;
  int n_reqs, width, n_cands, n_ends;
  const int32_t* ends;
  const float* scores;
  float* cand_scores;
  int32_t *cand_rows, *cand_tokens;
  float* next_scores;
  int32_t *parents, *tokens;
  int parts, part_chunks, list;  // parts of a row, chunks and keys of a part
  int per_cell;                // chunks of a cell
  FastDiv div_parts, div_width, div_row_keys, div_cell;  // by parts, width, parts * list, per_cell
  BeamPart* sums;             // [rows][parts]
  unsigned long long* lists;  // [rows][parts][list]
  int* tickets;               // [n_reqs], zero on entry and exit
  int* status;
};
// The most parts that up to `rows` rows are cut into, all together.
int64_t beam_parts_all(int64_t rows, int num_sms);
// The most keys of a part's list.
int beam_list_most(int cands);
cudaError_t launch_beam_select(BeamSelectArgs a, int num_sms, cudaStream_t st);

struct BeamAdvanceArgs {
  int n_rows;
  const int32_t *parents, *tokens, *history;
  int64_t ld, ld_out, room, room_out;  // row strides; ids that a row has room for
  const int32_t* lens;
  int32_t *out, *lens_out;
  int* status;
};
constexpr int kAdvIds = 4096;  // of a CTA
inline int64_t beam_advance_pieces(int64_t room) { return (room + kAdvIds - 1) / kAdvIds; }  // of a row
cudaError_t launch_beam_advance(const BeamAdvanceArgs& a, cudaStream_t st);

// What the fork and the compaction keep of a page in the workspace.
struct PageNote {
  uint32_t refs;   // how often rows name it; fork: afterwards, as a full page.  Zero between calls
  uint32_t first;  // fork: 1 + n_seqs - the first row that goes on writing to it, or 1 (held before).
                   // Zero between calls
  int32_t move;    // compaction: of a page that moves, its move and its rows
  int32_t rows;
};
constexpr int kShareCtas = 1024;  // CTAs at most
struct ShareHeader {
  unsigned arrived[3], bad;  // CTAs at each barrier; the verdict (the first and it are zero between calls)
  int2 counts[kShareCtas];         // of each CTA's pages and rows
  int32_t open[kMaxStepSeqs];      // fork: the page that each row goes on writing to, or -1
};
constexpr size_t kShareNotes = 49152;  // where the notes begin in the workspace
static_assert(sizeof(ShareHeader) <= kShareNotes, "the notes lie behind the header");

struct ForkArgs {
  int n_pages, ld_table, page_size;
  FastDiv div_page;
  const int32_t* table;
  int32_t* free_ring;
  const int32_t* free_state;
  int32_t *free_next, *holders;
  const int32_t* old_holders;  // not null: holders is another buffer, of which every page is written
  int n_seqs, cap;
  const int32_t *old_lens, *src, *keep_lens;
  int32_t *table_out, *new_lens, *moves, *n_moves;
  int col_tiles, page_share, row_share;  // tiles along a table row; pages and rows of a CTA
  FastDiv div_cols;                      // by col_tiles
  ShareHeader* head;
  PageNote* notes;
  int* status;
};
cudaError_t launch_fork_pages(const ForkArgs& a, int num_sms, cudaStream_t st);

struct CompactArgs {
  int n_pages, ld_table, page_size;
  FastDiv div_page;
  const int32_t *table, *ring, *free_state;
  int32_t *table_out, *ring_out, *free_next, *holders;
  const int32_t* old_holders;  // not null: holders is another buffer
  int n_seqs, cap;
  const int32_t* lens;
  int32_t *moves, *n_moves;
  int col_tiles, page_share, row_share;  // as in a fork
  FastDiv div_cols;
  ShareHeader* head;
  PageNote* notes;
  int* status;
};
cudaError_t launch_compact_pages(const CompactArgs& a, int num_sms, cudaStream_t st);

constexpr int kCopyLayers = 128;  // of a launch
struct CopyPagesArgs {
  int n_pages, page_size, max_moves;
  int row;                    // 16-byte words of a token's head
  int copies, kv_r, layers;
  FastDiv div_heads, div_kv;  // by copies * kv_r, by kv_r
  int run_pieces, move_pieces;  // of a head's page, of a move
  FastDiv div_run, div_move;
  const int32_t *moves, *n_moves;
  int* status;
  uint4* pools[2 * kCopyLayers];
};
cudaError_t launch_copy_pages(CopyPagesArgs a, int num_sms, cudaStream_t st);

}  // namespace tpk
