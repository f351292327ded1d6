// Host side of the paged-cache serving calls declared in include/tp.h:
// argument checks, workspace layout and kernel dispatch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "internal.h"
#include "model.h"
#include "paged.h"
#include "tp.h"

using namespace tpk;

namespace {

// The entry points run on the model's device and let no C++ exception out.
template <class F>
tp_status guarded(const tp_model* m, F&& f) {
  int dev = -1;
  if (!m) return TP_ERR_ARG;
  if (cudaGetDevice(&dev) != cudaSuccess) return TP_ERR_CUDA;
  if (dev != m->device) return TP_ERR_ARG;
  try {
    return f();
  } catch (...) {
    return TP_ERR_OOM;
  }
}

tp_status check_pages(const tp_pages_t* p) {
  if (!p || p->n_pages < 1 || p->page_size < 1) return TP_ERR_ARG;
  if (p->page_size % 8 || p->page_size > 65536 ||
      (int64_t)p->n_pages * p->page_size > INT32_MAX)
    return TP_ERR_UNSUPPORTED;
  return TP_OK;
}

// The longest sequence a table row and the caller's bound allow (the kernels
// round lengths up to key tiles and pages in 32 bits).
int length_cap(const tp_pages_t* p, int32_t max_ctx) {
  return (int)std::min({(int64_t)max_ctx, (int64_t)p->ld_table * p->page_size,
                        (int64_t)kMaxLength});
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

struct Span {
  const void* p;
  int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  return a.bytes > 0 && b.bytes > 0 && overlap(a.p, a.bytes, b.p, b.bytes);
}

// Tokens of a query tile, and query tiles of n new tokens.
int tile_tokens(const tp_model* m) { return kTreeRows / (m->cfg.n_heads / m->cfg.n_kv_heads); }
int query_tiles(const tp_model* m, int n) { return cdiv(n, tile_tokens(m)); }

// Workspace regions: the step tables' ticket, then tree attention's (m, l),
// pieces and tickets.  (Steps of more new tokens than tree attention takes,
// prompts, only use the first.)  The tickets, whose number is the step's, lie
// last: a workspace also serves smaller steps, and what one step writes must
// not lie where another expects tickets of zero.
struct StepWs {
  size_t ml, partials, tickets, total;
};
StepWs step_ws(const tp_model* m, int n_seqs, int max_new) {
  StepWs w;
  const size_t pieces = (size_t)m->num_sms * 2 * kTreeRows;
  const int tiles = query_tiles(m, std::min(max_new, kMaxTreeTokens));
  w.ml = kStepTicketBytes;
  w.partials = align_up(w.ml + pieces * sizeof(float2), 256);
  w.tickets = align_up(w.partials + pieces * m->cfg.head_dim * sizeof(float), 256);
  w.total = w.tickets + (size_t)n_seqs * m->cfg.n_kv_heads * tiles * sizeof(int);
  return w;
}

// The selection's limits; its workspace: the requests' tickets (first, and as many for
// every call, since what one call writes must not lie where another expects zeros), then
// sums and lists of the rows' parts.
bool beam_sizes(int n_reqs, int width, int n_cands) {
  return n_reqs >= 1 && n_reqs <= kMaxStepSeqs && width >= 1 && width <= kMaxBeams &&
         n_cands >= width && n_cands <= kMaxBeamCands;
}
struct BeamWs {
  size_t sums, lists, total;
};
BeamWs beam_ws(const tp_model* m, int n_reqs, int width, int n_cands) {
  const size_t parts = beam_parts_all((int64_t)n_reqs * width, m->num_sms);
  BeamWs w;
  w.sums = kMaxStepSeqs * sizeof(int);
  w.lists = align_up(w.sums + parts * sizeof(BeamPart), 256);
  w.total = w.lists + parts * beam_list_most(n_cands) * sizeof(unsigned long long);
  return w;
}

// Bytes from the first to past the last element of [rows, cols] at a row stride.
int64_t span_bytes(int64_t rows, int64_t ld, int64_t cols, int elem) {
  return ((rows - 1) * ld + cols) * elem;
}

// Whether rows of 32-bit words overlap: `cols` of each `ld` from p on.  Rows at one stride may
// lie between each other's.
struct Rows {
  const int32_t* p;
  int64_t ld, cols;
};
bool overlap(const Rows& a, const Rows& b, int64_t rows) {
  if (!overlap(a.p, span_bytes(rows, a.ld, a.cols, 4), b.p, span_bytes(rows, b.ld, b.cols, 4))) return false;
  if (a.ld != b.ld) return true;
  const int64_t ld = a.ld * 4;
  const int64_t at = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % ld;
  const int64_t behind = at < 0 ? at + ld : at;  // of a row of a: where one of b begins
  return behind < a.cols * 4 || behind + b.cols * 4 > ld;
}

// Bytes of a layer's K or V pages.
int64_t cache_bytes(const tp_config_t& c, const tp_pages_t* p) {
  return (int64_t)c.n_kv_heads * p->n_pages * p->page_size * c.head_dim * 2;
}

}  // namespace

extern "C" {

size_t tp_step_workspace_bytes(const tp_model* m, int32_t n_seqs, int32_t max_new) {
  if (!m || n_seqs < 1 || n_seqs > kMaxStepSeqs || max_new < 0) return 0;
  return step_ws(m, n_seqs, max_new).total;
}

tp_status tp_step_tables(const tp_model* m, const tp_pages_t* pages, const tp_step_t* step,
                         void* ws, size_t ws_bytes, void* stream) {
  return guarded(m, [&]() -> tp_status {
    tp_status s = check_pages(pages);
    if (s != TP_OK) return s;
    if (!step || step->n_seqs < 1 || step->n_tokens < 0 || step->max_new < 0 || step->max_ctx < 0 ||
        pages->ld_table < 1 || !pages->table || !pages->free_ring || !pages->free_state ||
        !pages->free_next || !step->old_lens || !step->new_lens || !step->q_start)
      return TP_ERR_ARG;
    if (step->n_tokens > 0 && (!step->slots || !step->positions || !step->token_seq))
      return TP_ERR_ARG;
    if (step->tree_mask && step->tree_words < 1) return TP_ERR_ARG;
    if (step->n_seqs > kMaxStepSeqs || step->n_tokens > kMaxLength ||
        ((step->tree_mask || step->parents) && step->max_new > kMaxTreeTokens) ||
        (step->tree_mask &&
         (step->tree_words > kMaxTreeWords || step->max_new > 64 * step->tree_words)))
      return TP_ERR_UNSUPPORTED;
    if (!ws || !aligned16(ws) ||
        ws_bytes < tp_step_workspace_bytes(m, step->n_seqs, step->max_new))
      return TP_ERR_WORKSPACE;
    StepTablesArgs a;
    memset(&a, 0, sizeof(a));
    a.n_pages = pages->n_pages;
    a.ld_table = pages->ld_table;
    a.page_size = pages->page_size;
    a.div_page = make_fastdiv((uint32_t)pages->page_size);
    a.table = pages->table;
    a.free_ring = pages->free_ring;
    a.free_state = pages->free_state;
    a.free_next = pages->free_next;
    a.holders = pages->holders;
    a.n_seqs = step->n_seqs;
    a.n_tokens = step->n_tokens;
    a.max_new = step->max_new;
    a.cap = length_cap(pages, step->max_ctx);
    a.tree_words = step->tree_words;
    a.old_lens = step->old_lens;
    a.new_lens = step->new_lens;
    a.parents = step->parents;
    a.q_start = step->q_start;
    a.slots = step->slots;
    a.positions = step->positions;
    a.token_seq = step->token_seq;
    a.tree_mask = step->tree_mask;
    a.ticket = static_cast<int*>(ws);
    a.status = m->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(m, "step_tables", st, [&] { return launch_step_tables(a, st); }));
  });
}

tp_status tp_cache_append(const tp_model* m, const tp_bf16* qkv, int64_t rank_stride, int32_t M,
                          const int32_t* positions, const int32_t* slots,
                          const tp_pages_t* pages, tp_bf16* k, tp_bf16* v, tp_bf16* q,
                          int64_t ld_q, void* stream) {
  return guarded(m, [&]() -> tp_status {
    if (M < 0) return TP_ERR_ARG;
    tp_status s = check_pages(pages);
    if (s != TP_OK) return s;
    if (M == 0) return TP_OK;
    const tp_config_t& c = m->cfg;
    const int n_r = (c.q_heads_per_rank + 2 * c.kv_heads_per_rank) * c.head_dim;
    const int nhd = c.n_heads * c.head_dim;
    if (!qkv || !positions || !slots || !k || !v || !aligned16(qkv) || !aligned16(k) ||
        !aligned16(v) || rank_stride % 8 || rank_stride < (int64_t)M * n_r)
      return TP_ERR_ARG;
    if (q && (!aligned16(q) || ld_q % 8 || ld_q < nhd)) return TP_ERR_ARG;
    const int64_t in = ((c.attn_tp - 1) * rank_stride + (int64_t)M * n_r) * 2;
    const int64_t cache = cache_bytes(c, pages);
    const int64_t out = q ? span_bytes(M, ld_q, nhd, 2) : 0;
    if (overlap(k, cache, v, cache) || overlap(qkv, in, k, cache) || overlap(qkv, in, v, cache) ||
        (q && (overlap(q, out, qkv, in) || overlap(q, out, k, cache) || overlap(q, out, v, cache))))
      return TP_ERR_ARG;
    CacheAppendArgs a;
    memset(&a, 0, sizeof(a));
    a.qkv = qkv;
    a.rank_stride = rank_stride;
    a.n_r = n_r;
    a.M = M;
    a.positions = positions;
    a.slots = slots;
    a.n_pages = pages->n_pages;
    a.page_size = pages->page_size;
    a.div_page = make_fastdiv((uint32_t)pages->page_size);
    a.k = k;
    a.v = v;
    a.q = q;
    a.ld_q = ld_q;
    a.n_heads = c.n_heads;
    a.n_kv = c.n_kv_heads;
    a.head_dim = c.head_dim;
    a.q_per_rank = c.q_heads_per_rank;
    a.kv_r = c.kv_heads_per_rank;
    a.kv_replicas = c.kv_replicas;
    a.div_q = make_fastdiv((uint32_t)a.q_per_rank);
    a.div_kv = make_fastdiv((uint32_t)a.kv_r);
    a.rope = m->rope;
    a.max_positions = c.max_positions;
    a.status = m->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(
        launch(m, "cache_append", st, [&] { return launch_cache_append(a, m->num_sms, st); }));
  });
}

tp_status tp_tree_attention(const tp_model* m, const tp_bf16* q, int64_t ld_q, tp_bf16* o,
                            int64_t ld_o, const tp_pages_t* pages, const tp_step_t* step,
                            const tp_bf16* k, const tp_bf16* v, void* ws, size_t ws_bytes,
                            void* stream) {
  return guarded(m, [&]() -> tp_status {
    tp_status s = check_pages(pages);
    if (s != TP_OK) return s;
    if (!step || step->n_seqs < 1 || step->n_tokens < 0 || step->max_new < 0 || step->max_ctx < 0 ||
        pages->ld_table < 1 || !pages->table || !step->old_lens || !step->q_start)
      return TP_ERR_ARG;
    if (step->tree_mask && step->tree_words < 1) return TP_ERR_ARG;
    if (step->n_seqs > kMaxStepSeqs || step->n_tokens > kMaxLength || step->max_new > kMaxTreeTokens ||
        (step->tree_mask &&
         (step->tree_words > kMaxTreeWords || step->max_new > 64 * step->tree_words)))
      return TP_ERR_UNSUPPORTED;
    if (step->n_tokens == 0 || step->max_new == 0) return TP_OK;
    const tp_config_t& c = m->cfg;
    const int nhd = c.n_heads * c.head_dim;
    if (!q || !o || !k || !v || !aligned16(q) || !aligned16(o) || !aligned16(k) || !aligned16(v) ||
        ld_q % 8 || ld_o % 8 || ld_q < nhd || ld_o < nhd)
      return TP_ERR_ARG;
    const uint64_t slices =
        (uint64_t)c.kv_copies * pages->n_pages * c.kv_heads_per_rank, d = c.head_dim;
    if (slices >= INT32_MAX) return TP_ERR_UNSUPPORTED;  // a tensor map coordinate
    const int64_t cache = cache_bytes(c, pages), out = span_bytes(step->n_tokens, ld_o, nhd, 2);
    if (overlap(q, span_bytes(step->n_tokens, ld_q, nhd, 2), o, out) || overlap(o, out, k, cache) ||
        overlap(o, out, v, cache))
      return TP_ERR_ARG;
    if (!ws || !aligned16(ws) ||
        ws_bytes < tp_step_workspace_bytes(m, step->n_seqs, step->max_new))
      return TP_ERR_WORKSPACE;
    TreeAttnArgs a;
    memset(&a, 0, sizeof(a));
    a.o = o;
    a.ld_o = ld_o;
    a.v = v;
    // boxes of as many keys as divide the page (and the key tile)
    a.box_rows = 8;
    while (a.box_rows < kTreeKeys && pages->page_size % (2 * a.box_rows) == 0) a.box_rows *= 2;
    a.slices = (int)slices;
    if (!make_tmap(&a.tmK, k, d, pages->page_size, slices, d * 2, pages->page_size * d * 2, a.box_rows) ||
        !make_tmap(&a.tmV, v, d, pages->page_size, slices, d * 2, pages->page_size * d * 2, a.box_rows))
      return TP_ERR_CUDA;
    a.n_pages = pages->n_pages;
    a.page_size = pages->page_size;
    a.ld_table = pages->ld_table;
    a.div_page = make_fastdiv((uint32_t)pages->page_size);
    a.table = pages->table;
    a.n_seqs = step->n_seqs;
    a.n_tokens = step->n_tokens;
    a.max_new = step->max_new;
    a.cap = length_cap(pages, step->max_ctx);
    a.old_lens = step->old_lens;
    a.q_start = step->q_start;
    a.tree_mask = step->tree_mask;
    a.tree_words = step->tree_words;
    a.n_heads = c.n_heads;
    a.n_kv = c.n_kv_heads;
    a.kv_r = c.kv_heads_per_rank;
    a.group = c.n_heads / c.n_kv_heads;
    a.head_dim = c.head_dim;
    a.div_group = make_fastdiv((uint32_t)a.group);
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.head_dim));
    a.tile_toks = tile_tokens(m);
    a.tile_rows = a.tile_toks * a.group;
    a.kv_once = step->max_new <= a.tile_toks;
    if (!make_tmap(&a.tmQ, q, d, c.n_heads, step->n_tokens, d * 2, ld_q * 2, a.group, nullptr,
                   a.tile_toks))
      return TP_ERR_CUDA;
    a.grid = m->num_sms;
    const StepWs w = step_ws(m, step->n_seqs, step->max_new);
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.tickets = reinterpret_cast<int*>(base + w.tickets);
    a.q_tiles_max = query_tiles(m, step->max_new);
    a.ml = reinterpret_cast<float2*>(base + w.ml);
    a.partials = reinterpret_cast<float*>(base + w.partials);
    a.status = m->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(launch(m, "tree_attn", st, [&] { return launch_tree_attn(a, st); }));
  });
}

tp_status tp_process_logits(const tp_model* m, const tp_bf16* logits, int64_t ld_logits,
                            int32_t S, const tp_logit_rules_t* rules, void* out, int64_t ld_out,
                            int32_t out_fp32, void* stream) {
  return guarded(m, [&]() -> tp_status {
    if (S < 0 || !rules || out_fp32 < 0 || out_fp32 > 1) return TP_ERR_ARG;
    if (S == 0) return TP_OK;
    const tp_logit_rules_t& r = *rules;
    const int V = m->cfg.vocab;
    const uintptr_t elem = out_fp32 ? 4 : 2;
    if (V < 1 || !logits || !out || reinterpret_cast<uintptr_t>(logits) % 2 ||
        reinterpret_cast<uintptr_t>(out) % elem || ld_logits < V || ld_out < V || r.n_reqs < 1)
      return TP_ERR_ARG;
    if (!r.row_req && r.n_reqs < S) return TP_ERR_ARG;
    if (r.history && (!r.history_lens || r.ld_history < 0)) return TP_ERR_ARG;
    if ((r.draft_tokens != nullptr) != (r.tree_mask != nullptr) ||
        (r.draft_tokens != nullptr) != (r.q_start != nullptr))
      return TP_ERR_ARG;
    if (r.draft_tokens && (r.tree_words < 1 || r.tree_words > kMaxTreeWords)) return TP_ERR_ARG;
    if (r.bias_start && (r.n_biases < 0 || (r.n_biases > 0 && (!r.bias_ids || !r.bias_values))))
      return TP_ERR_ARG;
    if (r.allowed && (r.ld_allowed < (V + 31) / 32 || r.n_allowed < 1 ||
                      (!r.allowed_row && r.n_allowed < S)))
      return TP_ERR_ARG;
    const bool in_place = !out_fp32 && out == logits && ld_out == ld_logits;
    if (!in_place && overlap(logits, span_bytes(S, ld_logits, V, 2), out,
                             span_bytes(S, ld_out, V, out_fp32 ? 4 : 2)))
      return TP_ERR_ARG;
    if (V > kMaxVocab || (int64_t)S * ((V + 1023) / 1024) > INT32_MAX) return TP_ERR_UNSUPPORTED;
    LogitsArgs a;
    memset(&a, 0, sizeof(a));
    a.logits = logits;
    a.ld = ld_logits;
    a.S = S;
    a.vocab = V;
    a.out = out;
    a.ld_out = ld_out;
    a.out_fp32 = out_fp32;
    a.n_reqs = r.n_reqs;
    a.row_req = r.row_req;
    a.history = r.history;
    a.ld_history = r.ld_history;
    a.history_lens = r.history_lens;
    a.prompt_lens = r.prompt_lens;
    a.repetition = r.repetition;
    a.frequency = r.frequency;
    a.presence = r.presence;
    a.draft_tokens = r.draft_tokens;
    a.tree_mask = r.tree_mask;
    a.q_start = r.q_start;
    a.tree_words = r.tree_words;
    a.n_biases = r.n_biases;
    a.bias_start = r.bias_start;
    a.bias_ids = r.bias_ids;
    a.bias_values = r.bias_values;
    a.n_allowed = r.n_allowed;
    a.ld_allowed = r.ld_allowed;
    a.allowed = r.allowed;
    a.allowed_row = r.allowed_row;
    a.status = m->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(
        launch(m, "process_logits", st, [&] { return launch_process_logits(a, m->num_sms, st); }));
  });
}

size_t tp_beam_workspace_bytes(const tp_model* m, int32_t n_reqs, int32_t width,
                               int32_t n_cands) {
  if (!m || !beam_sizes(n_reqs, width, n_cands)) return 0;
  return beam_ws(m, n_reqs, width, n_cands).total;
}

tp_status tp_beam_select(const tp_model* m, const void* logits, int64_t ld_logits, int32_t fp32,
                         const tp_beams_t* beams, void* ws, size_t ws_bytes, void* stream) {
  return guarded(m, [&]() -> tp_status {
    if (!beams || fp32 < 0 || fp32 > 1) return TP_ERR_ARG;
    const tp_beams_t& b = *beams;
    const int V = m->cfg.vocab;
    const uintptr_t elem = fp32 ? 4 : 2;
    if (b.n_reqs < 1 || b.width < 1 || b.n_cands < b.width || b.n_ends < 0 || V < 1 || !logits ||
        reinterpret_cast<uintptr_t>(logits) % elem || ld_logits < V || (b.n_ends > 0 && !b.ends) ||
        !b.scores || !b.cand_scores || !b.cand_rows || !b.cand_tokens || !b.next_scores ||
        !b.parents || !b.tokens)
      return TP_ERR_ARG;
    if (!beam_sizes(b.n_reqs, b.width, b.n_cands) || b.n_ends > kMaxEnds || V > kMaxVocab)
      return TP_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)b.n_reqs * b.width, cands = (int64_t)b.n_reqs * b.n_cands;
    const Span out[6] = {{b.cand_scores, cands * 4}, {b.cand_rows, cands * 4}, {b.cand_tokens, cands * 4},
                         {b.next_scores, rows * 4}, {b.parents, rows * 4}, {b.tokens, rows * 4}};
    const Span in[3] = {{logits, span_bytes(rows, ld_logits, V, (int)elem)}, {b.ends, b.n_ends * 4},
                        {b.scores, rows * 4}};
    for (int i = 0; i < 6; ++i) {
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return TP_ERR_ARG;
      for (int j = 0; j < 3; ++j)
        if (overlap(out[i], in[j]) && !(i == 3 && j == 2 && out[i].p == in[j].p)) return TP_ERR_ARG;
    }
    const BeamWs w = beam_ws(m, b.n_reqs, b.width, b.n_cands);
    if (!ws || !aligned16(ws) || ws_bytes < w.total) return TP_ERR_WORKSPACE;
    BeamSelectArgs a;
    memset(&a, 0, sizeof(a));
    a.logits = logits;
    a.ld = ld_logits;
    a.fp32 = fp32;
    a.vocab = V;
    a.n_reqs = b.n_reqs;
    a.width = b.width;
    a.n_cands = b.n_cands;
    a.n_ends = b.n_ends;
    a.ends = b.ends;
    a.scores = b.scores;
    a.cand_scores = b.cand_scores;
    a.cand_rows = b.cand_rows;
    a.cand_tokens = b.cand_tokens;
    a.next_scores = b.next_scores;
    a.parents = b.parents;
    a.tokens = b.tokens;
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.tickets = reinterpret_cast<int*>(base);
    a.sums = reinterpret_cast<BeamPart*>(base + w.sums);
    a.lists = reinterpret_cast<unsigned long long*>(base + w.lists);
    a.status = m->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(
        launch(m, "beam_select", st, [&] { return launch_beam_select(a, m->num_sms, st); }));
  });
}

tp_status tp_beam_advance(const tp_model* m, int32_t n_rows, const int32_t* parents,
                          const int32_t* tokens, const int32_t* history, int64_t ld_history,
                          const int32_t* lens, int32_t* out, int64_t ld_out, int32_t* lens_out,
                          void* stream) {
  return tp_beam_advance_rooms(m, n_rows, parents, tokens, history, ld_history, ld_history, lens, out,
                               ld_out, ld_out, lens_out, stream);
}

tp_status tp_beam_advance_rooms(const tp_model* m, int32_t n_rows, const int32_t* parents,
                                const int32_t* tokens, const int32_t* history, int64_t ld_history,
                                int64_t room, const int32_t* lens, int32_t* out, int64_t ld_out,
                                int64_t room_out, int32_t* lens_out, void* stream) {
  return guarded(m, [&]() -> tp_status {
    if (n_rows < 0) return TP_ERR_ARG;
    if (n_rows == 0) return TP_OK;
    if (!parents || !tokens || !history || !lens || !out || !lens_out || room < 1 || room > ld_history ||
        room_out < 1 || room_out > ld_out)
      return TP_ERR_ARG;
    const int64_t most = std::min(room, room_out);
    if (most > kMaxLength || n_rows * beam_advance_pieces(most) > INT32_MAX) return TP_ERR_UNSUPPORTED;
    const Span text{history, span_bytes(n_rows, ld_history, room, 4)};
    const Span to{out, span_bytes(n_rows, ld_out, room_out, 4)};
    const Span words[4] = {{parents, n_rows * 4ll}, {tokens, n_rows * 4ll}, {lens, n_rows * 4ll},
                           {lens_out, n_rows * 4ll}};
    if (overlap(Rows{history, ld_history, room}, Rows{out, ld_out, room_out}, n_rows) ||
        overlap(text, words[3]))
      return TP_ERR_ARG;
    for (int i = 0; i < 4; ++i)
      if (overlap(to, words[i]) || (i < 3 && overlap(words[3], words[i]))) return TP_ERR_ARG;
    BeamAdvanceArgs a;
    memset(&a, 0, sizeof(a));
    a.n_rows = n_rows;
    a.parents = parents;
    a.tokens = tokens;
    a.history = history;
    a.ld = ld_history;
    a.ld_out = ld_out;
    a.room = room;
    a.room_out = room_out;
    a.lens = lens;
    a.out = out;
    a.lens_out = lens_out;
    a.status = m->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(
        launch(m, "beam_advance", st, [&] { return launch_beam_advance(a, st); }));
  });
}

size_t tp_share_workspace_bytes(const tp_model* m, int32_t n_pages) {
  if (!m || n_pages < 1 || n_pages > INT32_MAX / 8) return 0;
  return kShareNotes + (size_t)n_pages * sizeof(PageNote);
}

tp_status tp_fork_pages(const tp_model* m, const tp_pages_t* pages, const tp_fork_t* fork,
                        void* ws, size_t ws_bytes, void* stream) {
  return guarded(m, [&]() -> tp_status {
    tp_status s = check_pages(pages);
    if (s != TP_OK) return s;
    if (!fork || fork->n_seqs < 1 || fork->max_ctx < 0 || pages->ld_table < 1 || !pages->table ||
        !pages->free_ring || !pages->free_state || !pages->free_next || !fork->old_lens || !fork->src ||
        !fork->table || !fork->new_lens || !fork->moves || !fork->n_moves ||
        (fork->holders && !pages->holders))
      return TP_ERR_ARG;
    if (fork->n_seqs > kMaxStepSeqs) return TP_ERR_UNSUPPORTED;
    const int64_t n = fork->n_seqs, table = n * pages->ld_table * 4;
    const int64_t ring = pages->n_pages * 4ll;
    const Span out[8] = {{fork->table, table}, {fork->new_lens, n * 4}, {fork->moves, n * 12},
                         {fork->n_moves, 4}, {pages->free_ring, ring}, {pages->free_next, 8},
                         {pages->holders, pages->holders ? ring : 0}, {fork->holders, fork->holders ? ring : 0}};
    const Span in[5] = {{pages->table, table}, {fork->old_lens, n * 4}, {fork->src, n * 4},
                        {fork->keep_lens, fork->keep_lens ? n * 4 : 0}, {pages->free_state, 8}};
    for (int i = 0; i < 8; ++i) {
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return TP_ERR_ARG;
      for (int j = 0; j < 5; ++j)
        if (overlap(out[i], in[j]) && !(i == 5 && j == 4 && out[i].p == in[j].p)) return TP_ERR_ARG;
    }
    if (!ws || !aligned16(ws) || ws_bytes < tp_share_workspace_bytes(m, pages->n_pages))
      return TP_ERR_WORKSPACE;
    ForkArgs a;
    memset(&a, 0, sizeof(a));
    a.n_pages = pages->n_pages;
    a.ld_table = pages->ld_table;
    a.page_size = pages->page_size;
    a.div_page = make_fastdiv((uint32_t)pages->page_size);
    a.table = pages->table;
    a.free_ring = pages->free_ring;
    a.free_state = pages->free_state;
    a.free_next = pages->free_next;
    a.holders = fork->holders ? fork->holders : pages->holders;
    a.old_holders = fork->holders ? pages->holders : nullptr;
    a.n_seqs = fork->n_seqs;
    a.cap = length_cap(pages, fork->max_ctx);
    a.old_lens = fork->old_lens;
    a.src = fork->src;
    a.keep_lens = fork->keep_lens;
    a.table_out = fork->table;
    a.new_lens = fork->new_lens;
    a.moves = fork->moves;
    a.n_moves = fork->n_moves;
    a.head = static_cast<ShareHeader*>(ws);
    a.notes = reinterpret_cast<PageNote*>(static_cast<uint8_t*>(ws) + kShareNotes);
    a.status = m->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(
        launch(m, "fork_pages", st, [&] { return launch_fork_pages(a, m->num_sms, st); }));
  });
}

tp_status tp_compact_pages(const tp_model* m, const tp_pages_t* pages, const tp_pages_t* to,
                           int32_t n_seqs, int32_t max_ctx, const int32_t* lens,
                           int32_t* moves, int32_t max_moves, int32_t* n_moves, void* ws,
                           size_t ws_bytes, void* stream) {
  return guarded(m, [&]() -> tp_status {
    tp_status s = check_pages(pages);
    if (s != TP_OK) return s;
    if (!to || n_seqs < 1 || max_ctx < 0 || pages->ld_table < 1 || !pages->table || !pages->free_ring ||
        !pages->free_state || to->n_pages != pages->n_pages || to->page_size != pages->page_size ||
        to->ld_table != pages->ld_table || !to->table || !to->free_ring || !to->free_next || !lens ||
        (!moves && max_moves > 0) || !n_moves || max_moves < pages->n_pages / 2)
      return TP_ERR_ARG;
    if (n_seqs > kMaxStepSeqs) return TP_ERR_UNSUPPORTED;
    const int64_t n = n_seqs, table = n * pages->ld_table * 4, ring = pages->n_pages * 4ll;
    // (in and out of the same index may be the same buffer)
    const Span out[6] = {{to->table, table}, {to->free_ring, ring}, {to->free_next, 8},
                         {to->holders, to->holders ? ring : 0}, {moves, max_moves * 12ll}, {n_moves, 4}};
    const Span in[5] = {{pages->table, table}, {pages->free_ring, ring}, {pages->free_state, 8},
                        {pages->holders, pages->holders ? ring : 0}, {lens, n * 4}};
    for (int i = 0; i < 6; ++i) {
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return TP_ERR_ARG;
      for (int j = 0; j < 5; ++j)
        if (overlap(out[i], in[j]) && !(i == j && i < 4 && out[i].p == in[j].p)) return TP_ERR_ARG;
    }
    if (!ws || !aligned16(ws) || ws_bytes < tp_share_workspace_bytes(m, pages->n_pages))
      return TP_ERR_WORKSPACE;
    CompactArgs a;
    memset(&a, 0, sizeof(a));
    a.n_pages = pages->n_pages;
    a.ld_table = pages->ld_table;
    a.page_size = pages->page_size;
    a.div_page = make_fastdiv((uint32_t)pages->page_size);
    a.table = pages->table;
    a.ring = pages->free_ring;
    a.free_state = pages->free_state;
    a.table_out = to->table;
    a.ring_out = to->free_ring;
    a.free_next = to->free_next;
    a.holders = to->holders;
    a.old_holders = to->holders && to->holders != pages->holders ? pages->holders : nullptr;
    a.n_seqs = n_seqs;
    a.cap = length_cap(pages, max_ctx);
    a.lens = lens;
    a.moves = moves;
    a.n_moves = n_moves;
    a.head = static_cast<ShareHeader*>(ws);
    a.notes = reinterpret_cast<PageNote*>(static_cast<uint8_t*>(ws) + kShareNotes);
    a.status = m->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(
        launch(m, "compact_pages", st, [&] { return launch_compact_pages(a, m->num_sms, st); }));
  });
}

tp_status tp_copy_pages(const tp_model* m, const tp_pages_t* pages, const int32_t* moves,
                        const int32_t* n_moves, int32_t max_moves, int32_t n_layers,
                        tp_bf16* const* k, tp_bf16* const* v, void* stream) {
  return guarded(m, [&]() -> tp_status {
    tp_status s = check_pages(pages);
    if (s != TP_OK) return s;
    if (max_moves < 0 || n_layers < 0) return TP_ERR_ARG;
    if (max_moves == 0 || n_layers == 0) return TP_OK;
    if (!moves || !n_moves || !k || !v) return TP_ERR_ARG;
    for (int i = 0; i < n_layers; ++i)
      if (!k[i] || !v[i] || !aligned16(k[i]) || !aligned16(v[i])) return TP_ERR_ARG;
    // (a launch's pieces of a move are counted in 32 bits)
    if ((int64_t)m->cfg.n_kv_heads * pages->page_size > (1 << 23)) return TP_ERR_UNSUPPORTED;
    CopyPagesArgs a;
    memset(&a, 0, sizeof(a));
    a.n_pages = pages->n_pages;
    a.page_size = pages->page_size;
    a.max_moves = max_moves;
    a.row = m->cfg.head_dim / 8;
    a.copies = m->cfg.kv_copies;
    a.kv_r = m->cfg.kv_heads_per_rank;
    a.div_kv = make_fastdiv((uint32_t)a.kv_r);
    a.div_heads = make_fastdiv((uint32_t)(a.copies * a.kv_r));
    a.moves = moves;
    a.n_moves = n_moves;
    a.status = m->status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    for (int first = 0; first < n_layers; first += kCopyLayers) {
      a.layers = std::min(n_layers - first, kCopyLayers);
      for (int i = 0; i < a.layers; ++i) {
        a.pools[2 * i] = reinterpret_cast<uint4*>(k[first + i]);
        a.pools[2 * i + 1] = reinterpret_cast<uint4*>(v[first + i]);
      }
      s = cuda_status(
          launch(m, "copy_pages", st, [&] { return launch_copy_pages(a, m->num_sms, st); }));
      if (s != TP_OK) return s;
    }
    return TP_OK;
  });
}

}  // extern "C"
