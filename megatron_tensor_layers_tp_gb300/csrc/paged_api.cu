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
int length_cap(const tp_pages_t* p, const tp_step_t* s) {
  return (int)std::min({(int64_t)s->max_ctx, (int64_t)p->ld_table * p->page_size,
                        (int64_t)kMaxLength});
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
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

// Bytes from the first to past the last element of [rows, cols] at a row stride.
int64_t span_bytes(int64_t rows, int64_t ld, int64_t cols, int elem) {
  return ((rows - 1) * ld + cols) * elem;
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
    a.n_seqs = step->n_seqs;
    a.n_tokens = step->n_tokens;
    a.max_new = step->max_new;
    a.cap = length_cap(pages, step);
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
    a.cap = length_cap(pages, step);
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

}  // extern "C"
