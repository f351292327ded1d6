"""PyTorch-facing wrapper over the C ABI.

PyTorch provides device memory and streams only: every tensor here is a buffer
whose address is handed to the library, and every computation is one of the
library's kernels.  Nothing falls back to PyTorch or the CPU.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Dict, List, Optional, Sequence

import torch

from . import binding as B


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def make_config(hidden, n_heads, n_kv_heads, head_dim, intermediate, vocab, n_layers, t,
                rms_eps=1e-5, rope_theta=10000.0, max_positions=8192,
                attn_dp=1, host_io=0, plain_column_shards=0, prefill_bn=0,
                prefill_cta_pairs=0) -> B.tp_config_t:
    c = B.tp_config_t()
    c.hidden, c.n_heads, c.n_kv_heads, c.head_dim = hidden, n_heads, n_kv_heads, head_dim
    c.intermediate, c.vocab, c.n_layers, c.t = intermediate, vocab, n_layers, t
    c.rms_eps, c.rope_theta, c.max_positions = rms_eps, rope_theta, max_positions
    c.attn_dp = attn_dp
    c.host_io = host_io
    c.plain_column_shards = plain_column_shards
    c.prefill_bn = prefill_bn
    c.prefill_cta_pairs = prefill_cta_pairs
    return c


@dataclass
class Batch:
    """Device-side description of one forward step (see tp_batch_t)."""
    mode: int
    n_seqs: int
    n_tokens: int
    max_q_per_seq: int
    max_ctx: int
    l_max: int
    positions: torch.Tensor
    token_seq: torch.Tensor
    seq_start: Optional[torch.Tensor]
    k_cache: List[torch.Tensor]
    v_cache: List[torch.Tensor]
    sample_rows: Optional[torch.Tensor] = None

    def to_c(self) -> B.tp_batch_t:
        b = B.tp_batch_t()
        b.mode, b.n_seqs, b.n_tokens = self.mode, self.n_seqs, self.n_tokens
        b.max_q_per_seq, b.max_ctx, b.l_max = self.max_q_per_seq, self.max_ctx, self.l_max
        b.seq_start = _ptr(self.seq_start)
        b.positions, b.token_seq = _ptr(self.positions), _ptr(self.token_seq)
        self._k = (ctypes.c_void_p * len(self.k_cache))(*[t.data_ptr() for t in self.k_cache])
        self._v = (ctypes.c_void_p * len(self.v_cache))(*[t.data_ptr() for t in self.v_cache])
        b.k_cache = ctypes.cast(self._k, ctypes.POINTER(ctypes.c_void_p))
        b.v_cache = ctypes.cast(self._v, ctypes.POINTER(ctypes.c_void_p))
        b.sample_rows = _ptr(self.sample_rows)
        b.n_samples = 0 if self.sample_rows is None else int(self.sample_rows.numel())
        return b


def _check(t: torch.Tensor, name: str, dtype, shape, device, rows: bool = False) -> None:
    """Raises ValueError unless t is a tensor on `device` of that dtype and shape (None: any
    size), contiguous; with `rows`, a matrix whose rows are contiguous (any row stride)."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: {dtype} on {device} expected, got {t.dtype} on {t.device}")
    if len(t.shape) != len(shape) or any(w is not None and g != w for g, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if rows:
        if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
            raise ValueError(f"{name}: rows must be contiguous and not overlap")
    elif not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor expected")


def _ld(t: torch.Tensor) -> int:
    """Row stride of a matrix (a single row may carry any)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class PageTable:
    """The page tables of a paged KV cache (see tp_pages_t).

    table [rows, ld] int32, free_ring [n_pages] int32 and free_state [2] int32 (first, count) as
    the C ABI wants them; free_next (default: free_state itself) receives the ring's state after
    step_tables.  holders [n_pages] int32 is needed where rows share pages (fork_pages).  For
    cache_append and copy_pages alone page_size and n_pages suffice, for tree_attention also
    the table.  The tensors' addresses are kept: refresh their contents, not the objects.
    """

    def __init__(self, page_size: int, table: Optional[torch.Tensor] = None,
                 free_ring: Optional[torch.Tensor] = None,
                 free_state: Optional[torch.Tensor] = None,
                 free_next: Optional[torch.Tensor] = None, n_pages: Optional[int] = None,
                 holders: Optional[torch.Tensor] = None):
        if n_pages is None:
            if free_ring is None:
                raise ValueError("n_pages or free_ring is needed")
            n_pages = free_ring.numel()
        if table is not None:
            _check(table, "table", torch.int32, (None, None), table.device)
        if free_ring is not None:
            if table is None or free_state is None:
                raise ValueError("a free_ring comes with its table and free_state")
            if free_next is None:
                free_next = free_state
            _check(free_ring, "free_ring", torch.int32, (n_pages,), table.device)
            _check(free_state, "free_state", torch.int32, (2,), table.device)
            _check(free_next, "free_next", torch.int32, (2,), table.device)
        if holders is not None:
            if table is None:
                raise ValueError("holders come with a table")
            _check(holders, "holders", torch.int32, (n_pages,), table.device)
        self.page_size, self.n_pages = page_size, n_pages
        self.table, self.free_ring = table, free_ring
        self.free_state, self.free_next, self.holders = free_state, free_next, holders
        c = self.c = B.tp_pages_t()
        c.n_pages, c.page_size = n_pages, page_size
        c.ld_table = 0 if table is None else table.shape[1]
        c.table, c.free_ring = _ptr(table), _ptr(free_ring)
        c.free_state, c.free_next = _ptr(free_state), _ptr(free_next)
        c.holders = _ptr(holders)

    @classmethod
    def alloc(cls, n_seqs: int, n_pages: int, page_size: int, max_len: int,
              device="cuda", shared: bool = False) -> "PageTable":
        """An empty table for n_seqs sequences of up to max_len tokens; every page is free.  With
        shared, fork_pages can let its rows share pages."""
        ld = max(1, -(-max_len // page_size))
        return cls(page_size, torch.zeros((n_seqs, ld), dtype=torch.int32, device=device),
                   torch.arange(n_pages, dtype=torch.int32, device=device),
                   torch.tensor([0, n_pages], dtype=torch.int32, device=device),
                   holders=torch.zeros(n_pages, dtype=torch.int32, device=device) if shared else None)

    def with_table(self, table: torch.Tensor, free_state: Optional[torch.Tensor] = None,
                   holders: Optional[torch.Tensor] = None) -> "PageTable":
        """The same pages, ring and ring state behind another table: what a fork writes to.  For a
        proposal that is kept, with the state (its free_next) and the holders that it left."""
        return PageTable(self.page_size, table, self.free_ring,
                         self.free_state if free_state is None else free_state,
                         self.free_next if free_state is None else None, self.n_pages,
                         self.holders if holders is None else holders)


class Step:
    """One step's lengths and index tables (see tp_step_t).

    step_tables fills q_start, slots, positions, token_seq and tree_mask; tree_attention reads
    old_lens, q_start and tree_mask.  What a call does not use may be None.  tree_mask is
    [n_tokens, words] int64 (the 64-bit words' patterns).
    """

    def __init__(self, n_tokens: int, max_new: int, max_ctx: int, old_lens: torch.Tensor,
                 new_lens: Optional[torch.Tensor] = None, parents: Optional[torch.Tensor] = None,
                 q_start: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None,
                 token_seq: Optional[torch.Tensor] = None,
                 tree_mask: Optional[torch.Tensor] = None):
        n, dev = old_lens.numel(), old_lens.device
        for name, t, shape in (("old_lens", old_lens, (n,)), ("new_lens", new_lens, (n,)),
                               ("parents", parents, (n_tokens,)), ("q_start", q_start, (n + 1,)),
                               ("slots", slots, (n_tokens,)), ("positions", positions, (n_tokens,)),
                               ("token_seq", token_seq, (n_tokens,))):
            if t is not None:
                _check(t, name, torch.int32, shape, dev)
        if tree_mask is not None:
            _check(tree_mask, "tree_mask", torch.int64, (n_tokens, None), dev)
        self.n_seqs, self.n_tokens, self.max_new, self.max_ctx = n, n_tokens, max_new, max_ctx
        self.old_lens, self.new_lens, self.parents = old_lens, new_lens, parents
        self.q_start, self.slots, self.positions = q_start, slots, positions
        self.token_seq, self.tree_mask = token_seq, tree_mask
        c = self.c = B.tp_step_t()
        c.n_seqs, c.n_tokens, c.max_new, c.max_ctx = n, n_tokens, max_new, max_ctx
        c.tree_words = 0 if tree_mask is None else tree_mask.shape[1]
        for name in ("old_lens", "new_lens", "parents", "q_start", "slots", "positions",
                     "token_seq", "tree_mask"):
            setattr(c, name, _ptr(getattr(self, name)))

    @classmethod
    def alloc(cls, n_seqs: int, n_tokens: int, max_new: int, max_ctx: int,
              old_lens: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
              parents: Optional[torch.Tensor] = None, tree_words: int = 0,
              device="cuda") -> "Step":
        """A step with its output tables allocated (and lengths of 0 where none are given);
        tree_words > 0 adds the tree masks."""
        def ints(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)
        mask = torch.zeros((n_tokens, tree_words), dtype=torch.int64, device=device) \
            if tree_words else None
        return cls(n_tokens, max_new, max_ctx, ints(n_seqs) if old_lens is None else old_lens,
                   ints(n_seqs) if new_lens is None else new_lens, parents, ints(n_seqs + 1),
                   ints(n_tokens), ints(n_tokens), ints(n_tokens), mask)


class LogitRules:
    """The rules process_logits applies (see tp_logit_rules_t); None leaves a rule out.

    Per request: history [R, ld] int32 with history_lens and prompt_lens [R] int32, repetition,
    frequency and presence [R] float32, biases as bias_start [R+1], bias_ids [n] int32 and
    bias_values [n] float32.  Per row: row_req [S] int32, draft_tokens [S] int32 with tree_mask
    [S, words] int64 and q_start [R+1] int32, allowed [rows, words] int32 (bit patterns) with
    allowed_row [S] int32.
    """

    def __init__(self, row_req=None, history=None, history_lens=None, prompt_lens=None,
                 repetition=None, frequency=None, presence=None, draft_tokens=None, tree_mask=None,
                 q_start=None, bias_start=None, bias_ids=None, bias_values=None, allowed=None,
                 allowed_row=None, n_reqs: Optional[int] = None):
        i32, f32 = torch.int32, torch.float32
        if (history is None) != (history_lens is None):
            raise ValueError("history and history_lens come together")
        if len({draft_tokens is None, tree_mask is None, q_start is None}) > 1:
            raise ValueError("draft_tokens, tree_mask and q_start come together")
        if len({bias_start is None, bias_ids is None, bias_values is None}) > 1:
            raise ValueError("bias_start, bias_ids and bias_values come together")
        per_req = [t.shape[0] for t in (history, prompt_lens, repetition, frequency, presence)
                   if t is not None]
        per_req += [t.numel() - 1 for t in (q_start, bias_start) if t is not None]
        per_row = [t.shape[0] for t in (row_req, draft_tokens, allowed_row) if t is not None]
        if allowed is not None and allowed_row is None:
            per_row.append(allowed.shape[0])
        self.n_rows = per_row[0] if per_row else None
        if n_reqs is None:
            if per_req:
                n_reqs = per_req[0]
            elif self.n_rows is not None and row_req is None:
                n_reqs = self.n_rows
            else:
                raise ValueError("n_reqs is needed: no rule here is given per request")
        if row_req is None and self.n_rows is not None and self.n_rows != n_reqs:
            raise ValueError("rows and requests differ in number: row_req is needed")
        R, S = n_reqs, self.n_rows
        tensors = {"row_req": (row_req, i32, (S,)), "history": (history, i32, (R, None)),
                   "history_lens": (history_lens, i32, (R,)),
                   "prompt_lens": (prompt_lens, i32, (R,)),
                   "repetition": (repetition, f32, (R,)), "frequency": (frequency, f32, (R,)),
                   "presence": (presence, f32, (R,)), "draft_tokens": (draft_tokens, i32, (S,)),
                   "tree_mask": (tree_mask, torch.int64, (S, None)),
                   "q_start": (q_start, i32, (R + 1,)), "bias_start": (bias_start, i32, (R + 1,)),
                   "bias_ids": (bias_ids, i32, (None,)),
                   "bias_values": (bias_values, f32, None if bias_ids is None else bias_ids.shape),
                   "allowed": (allowed, i32, (None, None)), "allowed_row": (allowed_row, i32, (S,))}
        given = [t for t, _, _ in tensors.values() if t is not None]
        self.device = given[0].device if given else None
        self._keep = given
        c = self.c = B.tp_logit_rules_t()
        for name, (t, dtype, shape) in tensors.items():
            if t is not None:
                _check(t, name, dtype, shape, self.device, rows=name == "allowed")
            setattr(c, name, _ptr(t))
        c.n_reqs = R
        c.ld_history = 0 if history is None else history.shape[1]
        c.tree_words = 0 if tree_mask is None else tree_mask.shape[1]
        c.n_biases = 0 if bias_ids is None else bias_ids.numel()
        c.n_allowed = 0 if allowed is None else allowed.shape[0]
        c.ld_allowed = 0 if allowed is None else _ld(allowed)
        # tokens that a grammar row has bits for (rows may lie further apart than they are long)
        self._allowed_tokens = None if allowed is None else 32 * allowed.shape[1]


class Beams:
    """A beam selection's sizes, inputs and outputs (see tp_beams_t).

    Inputs: scores [n_reqs*width] float32 (not finite: the row is not in use), ends [n] int32 (ids
    that end a text).  Outputs, written by beam_select: cand_scores, cand_rows, cand_tokens [n_reqs,
    n_cands], next_scores (which may be scores itself), parents and tokens [n_reqs*width].
    """

    def __init__(self, n_reqs: int, width: int, n_cands: int, scores: torch.Tensor,
                 cand_scores: torch.Tensor, cand_rows: torch.Tensor, cand_tokens: torch.Tensor,
                 next_scores: torch.Tensor, parents: torch.Tensor, tokens: torch.Tensor,
                 ends: Optional[torch.Tensor] = None):
        dev, rows, cands = scores.device, (n_reqs * width,), (n_reqs, n_cands)
        for name, t, dtype, shape in (
                ("scores", scores, torch.float32, rows), ("next_scores", next_scores, torch.float32, rows),
                ("parents", parents, torch.int32, rows), ("tokens", tokens, torch.int32, rows),
                ("cand_scores", cand_scores, torch.float32, cands),
                ("cand_rows", cand_rows, torch.int32, cands),
                ("cand_tokens", cand_tokens, torch.int32, cands)):
            _check(t, name, dtype, shape, dev)
        if ends is not None:
            _check(ends, "ends", torch.int32, (None,), dev)
        self.n_reqs, self.width, self.n_cands, self.ends = n_reqs, width, n_cands, ends
        self.scores, self.next_scores, self.parents, self.tokens = scores, next_scores, parents, tokens
        self.cand_scores, self.cand_rows, self.cand_tokens = cand_scores, cand_rows, cand_tokens
        self.sizes = (n_reqs, width, n_cands)
        c = self.c = B.tp_beams_t()
        c.n_reqs, c.width, c.n_cands = n_reqs, width, n_cands
        c.n_ends = 0 if ends is None else ends.numel()
        for name in ("ends", "scores", "cand_scores", "cand_rows", "cand_tokens", "next_scores",
                     "parents", "tokens"):
            setattr(c, name, _ptr(getattr(self, name)))

    @classmethod
    def alloc(cls, n_reqs: int, width: int, n_cands: Optional[int] = None,
              ends: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
              in_place: bool = False, device="cuda") -> "Beams":
        """With its outputs allocated.  n_cands: by default width * (1 + ends), which is enough for
        every next beam to be found, but 64 at most: where that is less (32 beams and two ending
        ids, say), candidates that end their texts can leave next beams without a parent although
        the request has continuations.  scores: by default those of a first step, one beam a request
        in use.  in_place: next_scores is scores."""
        if n_cands is None:
            n_cands = min(width * (1 + (0 if ends is None else ends.numel())), B.MAX_BEAM_CANDS)
        if scores is None:
            scores = torch.full((n_reqs, width), -float("inf"), device=device)
            scores[:, 0] = 0
            scores = scores.flatten()

        def ints(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=scores.device)
        return cls(n_reqs, width, n_cands, scores,
                   torch.zeros((n_reqs, n_cands), dtype=torch.float32, device=scores.device),
                   ints(n_reqs, n_cands), ints(n_reqs, n_cands),
                   scores if in_place else torch.zeros_like(scores), ints(n_reqs * width),
                   ints(n_reqs * width), ends)


class PageMoves:
    """Moves of pages: table [most, 3] int32 (page, new page, tokens) and their count [1] int32, on
    the GPU (see tp_copy_pages)."""

    def __init__(self, table: torch.Tensor, count: torch.Tensor):
        _check(table, "table", torch.int32, (None, 3), table.device)
        _check(count, "count", torch.int32, (1,), table.device)
        self.table, self.count, self.most = table, count, table.shape[0]
        self._ptrs = (_ptr(table), _ptr(count))

    @classmethod
    def alloc(cls, most: int, device="cuda") -> "PageMoves":
        return cls(torch.zeros((most, 3), dtype=torch.int32, device=device),
                   torch.zeros(1, dtype=torch.int32, device=device))


class PageFork:
    """A fork of a page table (see tp_fork_t): row b goes on as the first keep_lens[b] tokens
    (None: all) of row src[b] (-1: none).

    old_lens, src, keep_lens [n_seqs] int32.  fork_pages fills table (of the page table's shape, in
    another buffer), new_lens and moves (room for n_seqs), and holders [n_pages] int32 (None: the
    page table's).  A fork that may be dropped again (free_next of its own) of a table with holders
    needs holders of its own.
    """

    def __init__(self, max_ctx: int, old_lens: torch.Tensor, src: torch.Tensor,
                 keep_lens: Optional[torch.Tensor], table: torch.Tensor, new_lens: torch.Tensor,
                 moves: PageMoves, holders: Optional[torch.Tensor] = None):
        n, dev = old_lens.numel(), old_lens.device
        for name, t in (("old_lens", old_lens), ("src", src), ("keep_lens", keep_lens),
                        ("new_lens", new_lens)):
            if t is not None:
                _check(t, name, torch.int32, (n,), dev)
        _check(table, "table", torch.int32, (None, None), dev)
        if holders is not None:
            _check(holders, "holders", torch.int32, (None,), dev)
        if moves.most < n or moves.table.device != dev:
            raise ValueError(f"moves: room for {n} on {dev} expected")
        self.n_seqs, self.max_ctx = n, max_ctx
        self.old_lens, self.src, self.keep_lens = old_lens, src, keep_lens
        self.table, self.new_lens, self.moves, self.holders = table, new_lens, moves, holders
        c = self.c = B.tp_fork_t()
        c.n_seqs, c.max_ctx = n, max_ctx
        c.old_lens, c.src, c.keep_lens = _ptr(old_lens), _ptr(src), _ptr(keep_lens)
        c.table, c.new_lens = _ptr(table), _ptr(new_lens)
        c.moves, c.n_moves = moves._ptrs
        c.holders = _ptr(holders)

    @classmethod
    def alloc(cls, pages: PageTable, max_ctx: int, old_lens: torch.Tensor, src: torch.Tensor,
              keep_lens: Optional[torch.Tensor] = None, table: Optional[torch.Tensor] = None,
              own_holders: bool = False) -> "PageFork":
        """With its outputs (the table too, unless it is given) allocated, holders of its own
        among them where the fork may be dropped again."""
        return cls(max_ctx, old_lens, src, keep_lens,
                   torch.zeros_like(pages.table) if table is None else table,
                   torch.zeros_like(old_lens), PageMoves.alloc(old_lens.numel(), old_lens.device),
                   torch.zeros_like(pages.holders) if own_holders else None)


class LayerPages:
    """The K and V pages of every layer (alloc_pages's), for copy_pages.  Their addresses are
    kept."""

    def __init__(self, k: Sequence[torch.Tensor], v: Sequence[torch.Tensor]):
        if len(k) != len(v):
            raise ValueError("as many layers of K as of V are needed")
        self.k, self.v, self.n_layers = list(k), list(v), len(k)
        self.shape, self.device = (k[0].shape, k[0].device) if self.n_layers else (None, None)
        ends = []
        for i, t in enumerate(self.k + self.v):
            _check(t, f"layer {i % self.n_layers}", torch.bfloat16, self.shape, self.device)
            ends.append((t.data_ptr(), t.data_ptr() + t.nbytes))
        ends.sort()
        if any(a[1] > b[0] for a, b in zip(ends, ends[1:])):
            raise ValueError("the layers' pages must not overlap")
        self._k = (ctypes.c_void_p * max(1, self.n_layers))(*[t.data_ptr() for t in self.k])
        self._v = (ctypes.c_void_p * max(1, self.n_layers))(*[t.data_ptr() for t in self.v])


class TPModel:
    """Owns one tp_model (the t ranks' shards) plus a workspace."""

    LAYER_KEYS = ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "wg", "wu", "wd")
    BIAS_KEYS = ("bq", "bk", "bv", "bo", "bg", "bu", "bd")

    def __init__(self, cfg: B.tp_config_t, layers: Sequence[Dict[str, torch.Tensor]],
                 embed: Optional[torch.Tensor] = None, final_norm: Optional[torch.Tensor] = None,
                 lm_head: Optional[torch.Tensor] = None, max_tokens: int = 64, stream=None):
        B.check(B.tp_config(cfg), "tp_config")
        self.cfg = cfg
        arr = (B.tp_layer_weights_t * max(len(layers), 1))()
        for i, L in enumerate(layers):
            for k in self.LAYER_KEYS:
                t = L[k]
                assert t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous(), k
                setattr(arr[i], k, t.data_ptr())
            for k in self.BIAS_KEYS:  # optional
                t = L.get(k)
                if t is not None:
                    assert t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous(), k
                    setattr(arr[i], k, t.data_ptr())
        w = B.tp_weights_t()
        w.embed, w.final_norm, w.lm_head = _ptr(embed), _ptr(final_norm), _ptr(lm_head)
        w.layers = ctypes.cast(arr, ctypes.POINTER(B.tp_layer_weights_t))
        self.handle = B.tp_load_shards(cfg, w, _stream(stream))
        self.max_tokens = 0
        self.ws = None
        self.device = torch.device("cuda", torch.cuda.current_device())
        # sizes the paged calls check against (reading a ctypes field takes its time)
        self._ranks, self._qkv_cols = cfg.attn_tp, self.qkv_rows()
        self._width = cfg.n_heads * cfg.head_dim
        self._copies, self._kv_heads, self._dim = cfg.kv_copies, cfg.kv_heads_per_rank, cfg.head_dim
        self._vocab = cfg.vocab
        self.step_ws = None
        self._step_cover = 0  # sequences that it is large enough for
        self._old_step_ws = []
        self._own_ws = {}  # kind -> (workspaces, the last of them in use; the last call's sizes)
        self.ensure_workspace(max_tokens, stream)

    # ------------------------------------------------------------------ utils
    def close(self):
        if getattr(self, "handle", None):
            B.tp_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def ensure_workspace(self, max_tokens: int, stream=None):
        if max_tokens <= self.max_tokens and self.ws is not None:
            return
        n = B.tp_workspace_bytes(self.handle, max_tokens)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        B.tp_workspace_init(self.ws.data_ptr(), n, _stream(stream))
        self.max_tokens = max_tokens

    @property
    def ws_args(self):
        return self.ws.data_ptr(), self.ws.numel()

    def alloc_kv(self, n_seqs: int, l_max: int) -> torch.Tensor:
        c = self.cfg
        return torch.empty((c.kv_copies, n_seqs, c.kv_heads_per_rank, l_max, c.head_dim),
                           dtype=torch.bfloat16, device="cuda")

    def model_bytes(self) -> int:
        return B.tp_model_bytes(self.handle)

    def check_device(self, stream=None) -> int:
        return B.tp_check_device(self.handle, _stream(stream))

    def stats(self) -> B.tp_stats_t:
        return B.tp_get_stats(self.handle)

    def reset_stats(self):
        B.tp_reset_stats(self.handle)

    def qkv_rows(self) -> int:
        c = self.cfg
        return (c.q_heads_per_rank + 2 * c.kv_heads_per_rank) * c.head_dim

    # ------------------------------------------------------------------ ops
    def column_linear(self, layer: int, which: int, x: torch.Tensor, stream=None) -> torch.Tensor:
        M = x.shape[0]
        n = self.qkv_rows() if which == B.TP_QKV else 2 * self.cfg.inter_per_rank
        ranks = self.cfg.attn_tp if which == B.TP_QKV else self.cfg.t
        y = torch.empty((ranks, M, n), dtype=torch.bfloat16, device="cuda")
        self.ensure_workspace(M, stream)
        B.check(B.tp_column_linear(self.handle, layer, which, x.data_ptr(), M, y.data_ptr(), M * n,
                                   *self.ws_args, _stream(stream)), "tp_column_linear")
        return y

    def row_linear_reduce(self, layer: int, which: int, x: torch.Tensor, residual=None,
                          fused: bool = True, out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
        """x: [M, t*K_r] (rank r's shard in columns [r K_r, (r+1) K_r))."""
        M = x.shape[0]
        t = self.cfg.attn_tp if which == B.TP_O else self.cfg.t
        kr = x.shape[1] // t
        y = out if out is not None else torch.empty((M, self.cfg.hidden), dtype=torch.bfloat16,
                                                    device="cuda")
        self.ensure_workspace(M, stream)
        B.check(B.tp_row_linear_reduce(self.handle, layer, which, x.data_ptr(), kr, x.stride(0), M,
                                       _ptr(residual), y.data_ptr(), int(fused), *self.ws_args,
                                       _stream(stream)), "tp_row_linear_reduce")
        return y

    def vocab_embed(self, ids: torch.Tensor, stream=None) -> torch.Tensor:
        h = torch.empty((ids.numel(), self.cfg.hidden), dtype=torch.bfloat16, device="cuda")
        B.check(B.tp_vocab_embed(self.handle, ids.data_ptr(), ids.numel(), h.data_ptr(),
                                 _stream(stream)), "tp_vocab_embed")
        return h

    def lm_head_gather(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        S = x.shape[0]
        logits = torch.empty((S, self.cfg.vocab), dtype=torch.bfloat16, device="cuda")
        self.ensure_workspace(S, stream)
        B.check(B.tp_lm_head_gather(self.handle, x.data_ptr(), S, logits.data_ptr(), self.cfg.vocab,
                                    *self.ws_args, _stream(stream)), "tp_lm_head_gather")
        return logits

    def rmsnorm(self, x: torch.Tensor, w: torch.Tensor, stream=None) -> torch.Tensor:
        y = torch.empty_like(x)
        B.check(B.tp_rmsnorm(self.handle, x.data_ptr(), w.data_ptr(), x.shape[0], y.data_ptr(),
                             _stream(stream)), "tp_rmsnorm")
        return y

    def layer_forward(self, layer: int, batch: Batch, h: torch.Tensor, fused: bool = True,
                      stream=None, cbatch: Optional[B.tp_batch_t] = None) -> torch.Tensor:
        self.ensure_workspace(batch.n_tokens, stream)
        cb = cbatch if cbatch is not None else batch.to_c()
        B.check(B.tp_layer_forward(self.handle, layer, cb, h.data_ptr(), int(fused), *self.ws_args,
                                   _stream(stream)), "tp_layer_forward")
        return h

    def layer_forward_host(self, layer: int, batch: Batch, h_in_host: torch.Tensor,
                           h_out_host: torch.Tensor, h_dev: torch.Tensor, fused: bool = True,
                           stream=None, cbatch: Optional[B.tp_batch_t] = None) -> torch.Tensor:
        """tp_layer_forward_host: pinned host rows in, the layer on h_dev, host rows out."""
        self.ensure_workspace(batch.n_tokens, stream)
        cb = cbatch if cbatch is not None else batch.to_c()
        B.check(B.tp_layer_forward_host(self.handle, layer, cb, h_in_host.data_ptr(),
                                        h_out_host.data_ptr(), h_dev.data_ptr(), int(fused),
                                        *self.ws_args, _stream(stream)), "tp_layer_forward_host")
        return h_out_host

    def forward(self, ids: torch.Tensor, batch: Batch, fused: bool = True, stream=None,
                h: Optional[torch.Tensor] = None, logits: Optional[torch.Tensor] = None,
                cbatch: Optional[B.tp_batch_t] = None):
        M = batch.n_tokens
        S = int(batch.sample_rows.numel())
        self.ensure_workspace(max(M, S), stream)
        if h is None:
            h = torch.empty((M, self.cfg.hidden), dtype=torch.bfloat16, device="cuda")
        if logits is None:
            logits = torch.empty((S, self.cfg.vocab), dtype=torch.bfloat16, device="cuda")
        cb = cbatch if cbatch is not None else batch.to_c()
        B.check(B.tp_forward(self.handle, ids.data_ptr(), cb, h.data_ptr(), logits.data_ptr(),
                             self.cfg.vocab, int(fused), *self.ws_args, _stream(stream)),
                "tp_forward")
        return logits


    def stage_forward(self, first_layer: int, n_layers: int, batch: Batch, h: torch.Tensor,
                      ids: Optional[torch.Tensor] = None, logits: Optional[torch.Tensor] = None,
                      fused: bool = True, stream=None,
                      cbatch: Optional[B.tp_batch_t] = None) -> torch.Tensor:
        M = batch.n_tokens
        S = int(batch.sample_rows.numel()) if batch.sample_rows is not None else 0
        self.ensure_workspace(max(M, S), stream)
        cb = cbatch if cbatch is not None else batch.to_c()
        B.check(B.tp_stage_forward(self.handle, first_layer, n_layers, _ptr(ids), cb, h.data_ptr(),
                                   _ptr(logits), self.cfg.vocab, int(fused), *self.ws_args,
                                   _stream(stream)), "tp_stage_forward")
        return h

    def stage_send(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> torch.Tensor:
        B.check(B.tp_stage_send(self.handle, src.data_ptr(), dst.data_ptr(), src.shape[0],
                                _stream(stream)), "tp_stage_send")
        return dst

    # ------------------------------------------------------- paged cache
    def alloc_pages(self, n_pages: int, page_size: int) -> torch.Tensor:
        """K or V pages of one layer (contents undefined, as alloc_kv's)."""
        c = self.cfg
        return torch.empty((c.kv_copies, n_pages, c.kv_heads_per_rank, page_size, c.head_dim),
                           dtype=torch.bfloat16, device=self.device)

    def step_workspace(self, n_seqs: int, max_new: int, stream=None) -> torch.Tensor:
        """A workspace for step_tables and tree_attention on steps of up to n_seqs sequences with
        up to max_new new tokens each.  Calls that may overlap on the GPU (two streams, two graphs
        replayed at once) need one each; the others can share the model's own."""
        n = B.tp_step_workspace_bytes(self.handle, n_seqs, max_new)
        if n == 0:
            raise ValueError(f"step of {n_seqs} sequences with {max_new} new tokens: outside limits")
        ws = self._out((n,), torch.uint8, stream)
        B.tp_workspace_init(ws.data_ptr(), n, _stream(stream))
        return ws

    def ensure_step_workspace(self, n_seqs: int, max_new: int, stream=None) -> torch.Tensor:
        """The model's own step workspace, grown when too small (not inside a graph capture).
        Nearly all of it is the same for every step (20 MB with heads of 128; a sequence adds some
        hundred bytes) and the earlier ones are kept, since captured graphs may still use them: it
        is made for any number of new tokens and 1024 sequences, and at least doubled."""
        if 0 < n_seqs <= self._step_cover and max_new >= 0:
            return self.step_ws
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("call ensure_step_workspace before the graph capture")
        if n_seqs > 0 and max_new >= 0:  # (else step_workspace refuses them)
            n_seqs = max(n_seqs, min(max(1024, 2 * self._step_cover), B.MAX_STEP_SEQS))
            max_new = max(max_new, B.MAX_TREE_TOKENS)  # more take no more
        ws = self.step_workspace(n_seqs, max_new, stream)
        if self.step_ws is not None:
            self._old_step_ws.append(self.step_ws)
        self.step_ws, self._step_cover = ws, n_seqs
        return ws

    def _ws_args(self, ws: torch.Tensor):
        """Address and bytes of a step workspace."""
        if ws.device != self.device or not ws.is_contiguous():
            raise ValueError("the workspace has to be contiguous, on the model's device")
        return ws.data_ptr(), ws.nbytes

    def _stream(self, stream) -> int:
        """As _stream, without building a stream object (the call's own kernels take 2 to 5 us,
        torch.cuda.current_stream up to 4)."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        return _stream(stream)

    def _out(self, shape, dtype, stream) -> torch.Tensor:
        """An output buffer that belongs to the stream the call runs on."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream(stream), device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def step_tables(self, pages: PageTable, step: Step, ws: Optional[torch.Tensor] = None,
                    stream=None) -> Step:
        """Block tables, slots, positions and tree masks of the step from its lengths."""
        t = pages.table
        if t is None or pages.free_ring is None or step.new_lens is None or step.q_start is None:
            raise ValueError("step_tables needs a page table with its ring, and a step with "
                             "new_lens and its output tables")
        if t.shape[0] < step.n_seqs or t.device != self.device or step.old_lens.device != self.device:
            raise ValueError("the page table has too few rows, or the tables are on another device")
        if ws is None:
            ws = self.ensure_step_workspace(step.n_seqs, step.max_new, stream)
        B.check(B.tp_step_tables(self.handle, pages.c, step.c, *self._ws_args(ws),
                                 self._stream(stream)), "tp_step_tables")
        return step

    def cache_append(self, qkv: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                     pages: PageTable, k: torch.Tensor, v: torch.Tensor,
                     q: Optional[torch.Tensor] = None, want_q: bool = True,
                     stream=None) -> Optional[torch.Tensor]:
        """RoPE and the new K/V rows into their slots; returns the rotated queries
        [M, n_heads*d] (into q when given; None with want_q False).  qkv: column_linear's
        output [ranks, M, N_r]."""
        M = qkv.shape[1]
        dev = self.device
        _check(qkv, "qkv", torch.bfloat16, (self._ranks, M, self._qkv_cols), dev)
        _check(positions, "positions", torch.int32, (M,), dev)
        _check(slots, "slots", torch.int32, (M,), dev)
        self._check_pools(k, v, pages)
        if q is not None:
            _check(q, "q", torch.bfloat16, (M, self._width), dev, rows=True)
        elif want_q:
            q = self._out((M, self._width), torch.bfloat16, stream)
        B.check(B.tp_cache_append(self.handle, qkv.data_ptr(), M * self._qkv_cols, M,
                                  positions.data_ptr(), slots.data_ptr(), pages.c, k.data_ptr(),
                                  v.data_ptr(), _ptr(q), 0 if q is None else _ld(q),
                                  self._stream(stream)), "tp_cache_append")
        return q

    def tree_attention(self, q: torch.Tensor, step: Step, pages: PageTable, k: torch.Tensor,
                       v: torch.Tensor, out: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of the step's tokens over the paged cache; q, out [n_tokens, n_heads*d].
        Padding rows of out are not written (undefined in a buffer allocated here)."""
        t = pages.table
        shape = (step.n_tokens, self._width)
        _check(q, "q", torch.bfloat16, shape, self.device, rows=True)
        if step.q_start is None or t is None or t.shape[0] < step.n_seqs or \
                t.device != self.device or step.old_lens.device != self.device:
            raise ValueError("tree_attention needs q_start and a table row for every sequence, on "
                             "the model's device")
        self._check_pools(k, v, pages)
        if out is None:
            out = self._out(shape, torch.bfloat16, stream)
        else:
            _check(out, "out", torch.bfloat16, shape, self.device, rows=True)
        if ws is None:
            ws = self.ensure_step_workspace(step.n_seqs, step.max_new, stream)
        B.check(B.tp_tree_attention(self.handle, q.data_ptr(), _ld(q), out.data_ptr(), _ld(out),
                                    pages.c, step.c, k.data_ptr(), v.data_ptr(),
                                    *self._ws_args(ws), self._stream(stream)), "tp_tree_attention")
        return out

    def _check_pools(self, k: torch.Tensor, v: torch.Tensor, pages: PageTable) -> None:
        shape = (self._copies, pages.n_pages, self._kv_heads, pages.page_size, self._dim)
        _check(k, "k", torch.bfloat16, shape, self.device)
        _check(v, "v", torch.bfloat16, shape, self.device)

    def process_logits(self, logits: torch.Tensor, rules: LogitRules,
                       out: Optional[torch.Tensor] = None, dtype=torch.float32,
                       stream=None) -> torch.Tensor:
        """Penalties, biases and grammar masks on bf16 logits [S, vocab]; the result in a new
        tensor of `dtype` (float32 or bfloat16), or in `out`, which may be `logits` itself.
        Rows with row_req -1 are not written (undefined in a tensor allocated here)."""
        S, V = logits.shape[0], self._vocab
        _check(logits, "logits", torch.bfloat16, (S, V), self.device, rows=True)
        n = rules.c.n_reqs if rules.n_rows is None else rules.n_rows
        if n != S:
            raise ValueError(f"the rules are for {n} rows, not {S}")
        if rules.device is not None and rules.device != self.device:
            raise ValueError("the rules' tensors are on another device")
        if rules._allowed_tokens is not None and rules._allowed_tokens < V:
            raise ValueError(f"allowed: {rules._allowed_tokens // 32} words a row do not cover "
                             f"{V} tokens")
        if out is None:
            if dtype not in (torch.float32, torch.bfloat16):
                raise ValueError("dtype: float32 or bfloat16 expected")
            out = self._out((S, V), dtype, stream)
        else:
            if out.dtype not in (torch.float32, torch.bfloat16):
                raise ValueError("out: float32 or bfloat16 expected")
            _check(out, "out", out.dtype, (S, V), self.device, rows=True)
        B.check(B.tp_process_logits(self.handle, logits.data_ptr(), _ld(logits), S, rules.c,
                                    out.data_ptr(), _ld(out), int(out.dtype == torch.float32),
                                    self._stream(stream)), "tp_process_logits")
        return out

    # ------------------------------------------------------- beams, shared pages
    def beam_workspace(self, n_reqs: int, width: int, n_cands: int, stream=None) -> torch.Tensor:
        """A workspace for beam_select on up to n_reqs requests of these sizes.  Calls that may
        overlap on the GPU need one each; the others can share the model's own."""
        return self._workspace(B.tp_beam_workspace_bytes(self.handle, n_reqs, width, n_cands),
                               f"{n_reqs} requests of {width} beams, {n_cands} candidates", stream)

    def share_workspace(self, n_pages: int, stream=None) -> torch.Tensor:
        """A workspace for fork_pages and compact_pages on up to n_pages pages, as
        beam_workspace."""
        return self._workspace(B.tp_share_workspace_bytes(self.handle, n_pages),
                               f"{n_pages} pages", stream)

    def _workspace(self, n: int, what: str, stream) -> torch.Tensor:
        if n == 0:
            raise ValueError(f"{what}: outside limits")
        ws = self._out((n,), torch.uint8, stream)
        B.tp_workspace_init(ws.data_ptr(), n, _stream(stream))
        return ws

    def ensure_beam_workspace(self, n_reqs: int, width: int, n_cands: int, stream=None):
        """The model's own workspace of beam_select, at least doubled when too small (not inside a
        graph capture; the earlier ones are kept, since captured graphs may still use them)."""
        return self._ensure("beam", (n_reqs, width, n_cands), B.tp_beam_workspace_bytes, stream)

    def ensure_share_workspace(self, n_pages: int, stream=None):
        """The model's own workspace of fork_pages and compact_pages, as ensure_beam_workspace."""
        return self._ensure("share", (n_pages,), B.tp_share_workspace_bytes, stream)

    def _ensure(self, kind: str, sizes, size, stream) -> torch.Tensor:
        held, last = self._own_ws.setdefault(kind, ([], [None]))
        if last[0] == sizes:
            return held[-1]
        n = size(self.handle, *sizes)
        if n == 0 or not held or held[-1].numel() < n:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError(f"call ensure_{kind}_workspace before the graph capture")
            most = 2 * held[-1].numel() if n and held else 0
            held.append(self._workspace(max(n, most), f"{kind} of {sizes}", stream))
        last[0] = sizes
        return held[-1]

    def beam_select(self, logits: torch.Tensor, beams: Beams, ws: Optional[torch.Tensor] = None,
                    stream=None) -> Beams:
        """The best continuations of every request's beams; logits [n_reqs*width, vocab] bf16 or
        float32."""
        dtype = logits.dtype
        if dtype is not torch.bfloat16 and dtype is not torch.float32:
            raise ValueError("logits: float32 or bfloat16 expected")
        _check(logits, "logits", dtype, (beams.n_reqs * beams.width, self._vocab), self.device, rows=True)
        if beams.scores.device != self.device:
            raise ValueError("the beams' tensors are on another device")
        if ws is None:
            ws = self.ensure_beam_workspace(*beams.sizes, stream)
        B.check(B.tp_beam_select(self.handle, logits.data_ptr(), _ld(logits),
                                 int(dtype is torch.float32), beams.c, *self._ws_args(ws),
                                 self._stream(stream)), "tp_beam_select")
        return beams

    def beam_advance(self, parents: torch.Tensor, tokens: torch.Tensor, history: torch.Tensor,
                     lens: torch.Tensor, out: Optional[torch.Tensor] = None,
                     lens_out: Optional[torch.Tensor] = None, stream=None):
        """Row b of out becomes row parents[b] of history [rows, room] and tokens[b] behind it.
        Returns (out, lens_out); ids of out behind a text are not written (undefined in a buffer
        allocated here).  history and out may be views of wider rows: nothing beside them is read
        or written."""
        n, dev, i32 = parents.shape[0], self.device, torch.int32
        _check(parents, "parents", i32, (n,), dev)
        _check(tokens, "tokens", i32, (n,), dev)
        _check(lens, "lens", i32, (n,), dev)
        # (any row length, but named: the whole check of a contiguous tensor is its first line)
        room = room_out = history.shape[-1]
        _check(history, "history", i32, (n, room), dev, rows=True)
        if out is None:
            out = self._out((n, room), i32, stream)
        else:
            room_out = out.shape[-1]
            _check(out, "out", i32, (n, room_out), dev, rows=True)
        if lens_out is None:
            lens_out = self._out((n,), i32, stream)
        else:
            _check(lens_out, "lens_out", i32, (n,), dev)
        B.check(B.tp_beam_advance_rooms(self.handle, n, parents.data_ptr(), tokens.data_ptr(),
                                        history.data_ptr(), history.stride(0) if n > 1 else room, room,
                                        lens.data_ptr(), out.data_ptr(),
                                        out.stride(0) if n > 1 else room_out, room_out,
                                        lens_out.data_ptr(), self._stream(stream)),
                "tp_beam_advance_rooms")
        return out, lens_out

    def fork_pages(self, pages: PageTable, fork: PageFork, ws: Optional[torch.Tensor] = None,
                   stream=None) -> PageFork:
        """The page table behind the fork's sources, pages shared; fork.moves goes to copy_pages.
        pages.with_table(fork.table) is the page table from here on."""
        t = pages.table
        if t is None or pages.free_ring is None:
            raise ValueError("fork_pages needs a page table with its ring")
        if t.shape[0] < fork.n_seqs or fork.table.shape[0] < fork.n_seqs or \
                fork.table.shape[1] != t.shape[1] or t.device != self.device or \
                fork.table.device != self.device:
            raise ValueError("the page tables differ in row length, have too few rows, or are on "
                             "another device")
        if fork.holders is not None and (pages.holders is None or fork.holders.numel() != pages.n_pages):
            raise ValueError(f"the fork's holders: {pages.n_pages} of a page table with holders expected")
        if ws is None:
            ws = self.ensure_share_workspace(pages.n_pages, stream)
        B.check(B.tp_fork_pages(self.handle, pages.c, fork.c, *self._ws_args(ws),
                                self._stream(stream)), "tp_fork_pages")
        return fork

    def compact_pages(self, pages: PageTable, lens: torch.Tensor, max_ctx: int, moves: PageMoves,
                      out: Optional[PageTable] = None, ws: Optional[torch.Tensor] = None,
                      stream=None) -> PageTable:
        """Renames the pages in use to the first ones; moves (room for n_pages // 2) goes to
        copy_pages.  Written to `out` (None: pages itself), whose tensors may be those of pages."""
        out = pages if out is None else out
        n = lens.numel()
        _check(lens, "lens", torch.int32, (n,), self.device)
        for p in (pages, out):
            if p.table is None or p.free_ring is None or p.table.shape[0] < n or p.table.device != self.device:
                raise ValueError("compact_pages needs page tables with their rings and a row for every "
                                 "length, on the model's device")
        if moves.table.device != self.device:
            raise ValueError("the moves are on another device")
        if ws is None:
            ws = self.ensure_share_workspace(pages.n_pages, stream)
        table, count = moves._ptrs
        B.check(B.tp_compact_pages(self.handle, pages.c, out.c, n, max_ctx, lens.data_ptr(), table,
                                   moves.most, count, *self._ws_args(ws), self._stream(stream)),
                "tp_compact_pages")
        return out

    def copy_pages(self, moves: PageMoves, pages: PageTable, layers: LayerPages, stream=None) -> None:
        """Copies the moves' pages in every layer's K and V."""
        if moves.table.device != self.device:
            raise ValueError("the moves are on another device")
        if layers.n_layers:
            shape = (self._copies, pages.n_pages, self._kv_heads, pages.page_size, self._dim)
            if layers.shape != shape or layers.device != self.device:
                raise ValueError(f"layers: pages of shape {shape} on {self.device} expected, got "
                                 f"{tuple(layers.shape)} on {layers.device}")
        table, count = moves._ptrs
        B.check(B.tp_copy_pages(self.handle, pages.c, table, count, moves.most, layers.n_layers,
                                layers._k, layers._v, self._stream(stream)), "tp_copy_pages")

    def capture_forward(self, ids: torch.Tensor, batch: Batch, h: torch.Tensor,
                        logits: torch.Tensor, stream, fused: bool = True,
                        cbatch: Optional[B.tp_batch_t] = None) -> "Graph":
        """CUDA graph of tp_forward with these buffers (see tp_graph_capture_forward)."""
        M = batch.n_tokens
        S = int(batch.sample_rows.numel())
        self.ensure_workspace(max(M, S), stream)
        cb = cbatch if cbatch is not None else batch.to_c()
        st, g = B.tp_graph_capture_forward(self.handle, ids.data_ptr(), cb, h.data_ptr(),
                                           logits.data_ptr(), self.cfg.vocab, int(fused),
                                           *self.ws_args, _stream(stream))
        B.check(st, "tp_graph_capture_forward")
        return Graph(g, keep=(ids, batch, cb, h, logits, self.ws))

    def capture_layer(self, layer: int, batch: Batch, h: torch.Tensor, stream, fused: bool = True,
                      cbatch: Optional[B.tp_batch_t] = None) -> "Graph":
        """CUDA graph of tp_layer_forward with these buffers."""
        self.ensure_workspace(batch.n_tokens, stream)
        cb = cbatch if cbatch is not None else batch.to_c()
        st, g = B.tp_graph_capture_layer(self.handle, layer, cb, h.data_ptr(), int(fused),
                                         *self.ws_args, _stream(stream))
        B.check(st, "tp_graph_capture_layer")
        return Graph(g, keep=(batch, cb, h, self.ws))


class Graph:
    """An executable graph of one captured call; keeps the captured buffers alive."""

    def __init__(self, handle, keep):
        self.handle = handle
        self._keep = keep

    def launch(self, stream=None) -> None:
        B.check(B.tp_graph_launch(self.handle, _stream(stream)), "tp_graph_launch")

    def close(self) -> None:
        if self.handle:
            B.tp_graph_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def decode_batch(n_seqs: int, ctx: int, k_cache, v_cache, l_max: Optional[int] = None,
                 with_samples: bool = True) -> Batch:
    dev = "cuda"
    pos = torch.full((n_seqs,), ctx - 1, dtype=torch.int32, device=dev)
    seq = torch.arange(n_seqs, dtype=torch.int32, device=dev)
    return Batch(B.TP_DECODE, n_seqs, n_seqs, 1, ctx, l_max or ctx, pos, seq, None,
                 list(k_cache), list(v_cache), seq.clone() if with_samples else None)


def prefill_batch(n_seqs: int, seq_len: int, k_cache, v_cache, l_max: Optional[int] = None) -> Batch:
    dev = "cuda"
    M = n_seqs * seq_len
    pos = torch.arange(seq_len, dtype=torch.int32, device=dev).repeat(n_seqs)
    seq = torch.arange(n_seqs, dtype=torch.int32, device=dev).repeat_interleave(seq_len)
    start = torch.arange(0, M + 1, seq_len, dtype=torch.int32, device=dev)
    samples = torch.arange(seq_len - 1, M, seq_len, dtype=torch.int32, device=dev)
    return Batch(B.TP_PREFILL, n_seqs, M, seq_len, seq_len, l_max or seq_len, pos, seq, start,
                 list(k_cache), list(v_cache), samples)
