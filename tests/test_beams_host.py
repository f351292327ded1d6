"""Beam search and shared pages on the host (no GPU): the ctypes structures against the C
header, refusals without a model, the checks of the Python wrappers, and the plain
implementations that the GPU tests compare with."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import megatron_tensor_layers_tp_gb300.binding as B  # noqa: E402
from megatron_tensor_layers_tp_gb300.runtime import (Beams, LayerPages, PageFork, PageMoves,  # noqa: E402
                                                     PageTable, TPModel)
from tests import beam_reference as R  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_structures_match_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "tp.h"', "int main(void) {"]
    types = (B.tp_pages_t, B.tp_beams_t, B.tp_fork_t)
    for t in types:
        lines.append(f'printf("%zu\\n", sizeof({t.__name__}));')
        lines += [f'printf("%zu\\n", offsetof({t.__name__}, {n}));' for n, _ in t._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    want = []
    for t in types:
        want += [ctypes.sizeof(t)] + [getattr(t, n).offset for n, _ in t._fields_]
    assert got == want


def test_calls_without_a_model_are_rejected():
    ARG = B.STATUS["TP_ERR_ARG"]
    p, b, f = B.tp_pages_t(), B.tp_beams_t(), B.tp_fork_t()
    assert B.tp_beam_workspace_bytes(None, 1, 1, 1) == 0 and B.tp_share_workspace_bytes(None, 4) == 0
    assert B.tp_beam_select(None, 0, 0, 0, b, 0, 0, 0) == ARG
    assert B.tp_beam_advance(None, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0) == ARG
    assert B.tp_fork_pages(None, p, f, 0, 0, 0) == ARG
    assert B.tp_compact_pages(None, p, p, 1, 1, 0, 0, 0, 0, 0, 0, 0) == ARG
    assert B.tp_copy_pages(None, p, 0, 0, 1, 1, None, None, 0) == ARG


def test_texts_in_views_without_a_model_are_rejected():
    assert B.tp_beam_advance_rooms(None, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) == B.STATUS["TP_ERR_ARG"]


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_holders_of_a_page_table():
    p = PageTable.alloc(3, 10, 16, 33, device="cpu", shared=True)
    assert p.holders.shape == (10,) and p.c.holders == p.holders.data_ptr()
    assert PageTable.alloc(3, 10, 16, 33, device="cpu").c.holders is None
    q = p.with_table(ints(3, 3))
    assert q.c.free_ring == p.c.free_ring and q.c.holders == p.c.holders and q.c.table != p.c.table
    for bad in (dict(holders=ints(9)), dict(holders=ints(10).long()), dict(table=None, holders=ints(10))):
        kw = dict(dict(table=ints(3, 3), n_pages=10), **bad)
        with pytest.raises(ValueError):
            PageTable(16, **kw)


def test_beams_checks():
    b = Beams.alloc(3, 4, ends=ints(2), device="cpu")
    assert b.n_cands == 12 and b.c.n_ends == 2 and b.cand_rows.shape == (3, 12)
    assert b.scores.view(3, 4)[:, 0].tolist() == [0, 0, 0] and (b.scores.view(3, 4)[:, 1:] == -np.inf).all()
    assert Beams.alloc(1, 32, ends=ints(8), device="cpu").n_cands == 64
    c = Beams.alloc(3, 4, 5, scores=torch.zeros(12), in_place=True, device="cpu")
    assert c.next_scores is c.scores and c.c.next_scores == c.c.scores and c.c.n_ends == 0 and not c.c.ends
    good = {k: getattr(b, k) for k in ("scores", "cand_scores", "cand_rows", "cand_tokens", "next_scores", "parents",
                                       "tokens", "ends")}
    Beams(3, 4, 12, **good)
    for name, t in (("scores", torch.zeros(11)), ("scores", torch.zeros(12).double()), ("cand_scores", torch.zeros(3, 11)),
                    ("cand_rows", torch.zeros(3, 12)), ("cand_tokens", ints(12, 3).t()), ("next_scores", ints(12)),
                    ("parents", ints(13)), ("tokens", ints(24)[::2]), ("ends", ints(2).long()), ("ends", ints(2, 1))):
        with pytest.raises(ValueError):
            Beams(3, 4, 12, **dict(good, **{name: t}))


def test_fork_and_moves_checks():
    p = PageTable.alloc(3, 10, 16, 33, device="cpu")
    f = PageFork.alloc(p, 33, ints(3), ints(3))
    assert f.table.shape == p.table.shape and f.moves.most == 3 and not f.c.keep_lens and f.c.max_ctx == 33
    good = dict(max_ctx=33, old_lens=ints(3), src=ints(3), keep_lens=None, table=ints(3, 3), new_lens=ints(3),
                moves=PageMoves.alloc(3, device="cpu"))
    PageFork(**good)
    for bad in (dict(src=ints(2)), dict(keep_lens=ints(4)), dict(new_lens=ints(3).long()), dict(table=ints(3)),
                dict(moves=PageMoves.alloc(2, device="cpu")), dict(table=ints(6, 3)[::2])):
        with pytest.raises(ValueError):
            PageFork(**dict(good, **bad))
    for bad in ((ints(3, 2), ints(1)), (ints(3, 3), ints(2)), (ints(3, 3).long(), ints(1)), (ints(3, 6)[:, :3], ints(1))):
        with pytest.raises(ValueError):
            PageMoves(*bad)


def test_holders_of_a_fork():
    p = PageTable.alloc(3, 10, 16, 33, device="cpu", shared=True)
    f = PageFork.alloc(p, 33, ints(3), ints(3), own_holders=True)
    assert f.holders.shape == (10,) and f.c.holders == f.holders.data_ptr() != p.c.holders
    assert not PageFork.alloc(p, 33, ints(3), ints(3)).c.holders
    state = ints(2)
    q = p.with_table(f.table, state, f.holders)
    assert q.c.free_state == q.c.free_next == state.data_ptr() and q.c.holders == f.c.holders
    assert q.c.free_ring == p.c.free_ring
    with pytest.raises(ValueError):
        PageFork(33, ints(3), ints(3), None, ints(3, 3), ints(3), PageMoves.alloc(3, device="cpu"), ints(10).long())
    ws = torch.empty(1 << 16, dtype=torch.uint8)
    with pytest.raises(B.TPError):  # on to the call
        TPModel.fork_pages(Host(), p, f, ws=ws)
    plain = PageTable.alloc(3, 10, 16, 33, device="cpu")
    few = PageTable.alloc(3, 9, 16, 33, device="cpu", shared=True)
    for pages in (plain, few):
        with pytest.raises(ValueError):
            TPModel.fork_pages(Host(), pages, f, ws=ws)


def test_layer_pages_checks():
    def page(n=3):
        return torch.zeros((2, n, 1, 8, 64), dtype=torch.bfloat16)
    a = LayerPages([page(), page()], [page(), page()])
    assert a.n_layers == 2 and a.shape == (2, 3, 1, 8, 64)
    assert LayerPages([], []).n_layers == 0
    one, wide = page(), torch.zeros((2, 6, 1, 8, 64), dtype=torch.bfloat16)
    for k, v in (([page()], []), ([page(), page(4)], [page(), page()]), ([page()], [page().float()]), ([one], [one]),
                 ([one, page()], [page(), one]), ([page()], [wide[:, ::2]])):
        with pytest.raises(ValueError):
            LayerPages(k, v)


class Host:
    """What the wrappers read of a model, on the CPU: their checks come before the C call, which
    refuses the missing handle with another error."""
    handle, device = None, torch.device("cpu")
    _vocab, _copies, _kv_heads, _dim = 100, 2, 1, 64
    _ws_args = TPModel._ws_args

    def _out(self, shape, dtype, stream):
        return torch.empty(shape, dtype=dtype)

    def _stream(self, stream):
        return 0


def test_wrapper_checks():
    ws = torch.empty(1 << 16, dtype=torch.uint8)
    beams = Beams.alloc(2, 3, 6, device="cpu")
    pages = PageTable.alloc(3, 10, 16, 33, device="cpu")
    fork = PageFork.alloc(pages, 33, ints(3), ints(3))
    moves = PageMoves.alloc(5, device="cpu")
    page = lambda n=10, P=16: torch.zeros((2, n, 1, P, 64), dtype=torch.bfloat16)  # noqa: E731
    layers = LayerPages([page()], [page()])
    narrow = PageTable.alloc(3, 10, 16, 16, device="cpu")
    few = PageTable.alloc(2, 10, 16, 33, device="cpu")

    def select(logits=torch.zeros(6, 100), b=beams, ws=ws):
        return TPModel.beam_select(Host(), logits, b, ws=ws)

    def advance(parents=ints(4), tokens=ints(4), history=ints(4, 9), lens=ints(4), **kw):
        return TPModel.beam_advance(Host(), parents, tokens, history, lens, **kw)

    def forks(p=pages, f=fork, ws=ws):
        return TPModel.fork_pages(Host(), p, f, ws=ws)

    def compact(p=pages, lens=ints(3), out=None, mv=moves, ws=ws):
        return TPModel.compact_pages(Host(), p, lens, 33, mv, out=out, ws=ws)

    def copy(mv=moves, p=pages, lay=layers):
        return TPModel.copy_pages(Host(), mv, p, lay)

    for call in (select, advance, forks, compact, copy,
                 lambda: select(torch.zeros(6, 100, dtype=torch.bfloat16)), lambda: select(torch.zeros(6, 128)[:, :100]),
                 lambda: advance(history=ints(4, 12)[:, :9], out=ints(4, 20)[:, 3:], lens_out=ints(4)),
                 lambda: compact(out=PageTable.alloc(3, 10, 16, 33, device="cpu")), lambda: copy(lay=LayerPages([], []))):
        with pytest.raises(B.TPError):  # on to the call
            call()
    odd = torch.empty(1 << 17, dtype=torch.uint8)[::2]
    for call in (lambda: select(torch.zeros(5, 100)), lambda: select(torch.zeros(6, 99)), lambda: select(torch.zeros(6, 100).half()),
                 lambda: select(torch.zeros(100, 6).t()), lambda: select(torch.zeros(6, 100).double()), lambda: select(ws=odd),
                 lambda: advance(parents=ints(3)), lambda: advance(tokens=ints(4).long()), lambda: advance(lens=ints(5)),
                 lambda: advance(history=ints(3, 9)), lambda: advance(history=ints(9, 4).t()),
                 lambda: advance(history=ints(1, 9).expand(4, 9)), lambda: advance(out=ints(3, 9)),
                 lambda: advance(lens_out=ints(3)), lambda: forks(p=PageTable(16, n_pages=10)), lambda: forks(p=narrow),
                 lambda: forks(p=few), lambda: forks(ws=odd), lambda: compact(p=few), lambda: compact(out=few),
                 lambda: compact(lens=ints(3).long()), lambda: compact(out=PageTable(16, ints(3, 3), n_pages=10)),
                 lambda: compact(ws=odd), lambda: copy(p=PageTable(16, n_pages=9)), lambda: copy(p=PageTable(8, n_pages=10)),
                 lambda: copy(lay=LayerPages([page(10, 8)], [page(10, 8)]))):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------------------
# the plain implementations against worked cases
# ---------------------------------------------------------------------------
def test_reference_selection_by_hand():
    log = np.log
    x = log(np.array([[0.5, 0.25, 0.25, 0.0 + 1e-300], [0.1, 0.2, 0.3, 0.4]]))
    (pool, alive), = R.select(x, np.array([log(0.6), log(0.4)]), 2, 5, ends=(0,))
    assert [(b, v) for _, b, v in pool] == [(0, 0), (1, 3), (0, 1), (0, 2), (1, 2)]
    assert np.allclose(np.exp([c[0] for c in pool]), [0.3, 0.16, 0.15, 0.15, 0.12])
    assert [(b, v) for _, b, v in alive] == [(1, 3), (0, 1)]
    x[0, 1], x[1] = np.nan, -np.inf
    (pool, alive), = R.select(x, np.array([0.0, 0.0]), 2, 9)
    assert [(b, v) for _, b, v in pool] == [(0, 0), (0, 2), (0, 3)] and len(alive) == 2
    assert np.allclose(np.exp([c[0] for c in pool[:2]]), [2 / 3, 1 / 3])
    assert R.select(x, np.array([-np.inf, np.nan]), 2, 3) == [([], [])]


def test_reference_fork_by_hand():
    """Pages of 4: row 0 holds 10 tokens in pages 3, 1, 7; row 1 nothing; row 2 four in page 0."""
    table, lens, ring = [[3, 1, 7], [9, 9, 9], [0, 9, 9]], [10, 0, 4], [2, 4, 5, 6, -1, -1, -1, -1]
    rows, keep, moves, new, first, count, holders = R.fork(table, lens, [0, 0, 0], None, 4, ring, 0, 4)
    assert rows == [[3, 1, 7], [3, 1, 2], [3, 1, 4]] and keep == [10, 10, 10]
    assert moves == [(7, 2, 2), (7, 4, 2)] and (first, count) == (2, 3) and new[4] == 0
    assert holders == {3: 3, 1: 3, 7: 1, 2: 1, 4: 1}
    # a row that ends inside a page that is another's full one gets a copy; the page of ten goes back
    rows, keep, moves, new, first, count, holders = R.fork(table, lens, [0, 0, 2], [8, 6, 4], 4, ring, 0, 4)
    assert rows == [[3, 1], [3, 2], [0]] and moves == [(1, 2, 2)] and (first, count) == (1, 4) and new[4] == 7
    rows, keep, moves, new, first, count, holders = R.fork(table, lens, [-1, -1, -1], None, 4, ring, 2, 2)
    assert rows == [[], [], []] and new[4:] == [0, 1, 3, 7] and (first, count) == (2, 6) and holders == {}


def test_reference_compaction_by_hand():
    rows, moves, used, holders = R.compact([[6, 1, 9], [6, 4, 9], [8, 9, 9]], [8, 5, 1], 4, 10)
    assert used == 4 and moves == [(8, 0, 4), (6, 2, 4), (4, 3, 4)]
    assert rows == [[2, 1], [2, 3], [0]] and holders == {2: 2, 1: 1, 3: 1, 0: 1}
