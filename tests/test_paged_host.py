"""The paged-cache serving calls on the host (no GPU): the ctypes structures
against the C header, refusals without a model, and the checks of the Python
wrappers."""
import ctypes
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

import megatron_tensor_layers_tp_gb300.binding as B  # noqa: E402
from megatron_tensor_layers_tp_gb300.runtime import LogitRules, PageTable, Step, TPModel  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_structures_match_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "tp.h"', "int main(void) {"]
    types = (B.tp_pages_t, B.tp_step_t, B.tp_logit_rules_t)
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
    p, s, r = B.tp_pages_t(), B.tp_step_t(), B.tp_logit_rules_t()
    assert B.tp_step_workspace_bytes(None, 4, 4) == 0
    assert B.tp_step_tables(None, p, s, 0, 0, 0) == ARG
    assert B.tp_cache_append(None, 0, 0, 1, 0, 0, p, 0, 0, 0, 0, 0) == ARG
    assert B.tp_tree_attention(None, 0, 0, 0, 0, p, s, 0, 0, 0, 0, 0) == ARG
    assert B.tp_process_logits(None, 0, 0, 1, r, 0, 0, 0, 0) == ARG
    assert B.STATUS["TP_ERR_TABLE_RANGE"] == 10


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_page_table_checks():
    PageTable(8, n_pages=3)
    PageTable(8, ints(2, 4), ints(9), ints(2))
    p = PageTable.alloc(3, 10, 16, 33, device="cpu")
    assert p.table.shape == (3, 3) and p.free_state.tolist() == [0, 10] and p.c.ld_table == 3
    assert p.c.free_next == p.c.free_state
    for bad in (dict(), dict(table=ints(2, 4)), dict(free_ring=ints(9)),
                dict(table=ints(2, 4), free_ring=ints(9)),
                dict(table=ints(2, 4), free_ring=ints(9), free_state=ints(3)),
                dict(table=ints(2, 4), free_ring=ints(9), free_state=ints(2), free_next=ints(1)),
                dict(table=ints(2, 4).long(), n_pages=9), dict(table=ints(4), n_pages=9),
                dict(table=ints(4, 2).t(), n_pages=9)):
        with pytest.raises(ValueError):
            PageTable(8, **bad)


def test_step_checks():
    s = Step.alloc(3, 7, 4, 100, tree_words=2, device="cpu")
    assert s.c.n_seqs == 3 and s.c.tree_words == 2 and s.q_start.shape == (4,)
    assert Step.alloc(3, 7, 4, 100, device="cpu").c.tree_words == 0
    for bad in (dict(new_lens=ints(2)), dict(q_start=ints(3)), dict(slots=ints(6)),
                dict(parents=ints(8)), dict(positions=ints(7).long()),
                dict(tree_mask=torch.zeros((6, 1), dtype=torch.int64)), dict(tree_mask=ints(7, 1)),
                dict(token_seq=ints(14)[::2])):
        with pytest.raises(ValueError):
            Step(7, 4, 100, ints(3), **bad)


def test_logit_rules_checks():
    f = torch.zeros
    r = LogitRules(history=ints(2, 5), history_lens=ints(2), presence=f(2))
    assert r.c.n_reqs == 2 and r.n_rows is None and r.c.ld_history == 5
    r = LogitRules(row_req=ints(6), repetition=f(2))
    assert r.c.n_reqs == 2 and r.n_rows == 6
    assert LogitRules(allowed=ints(4, 9)).c.n_reqs == 4
    assert LogitRules(allowed=ints(9, 4).repeat(1, 3)[:, :5], n_reqs=9).c.ld_allowed == 12
    mask = torch.zeros((6, 1), dtype=torch.int64)
    LogitRules(row_req=ints(6), draft_tokens=ints(6), tree_mask=mask, q_start=ints(3))
    for bad in (dict(row_req=ints(4)), dict(), dict(history=ints(2, 5)), dict(history_lens=ints(2)),
                dict(history=ints(2, 5), history_lens=ints(3)), dict(presence=f(2), repetition=f(3)),
                dict(presence=f(2).double()), dict(draft_tokens=ints(6), row_req=ints(6), n_reqs=2),
                dict(row_req=ints(6), draft_tokens=ints(5), tree_mask=mask, q_start=ints(3)),
                dict(bias_start=ints(3), bias_ids=ints(2)), dict(presence=f(2), allowed=ints(4, 9)),
                dict(bias_start=ints(3), bias_ids=ints(2), bias_values=f(3)),
                dict(allowed=ints(4, 9).long()), dict(history=ints(5, 2).t(), history_lens=ints(2))):
        with pytest.raises(ValueError):
            LogitRules(**bad)


class Host:
    """What the paged wrappers read of a model, on the CPU: their checks come before the C call,
    which refuses the missing handle with another error."""
    handle, device = None, torch.device("cpu")
    _vocab, _width, _copies, _kv_heads, _dim = 100, 512, 1, 2, 64
    _check_pools, _ws_args = TPModel._check_pools, TPModel._ws_args

    def _out(self, shape, dtype, stream):
        return torch.empty(shape, dtype=dtype)

    def _stream(self, stream):
        return 0


def test_allowed_words_must_cover_the_vocabulary():
    """A view of fewer words than the vocabulary needs, in rows that lie as far apart as it needs:
    its last row would be read behind its end."""
    logits = torch.zeros((3, 100), dtype=torch.bfloat16)
    for allowed in (ints(11).as_strided((3, 3), (4, 1)), ints(3, 8)[:, :1], ints(3, 3)):
        with pytest.raises(ValueError, match="allowed"):
            TPModel.process_logits(Host(), logits, LogitRules(allowed=allowed))
    with pytest.raises(B.TPError):  # as many as it needs: on to the call
        TPModel.process_logits(Host(), logits, LogitRules(allowed=ints(3, 4)))


def test_workspaces_that_are_refused():
    """A workspace on another device, or one whose bytes are not one run: its size in bytes would
    not be what the kernels may write."""
    pages, step = PageTable.alloc(2, 9, 8, 32, device="cpu"), Step.alloc(2, 4, 4, 32, device="cpu")
    q = torch.zeros((4, 512), dtype=torch.bfloat16)
    k = torch.zeros((1, 9, 2, 8, 64), dtype=torch.bfloat16)
    calls = (lambda ws: TPModel.step_tables(Host(), pages, step, ws=ws),
             lambda ws: TPModel.tree_attention(Host(), q, step, pages, k, k, ws=ws))
    for call in calls:
        for ws in (torch.empty(512, dtype=torch.uint8, device="meta"),
                   torch.empty(1024, dtype=torch.uint8)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(ws)
        with pytest.raises(B.TPError):  # on to the call
            call(torch.empty(512, dtype=torch.uint8))
