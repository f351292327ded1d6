"""The paged-cache serving calls against plain 64-bit implementations: step
tables, rotary embedding with the page store, attention of drafted trees over
the pages, rules on logits, and their run together.

Tolerances (a rounding to bf16 is off by at most 2^-8 of the value, one to
fp32 by 2^-24):
- append: one rounding of a*c - b*s; the fp32 arithmetic in front of it (c and
  s rounded, two products, a sum) is off by at most 4 * 2^-24 (|a| + |b|);
- attention: with A = sum_j p_j |v_j|, the rounding of each p to bf16 moves o
  by at most 2^-8 A and the output's own rounding by 2^-8 |o|.  A score is off
  by at most (d + 4) 2^-24 S, S = sum |q||k| / sqrt(d) (d products and sums in
  fp32, the scale), and exp2 and the sums over keys are each good to 2^-20 or
  better, so numerator and denominator add 2 ((d + 4) 2^-24 S + 2^-19) A;
- logits: at most six fp32 roundings of terms whose magnitudes add up to m:
  6 * 2^-24 m, and 2^-8 |x| more for a bf16 result.
"""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from megatron_tensor_layers_tp_gb300 import binding as B  # noqa: E402
from megatron_tensor_layers_tp_gb300.runtime import (LogitRules, PageTable, Step,  # noqa: E402
                                                     TPModel, make_config)
from tests import paged_reference as R  # noqa: E402

THETA = 10000.0
TABLE_RANGE = B.STATUS["TP_ERR_TABLE_RANGE"]
_models = {}


def model(heads=8, kv=4, dim=64, t=2, vocab=1000, attn_dp=1):
    """A model without layers: the paged calls read no weights."""
    key = (heads, kv, dim, t, vocab, attn_dp)
    if key not in _models:
        cfg = make_config(heads * dim, heads, kv, dim, 64 * t, vocab, 0, t, rope_theta=THETA,
                          max_positions=20000, attn_dp=attn_dp)
        _models[key] = TPModel(cfg, [], max_tokens=1)
    return _models[key]


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).bfloat16().cuda()


# ---------------------------------------------------------------------------
# step tables
# ---------------------------------------------------------------------------
def tables_case(rng, n_seqs, max_new, page, max_len, tree, shrink, pad=3, spare=5):
    old = rng.integers(0, max_len + 1, n_seqs)
    new = old + rng.integers(0, max_new + 1, n_seqs)
    gone = rng.random(n_seqs) < shrink
    new = np.where(gone, (old * rng.random(n_seqs)).astype(np.int64), new)
    have = [R.ceil_div(int(o), page) for o in old]
    ld = R.ceil_div(max_len + max_new, page) + 1
    need = sum(max(R.ceil_div(int(n), page) - h, 0) for n, h in zip(new, have))
    n_pages = sum(have) + need + spare
    perm = rng.permutation(n_pages)
    table = -7 * np.ones((n_seqs, ld), dtype=np.int64)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = perm[at:at + h]
        at += h
    first = int(rng.integers(0, n_pages))
    ring = -9 * np.ones(n_pages, dtype=np.int64)
    for i, p in enumerate(perm[at:]):
        ring[(first + i) % n_pages] = p
    sizes = np.maximum(new - old, 0)
    n_tokens = int(sizes.sum()) + pad
    parents = None
    if tree:
        parents = sum((R.random_tree(rng, int(s)) for s in sizes), []) + [-1] * pad
    return dict(old=old, new=new, table=table, ring=ring, first=first, count=n_pages - at, page=page,
                n_tokens=n_tokens, parents=parents, max_new=max_new,
                max_ctx=int(max(old.max(), new.max())))


def run_tables(m, c, words, in_place=True):
    pages = PageTable(c["page"], i32(c["table"]), i32(c["ring"]), i32([c["first"], c["count"]]),
                      None if in_place else i32([0, 0]))
    step = Step.alloc(len(c["old"]), c["n_tokens"], c["max_new"], c["max_ctx"], i32(c["old"]),
                      i32(c["new"]), None if c["parents"] is None else i32(c["parents"]), words)
    m.step_tables(pages, step)
    return pages, step


def check_tables(c, words, pages, step):
    table, ring = c["table"].tolist(), c["ring"].tolist()
    first, count, q_start, slots, pos, seq, masks = R.step_tables(
        c["old"].tolist(), c["new"].tolist(), table, ring, c["first"], c["count"], c["page"],
        c["n_tokens"], c["parents"], words)
    assert pages.free_next.tolist() == [first, count]
    assert pages.table.tolist() == table
    assert pages.free_ring.tolist() == ring
    assert step.q_start.tolist() == q_start
    assert step.slots.tolist() == slots
    assert step.positions.tolist() == pos
    assert step.token_seq.tolist() == seq
    if words:
        got = step.tree_mask.cpu().numpy().view(np.uint64).tolist()
        assert got == masks


@pytest.mark.parametrize("n_seqs,max_new,page,max_len,tree,shrink,words", [
    (1, 1, 8, 0, False, 0.0, 0),
    (1, 1, 8, 40, True, 0.0, 1),
    (7, 9, 16, 100, True, 0.3, 1),
    (33, 64, 24, 300, True, 0.2, 1),
    (5, 200, 16, 500, True, 0.0, 4),
    (9, 130, 40, 90, False, 0.5, 3),
    (600, 5, 8, 60, True, 0.4, 2),
    (3, 5000, 64, 100, False, 0.0, 0),
    (1100, 3, 128, 1000, False, 0.5, 0),
])
def test_step_tables(n_seqs, max_new, page, max_len, tree, shrink, words):
    rng = np.random.default_rng(n_seqs * 131 + max_new)
    m = model()
    for in_place in (True, False):
        c = tables_case(rng, n_seqs, max_new, page, max_len, tree, shrink)
        pages, step = run_tables(m, c, words, in_place)
        check_tables(c, words, pages, step)
        if not in_place:  # a proposal: the same call again gives the same tables
            before = step.slots.clone()
            m.step_tables(pages, step)
            assert torch.equal(before, step.slots)
            check_tables(c, words, pages, step)
    assert m.check_device() == 0


def test_step_tables_most_sequences():
    rng = np.random.default_rng(5)
    m = model()
    c = tables_case(rng, 8192, 1, 8, 20, False, 0.2, spare=0)
    pages, step = run_tables(m, c, 0)
    check_tables(c, 0, pages, step)
    assert m.check_device() == 0


def test_step_tables_pages_come_back():
    """Steps that grow and shrink until every page has been round the ring."""
    rng = np.random.default_rng(8)
    m = model()
    n, page, n_pages = 6, 8, 40
    pages = PageTable.alloc(n, n_pages, page, 64)
    lens = [0] * n
    table, ring, first, count = pages.table.tolist(), pages.free_ring.tolist(), 0, n_pages
    step = Step.alloc(n, 64 * n, 64, 64)
    for _ in range(40):
        new = [int(rng.integers(0, 50)) if rng.random() < 0.7 else 0 for _ in range(n)]
        need = sum(max(R.ceil_div(a, page) - R.ceil_div(b, page), 0) for a, b in zip(new, lens))
        if need > count:
            new = [0] * n
        step.old_lens.copy_(i32(lens))
        step.new_lens.copy_(i32(new))
        m.step_tables(pages, step)
        first, count, q_start, slots, *_ = R.step_tables(lens, new, table, ring, first, count, page,
                                                         64 * n)
        assert pages.free_state.tolist() == [first, count]
        assert step.slots.tolist() == slots and step.q_start.tolist() == q_start
        owned = [p for b in range(n) for p in table[b][:R.ceil_div(new[b], page)]]
        assert len(set(owned)) == len(owned) and len(owned) + count == n_pages
        lens = new
    assert m.check_device() == 0


@pytest.mark.parametrize("what", ["pages", "old", "new", "long", "many", "tokens", "ring", "count"])
def test_step_tables_refuse_as_a_whole(what):
    rng = np.random.default_rng(3)
    m = model()
    c = tables_case(rng, 5, 6, 8, 40, True, 0.2)
    if what == "pages":
        c["count"] = 0
        c["old"][:], c["new"][:] = 8, 9
    elif what == "old":
        c["old"][2] = -1
    elif what == "new":
        c["new"][1] = -5
    elif what == "long":
        c["new"][3] = c["table"].shape[1] * 8 + 1
        c["old"][3] = c["new"][3] - 1
        c["max_ctx"] = 10**6
    elif what == "many":
        c["new"][0] = c["old"][0] + 7
        c["max_ctx"] = 10**6
    elif what == "tokens":
        c["n_tokens"] = int(np.maximum(c["new"] - c["old"], 0).sum()) - 1
        c["parents"] = c["parents"][:c["n_tokens"]]
    elif what == "ring":
        c["first"] = len(c["ring"])
    elif what == "count":
        c["count"] = len(c["ring"]) + 1
    pages, step = run_tables(m, c, 1, in_place=False)
    assert m.check_device() == TABLE_RANGE
    assert pages.table.tolist() == c["table"].tolist()
    assert pages.free_ring.tolist() == c["ring"].tolist()
    assert pages.free_next.tolist() == [c["first"], c["count"]]
    assert step.q_start.tolist() == [0] * 6
    assert step.slots.tolist() == [-1] * c["n_tokens"] == step.token_seq.tolist()
    assert step.positions.tolist() == [0] * c["n_tokens"]
    assert not step.tree_mask.any()
    assert m.check_device() == 0


def test_step_tables_bad_parent_and_bad_page():
    rng = np.random.default_rng(4)
    m = model()
    c = tables_case(rng, 3, 8, 8, 30, True, 0.0)
    c["old"][:], c["new"][:] = [3, 5, 9], [9, 9, 12]
    c["table"][:, :2] = [[0, 1], [2, 3], [4, 5]]
    c["ring"][:] = np.arange(len(c["ring"]))
    c["first"], c["count"] = 6, len(c["ring"]) - 6
    c["n_tokens"], c["max_ctx"] = 16, 40
    c["parents"] = [-1, 0, 5, 1, 0, -3, -1, 0, 1, 2, -1, 0, 1, -1, -1, -1]
    good = dict(c, parents=[-1, 0, -1, 1, 0, -1] + c["parents"][6:])
    pages, step = run_tables(m, c, 1)
    assert m.check_device() == TABLE_RANGE
    check_tables(good, 1, pages, step)
    c["table"][2, 1] = len(c["ring"])  # the page of sequence 2's new tokens
    pages, step = run_tables(m, dict(c, parents=good["parents"]), 1)
    assert m.check_device() == TABLE_RANGE
    assert step.slots.tolist()[10:13] == [-1, -1, -1] and min(step.slots.tolist()[:10]) >= 0


@pytest.mark.parametrize("value", [-1, "n_pages", 2**31 - 1, -2**31])
@pytest.mark.parametrize("n_seqs,which", [(5, 1), (600, 599)])
def test_step_tables_bad_page_given_back(n_seqs, which, value):
    """A page number outside the cache in a row that shrinks must not get into the ring: nothing
    moves, in every CTA's part of the step, and the step goes through once the row is mended."""
    rng = np.random.default_rng(6)
    m = model()
    for at in (0, 2):  # of the three pages that it gives back
        c = tables_case(rng, n_seqs, 9, 8, 60, True, 0.2)
        c["old"][which], c["new"][which] = 30, 7
        have = [R.ceil_div(int(o), 8) for o in c["old"]]
        n = len(c["ring"]) + 4  # room for that sequence's pages, whatever it held before
        perm = rng.permutation(n)
        table, used = -7 * np.ones_like(c["table"]), 0
        for b, h in enumerate(have):
            table[b, :h] = perm[used:used + h]
            used += h
        c["table"], c["count"] = table, n - used
        c["ring"], c["first"] = np.roll(np.concatenate([perm[used:], -9 * np.ones(used, dtype=np.int64)]), 11), 11
        sizes = np.maximum(c["new"] - c["old"], 0)
        c["n_tokens"] = int(sizes.sum()) + 3
        c["parents"] = sum((R.random_tree(rng, int(s)) for s in sizes), []) + [-1] * 3
        c["max_ctx"] = int(max(c["old"].max(), c["new"].max()))
        good, bad = dict(c), dict(c, table=table.copy())
        bad["table"][which, 1 + at] = n if value == "n_pages" else value
        for in_place in (False, True):
            pages, step = run_tables(m, bad, 1, in_place)
            assert m.check_device() == TABLE_RANGE
            assert pages.table.tolist() == bad["table"].tolist()
            assert pages.free_ring.tolist() == bad["ring"].tolist()
            assert pages.free_next.tolist() == [bad["first"], bad["count"]]
            assert not step.q_start.any() and not step.tree_mask.any() and not step.positions.any()
            assert step.slots.tolist() == [-1] * bad["n_tokens"] == step.token_seq.tolist()
        pages, step = run_tables(m, good, 1)
        check_tables(good, 1, pages, step)
        assert m.check_device() == 0


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
HEADS = [(32, 8, 128, 8, 1), (40, 4, 128, 8, 1), (8, 8, 64, 4, 1), (28, 4, 128, 1, 1),
         (16, 2, 64, 8, 2)]


def append_reference(m, qkv, pos, slots, k, v, page):
    c = m.cfg
    nq, kvr, rep, d = c.q_heads_per_rank, c.kv_heads_per_rank, c.kv_replicas, c.head_dim
    M = qkv.shape[1]
    x = qkv.reshape(c.attn_tp, M, nq + 2 * kvr, d)
    rot = np.stack([R.rotate(x[r, :, :nq + kvr], pos, c.rope_theta) for r in range(c.attn_tp)])
    q = rot[:, :, :nq].transpose(1, 0, 2, 3).reshape(M, -1)
    mag = np.abs(x[:, :, :nq + kvr])
    mag = mag + np.roll(mag, d // 2, axis=-1)
    qmag = mag[:, :, :nq].transpose(1, 0, 2, 3).reshape(M, -1)
    kmag = np.zeros_like(k)
    for i, s in enumerate(slots):
        if s < 0:
            continue
        for copy in range(c.kv_copies):
            k[copy, s // page, :, s % page] = rot[copy * rep, i, nq:]
            v[copy, s // page, :, s % page] = x[copy * rep, i, nq + kvr:]
            kmag[copy, s // page, :, s % page] = mag[copy * rep, i, nq:]
    return q, qmag, k, kmag, v


def near(got, ref, mag):
    assert np.all(np.abs(got - ref) <= 2.0**-8 * np.abs(ref) + 4 * 2.0**-24 * mag)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("M,page", [(1, 8), (7, 24), (301, 64), (1003, 16)])
def test_cache_append(heads, M, page):
    h, kv, d, t, dp = heads
    rng = np.random.default_rng(M + h)
    m = model(h, kv, d, t, attn_dp=dp)
    n_pages = R.ceil_div(M, page) + 2
    qkv = bf16(rng, m.cfg.attn_tp, M, m.qkv_rows())
    pos = rng.integers(0, 20000, M)
    pos[-1] = 19999
    slots = rng.permutation(n_pages * page)[:M]
    if M > 1:
        slots[rng.integers(0, M, M // 4 + 1)] = -1
    k, v = (bf16(rng, m.cfg.kv_copies, n_pages, m.cfg.kv_heads_per_rank, page, d) for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    rq, qmag, rk, kmag, rv = append_reference(m, f64(qkv), pos, slots, f64(k), f64(v), page)
    pages = PageTable(page, n_pages=n_pages)
    q = m.cache_append(qkv, i32(pos), i32(slots), pages, k, v)
    near(f64(q), rq, qmag)
    near(f64(k), rk, kmag)
    assert np.array_equal(f64(v), rv)
    # strided q, and no q: the cache is the same either way
    for want_q in (True, False):
        k2, v2 = k0.clone(), v0.clone()
        wide = torch.full((M, h * d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        got = m.cache_append(qkv, i32(pos), i32(slots), pages, k2, v2,
                             q=wide[:, 8:-8] if want_q else None, want_q=want_q)
        assert torch.equal(k2, k) and torch.equal(v2, v)
        if want_q:
            assert torch.equal(wide[:, 8:-8], q) and torch.all(wide[:, :8] == 7)
        else:
            assert got is None
    assert m.check_device() == 0


def test_cache_append_rows_out_of_range():
    rng = np.random.default_rng(1)
    m = model(8, 4, 64, 2)
    qkv = bf16(rng, 2, 4, m.qkv_rows())
    k, v = (bf16(rng, 2, 3, 2, 8, 64) for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    pages = PageTable(8, n_pages=3)
    for pos, slots in (([0, 20000, 5, 3], [3, 4, -1, -1]), ([0, -1, 5, 3], [3, 4, -1, -1]),
                       ([0, 9, 5, 3], [3, 24, -1, -1]), ([0, 9, 5, 3], [3, -2, -1, -1])):
        k.copy_(k0)
        v.copy_(v0)
        q = m.cache_append(qkv, i32(pos), i32(slots), pages, k, v)
        assert m.check_device() == TABLE_RANGE
        assert bool(q[1].any()) == (0 <= pos[1] < 20000)
        assert torch.all(q[0].any()) and torch.all(q[2].any())
        k[:, 0, :, 3] = k0[:, 0, :, 3]
        v[:, 0, :, 3] = v0[:, 0, :, 3]
        assert torch.equal(k, k0) and torch.equal(v, v0)  # only row 0 was stored
    assert m.check_device() == 0


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attn_case(rng, m, ctx, T, page, tree=True, pad=2, q_scale=1.0, poison=None, mask=None, spare=2):
    """Inputs over a cache whose unowned slots hold `poison` (NaN by default)."""
    c = m.cfg
    n, d = len(ctx), c.head_dim
    have = [R.ceil_div(a + b, page) for a, b in zip(ctx, T)]
    ld, n_pages = max(max(have), 1), sum(have) + spare
    perm = rng.permutation(n_pages)
    table = -np.ones((n, ld), dtype=np.int64)
    shape = (c.kv_copies, n_pages, c.kv_heads_per_rank, page, d)
    k = torch.full(shape, float("nan") if poison is None else poison, dtype=torch.bfloat16,
                   device="cuda")
    v = k.clone()
    dense = []
    at = 0
    for b in range(n):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
        L = ctx[b] + T[b]
        kb, vb = (bf16(rng, L, c.kv_copies, c.kv_heads_per_rank, d) for _ in range(2))
        j = torch.arange(L)
        pg = torch.from_numpy(table[b])[j // page].cuda()
        off = (j % page).cuda()
        k[:, pg, :, off] = kb
        v[:, pg, :, off] = vb
        dense.append((f64(kb).reshape(L, c.n_kv_heads, d), f64(vb).reshape(L, c.n_kv_heads, d)))
    M = sum(T) + pad
    if mask is None:
        if tree:
            mask = [R.tree_bits(R.random_tree(rng, t)) for t in T]
        else:
            mask = [np.tril(np.ones((t, t), dtype=bool)) for t in T]
    words = max(1, R.ceil_div(max(T), 64))
    packed = np.zeros((M, words), dtype=np.int64)
    q0 = 0
    for b, t in enumerate(T):
        packed[q0:q0 + t] = R.pack_bits(mask[b], words)
        q0 += t
    start = np.concatenate([[0], np.cumsum(T)])
    q = bf16(rng, M, c.n_heads * d, scale=q_scale)
    step = Step(n_tokens=M, max_new=max(max(T), 1), max_ctx=max(a + b for a, b in zip(ctx, T)),
                old_lens=i32(ctx), q_start=i32(start),
                tree_mask=torch.from_numpy(packed).cuda() if tree else None)
    return dict(ctx=ctx, T=T, q=q, k=k, v=v, dense=dense, mask=mask, start=start, step=step,
                pages=PageTable(page, i32(table), n_pages=n_pages), table=table, page=page)


def check_attn(m, c, out, rows=None):
    """Every row (or those `rows` picks) against the 64-bit form."""
    d, group = m.cfg.head_dim, m.cfg.n_heads // m.cfg.n_kv_heads
    q, got = f64(c["q"]), f64(out)
    for b in range(len(c["ctx"])):
        k, v = c["dense"][b]
        for i in range(c["T"][b]):
            row = c["start"][b] + i
            if rows is not None and not rows(b, i):
                continue
            sees = np.concatenate([np.ones(c["ctx"][b], dtype=bool), c["mask"][b][i]])
            for h in range(m.cfg.n_heads):
                o, A, S = R.attention_row(q[row, h * d:(h + 1) * d], k[:, h // group],
                                          v[:, h // group], sees)
                tol = 2.0**-8 * np.abs(o) + (2.0**-8 + 2 * ((d + 4) * 2.0**-24 * S + 2.0**-19)) * A
                err = np.abs(got[row, h * d:(h + 1) * d] - o)
                assert np.all(err <= tol), (b, i, h, float((err - tol).max()))


ATTN_HEADS = [(8, 2, 64, 2), (8, 2, 128, 4), (5, 1, 128, 1), (4, 4, 64, 4), (16, 1, 128, 1)]


@pytest.mark.parametrize("heads", ATTN_HEADS)
@pytest.mark.parametrize("ctx,T,page,tree", [
    ([0], [1], 8, True),
    ([1], [1], 16, False),
    ([63, 64, 65, 127, 128, 129], [1, 1, 1, 1, 1, 1], 16, True),
    ([0, 40, 300, 0, 7], [3, 0, 17, 1, 33], 24, True),
    ([120, 0, 500], [9, 70, 40], 64, False),
    ([250], [130], 40, True),
    ([1000, 3], [5, 2], 1024, True),
])
def test_tree_attention(heads, ctx, T, page, tree):
    h, kv, d, t = heads
    rng = np.random.default_rng(sum(ctx) + h + d)
    m = model(h, kv, d, t)
    c = attn_case(rng, m, ctx, T, page, tree)
    out = torch.full_like(c["q"], 3.0)
    m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"], out=out)
    assert torch.all(out[sum(T):] == 3.0)  # padding rows as they were
    check_attn(m, c, out)
    again = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    assert torch.equal(again[:sum(T)], out[:sum(T)])  # deterministic
    assert m.check_device() == 0


@pytest.mark.parametrize("heads", [(16, 2, 64, 8, 2), (8, 4, 128, 4, 4), (8, 2, 64, 4, 2)])
def test_tree_attention_with_dp_attention(heads):
    """The heads sharded over t / attn_dp ranks: fewer cache copies, more heads in each."""
    h, kv, d, t, dp = heads
    rng = np.random.default_rng(h + t)
    m = model(h, kv, d, t, attn_dp=dp)
    c = attn_case(rng, m, [0, 40, 300], [3, 1, 17], 24)
    assert c["k"].shape[0] == min(t // dp, kv)
    out = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    check_attn(m, c, out)
    assert m.check_device() == 0


@pytest.mark.parametrize("heads", [(32, 8, 128, 8), (32, 4, 64, 2)])
def test_tree_attention_full_trees(heads):
    """256 drafted tokens (many query tiles) next to a single one, long and short contexts."""
    h, kv, d, t = heads
    rng = np.random.default_rng(2)
    m = model(h, kv, d, t)
    c = attn_case(rng, m, [700, 2100], [256, 1], 16)
    out = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    check_attn(m, c, out, rows=lambda b, i: i % 37 == 0 or i == 255)
    assert m.check_device() == 0


def test_tree_attention_many_sequences():
    rng = np.random.default_rng(12)
    m = model(8, 2, 64, 2)
    ctx = rng.integers(0, 60, 700).tolist()
    T = rng.integers(0, 3, 700).tolist()
    c = attn_case(rng, m, ctx, T, 8)
    out = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    check_attn(m, c, out, rows=lambda b, i: b % 11 == 0)
    assert m.check_device() == 0


def test_tree_attention_long_context_of_one_sequence():
    """One sequence spread over every SM: the pieces' join."""
    rng = np.random.default_rng(21)
    m = model(4, 1, 128, 1)
    for T in (1, 40):
        c = attn_case(rng, m, [30001], [T], 64)
        out = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
        check_attn(m, c, out, rows=lambda b, i: i % 13 == 0)
    assert m.check_device() == 0


@pytest.mark.parametrize("scale", [1e-3, 40.0])
def test_tree_attention_flat_and_peaked_scores(scale):
    rng = np.random.default_rng(31)
    m = model(8, 2, 128, 4)
    c = attn_case(rng, m, [333, 10], [12, 4], 16, q_scale=scale)
    out = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    check_attn(m, c, out)


def test_tree_attention_rising_maximum():
    """Keys that grow along the sequence: the running maximum moves in every tile."""
    rng = np.random.default_rng(32)
    m = model(4, 1, 128, 1)
    c = attn_case(rng, m, [1500], [3], 16, tree=False)
    k = c["dense"][0][0]
    L = k.shape[0]
    u = rng.standard_normal(128)
    grown = torch.from_numpy((u[None, :] * np.linspace(-3, 3, L)[:, None]).astype(np.float32)).bfloat16()
    j = torch.arange(L)
    c["k"][0, torch.from_numpy(c["table"][0])[j // 16].cuda(), 0, (j % 16).cuda()] = grown.cuda()
    c["dense"][0] = (f64(grown)[:, None, :], c["dense"][0][1])
    c["q"].copy_(torch.from_numpy(np.tile(u, (c["q"].shape[0], 4)).astype(np.float32)))
    out = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    check_attn(m, c, out)


def test_tree_attention_rows_that_see_nothing():
    rng = np.random.default_rng(33)
    m = model(8, 2, 64, 2)
    empty = [np.zeros((5, 5), dtype=bool), np.eye(70, dtype=bool), np.zeros((4, 4), dtype=bool)]
    empty[0][3, 1] = True
    empty[1][::2] = False
    c = attn_case(rng, m, [0, 0, 9], [5, 70, 4], 8, mask=empty)
    out = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    check_attn(m, c, out)
    assert not out[0].any() and not out[5].any() and out[75].any()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), -3.3e38])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("where", ["k", "v", "kv"])
def test_tree_attention_unseen_keys_do_not_matter(value, tree, where):
    """Drafted tokens that a row does not see, and slots nobody owns, hold infinities and NaN."""
    rng = np.random.default_rng(34)
    m = model(8, 2, 128, 4)
    ctx, T = [130, 0, 77], [40, 9, 3]
    c = attn_case(rng, m, ctx, T, 16, tree, poison=value)
    bad = [7, 30]  # tokens of sequence 0
    for t in bad:
        j = ctx[0] + t
        pg, off = int(c["table"][0, j // 16]), j % 16
        for name in where:
            c[name][:, pg, :, off, ::3] = value
    sees_bad = c["mask"][0][:, bad].any(axis=1)
    assert sees_bad.any() and not sees_bad.all()
    out = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    check_attn(m, c, out, rows=lambda b, i: b > 0 or not sees_bad[i])
    if not np.isfinite(value) and where == "v":  # rows that see it show it
        rows = f64(out)[:T[0]][sees_bad].reshape(sees_bad.sum(), -1, 128)
        assert not np.isfinite(rows[:, :, ::3]).any()
        assert np.isfinite(rows[:, :, 1::3]).all()
        if np.isinf(value):
            one = c["mask"][0][sees_bad][:, bad].sum(axis=1) == 1
            assert (rows[one][:, :, ::3] == value).all()


def test_tree_attention_time_does_not_hang_on_padding_queries():
    """Rows of a query tile behind the item's own hold other queries, here padding; NaN among
    them must not make every tile look like one that raises the maximum.  (Both sides in turn,
    the fastest of ten graphs each: they agree to 2 %; with such rows in the vote NaN took 18 %
    more.)"""
    rng = np.random.default_rng(38)
    m = model(32, 8, 128, 8)
    c = attn_case(rng, m, [20000], [1], 64, pad=31)
    out, graphs, q = torch.zeros_like(c["q"]), [], [c["q"].clone(), c["q"].clone()]
    q[0][1:], q[1][1:] = 0.0, float("nan")
    m.tree_attention(q[0], c["step"], c["pages"], c["k"], c["v"], out=out)
    torch.cuda.synchronize()
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(30):
                m.tree_attention(x, c["step"], c["pages"], c["k"], c["v"], out=out)
        graphs.append(g)
    times = [[], []]
    for _ in range(11):
        for g, t in zip(graphs, times):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            t.append(a.elapsed_time(b))
    zeros, nans = (min(t[1:]) for t in times)
    assert nans < 1.09 * zeros, (zeros / 30, nans / 30)
    check_attn(m, c, out)


def test_tree_attention_strided_rows():
    rng = np.random.default_rng(35)
    m = model(8, 2, 64, 2)
    c = attn_case(rng, m, [90, 5], [6, 11], 16)
    M = c["q"].shape[0]
    wide = torch.zeros((M, 3 * 512), dtype=torch.bfloat16, device="cuda")
    wide[:, 512:1024] = c["q"]
    ref = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    into = torch.full((M, 512 + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    m.tree_attention(wide[:, 512:1024], c["step"], c["pages"], c["k"], c["v"], out=into[:, :512])
    assert torch.equal(into[:17, :512], ref[:17]) and torch.all(into[:, 512:] == 5)


def test_tree_attention_pages_past_32_bits():
    """Element offsets above 2^32 in a large cache."""
    rng = np.random.default_rng(36)
    m = model(8, 2, 128, 1)
    n_pages, page = 70000, 256  # 70000 * 2 * 256 * 128 elements = 4.6e9
    k = torch.zeros((1, n_pages, 2, page, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = attn_case(rng, m, [600], [4], page)
    small = c["table"][0]
    far = np.array([n_pages - 1, 66001, 3][:len(small)])
    k[:, far], v[:, far] = c["k"][:, small], c["v"][:, small]
    pages = PageTable(page, i32(far[None, :]), n_pages=n_pages)
    out = m.tree_attention(c["q"], c["step"], pages, k, v)
    check_attn(m, c, out)
    # and the store into the last page
    qkv = bf16(rng, 1, 1, m.qkv_rows())
    m.cache_append(qkv, i32([0]), i32([n_pages * page - 1]), pages, k, v)
    assert torch.equal(v[0, -1, :, -1].flatten(), qkv[0, 0, 10 * 128:])
    assert m.check_device() == 0


def test_tree_attention_bad_tables():
    rng = np.random.default_rng(37)
    m = model(8, 2, 64, 2)
    c = attn_case(rng, m, [100, 50, 30], [4, 5, 6], 16)
    pages, step = c["pages"], c["step"]
    good = m.tree_attention(c["q"], step, pages, c["k"], c["v"])
    # a page number outside the cache reads as zeros: sequence 1's keys lose one page
    for bad in (-1, pages.n_pages, 2**31 - 1, -2**31):
        table = i32(c["table"])
        table[1, 0] = bad
        other = PageTable(16, table, n_pages=pages.n_pages)
        out = m.tree_attention(c["q"], step, other, c["k"], c["v"])
        assert m.check_device() == TABLE_RANGE
        assert torch.equal(out[:4], good[:4]) and torch.equal(out[9:15], good[9:15])
        dense = c["dense"][1]
        z = [x.copy() for x in dense]
        for x in z:
            x[:16] = 0
        c["dense"][1] = tuple(z)
        check_attn(m, c, out)
        c["dense"][1] = dense
    # lengths and starts outside their bounds: those sequences are skipped
    for what in ("neg", "long", "start", "rows", "wide"):
        lens, start = c["ctx"].copy(), c["start"].copy()
        if what == "neg":
            lens[1] = -1
        elif what == "long":
            lens[1] = step.max_ctx
        elif what == "start":
            start[1], start[2] = start[2], start[1]
        elif what == "rows":
            start[3] = c["q"].shape[0] + 1
        else:
            start = np.array([0, 4, 15, 15])  # 11 new tokens: more than max_new
        s2 = Step(step.n_tokens, step.max_new, step.max_ctx, i32(lens), q_start=i32(start),
                  tree_mask=step.tree_mask)
        out = torch.full_like(c["q"], 9.0)
        m.tree_attention(c["q"], s2, pages, c["k"], c["v"], out=out)
        assert m.check_device() == TABLE_RANGE
        if what in ("neg", "long"):
            assert torch.all(out[4:9] == 9.0)
            assert torch.equal(out[:4], good[:4]) and torch.equal(out[9:15], good[9:15])
        elif what == "rows":
            assert torch.all(out[9:] == 9.0) and torch.equal(out[:9], good[:9])
        elif what == "wide":
            assert torch.all(out[4:] == 9.0) and torch.equal(out[:4], good[:4])
    assert m.check_device() == 0


# ---------------------------------------------------------------------------
# logits
# ---------------------------------------------------------------------------
def check_logits(got, ref, mag, is_bf16):
    tol = 6 * 2.0**-24 * mag + (2.0**-8 * np.abs(np.where(np.isfinite(ref), ref, 0)) if is_bf16 else 0)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref))
    fin = np.isfinite(ref)
    assert np.all(np.abs(got[fin] - ref[fin]) <= tol[fin])


def logits_case(rng, V, reqs, nodes=1, history=40, biases=6, grammar=True, pad=1):
    S = reqs * nodes + pad
    words = R.ceil_div(V, 32)
    row_req = np.concatenate([np.repeat(np.arange(reqs), nodes), -np.ones(pad)]).astype(np.int64)
    hist = rng.integers(0, max(2, V // 7), (reqs, history))
    hist[rng.random(hist.shape) < 0.05] = -1
    hist[rng.random(hist.shape) < 0.05] = V
    lens = rng.integers(0, history + 1, reqs)
    lens[0] = history
    prompt = (lens * rng.random(reqs)).astype(np.int64)
    rep, freq, pres = rng.uniform(0.5, 2, reqs), rng.uniform(-1, 1, reqs), rng.uniform(-1, 1, reqs)
    count = rng.integers(0, biases + 1, reqs)
    ids = rng.integers(0, V, int(count.sum()))
    if len(ids) > 3:
        ids[1] = ids[0]
        ids[-1] = V
    start = np.concatenate([[0], np.cumsum(count)])
    vals = rng.standard_normal(len(ids)) * 5
    parents = [R.random_tree(rng, nodes) for _ in range(reqs)]
    draft = rng.integers(0, max(2, V // 7), S)
    bits = [R.tree_bits(p) for p in parents]
    allowed = rng.random((S, 32 * words)) < 0.7
    allowed_row = rng.permutation(S)
    allowed_row[0] = -1
    return dict(V=V, S=S, reqs=reqs, nodes=nodes, row_req=row_req, hist=hist, lens=lens, prompt=prompt,
                rep=rep.astype(np.float32), freq=freq.astype(np.float32), pres=pres.astype(np.float32),
                ids=ids, start=start, vals=vals.astype(np.float32), draft=draft, bits=bits,
                allowed=allowed, allowed_row=allowed_row, grammar=grammar, tree=nodes > 1)


def rules_of(c):
    f32 = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    kw = dict(row_req=i32(c["row_req"]), history=i32(c["hist"]), history_lens=i32(c["lens"]),
              prompt_lens=i32(c["prompt"]), repetition=f32(c["rep"]), frequency=f32(c["freq"]),
              presence=f32(c["pres"]), bias_start=i32(c["start"]), bias_ids=i32(c["ids"]),
              bias_values=f32(c["vals"]))
    if c["tree"]:
        mask = np.zeros((c["S"], 1), dtype=np.int64)
        mask[:c["reqs"] * c["nodes"]] = np.concatenate([R.pack_bits(b, 1) for b in c["bits"]])
        kw.update(draft_tokens=i32(c["draft"]), tree_mask=torch.from_numpy(mask).cuda(),
                  q_start=i32(np.arange(c["reqs"] + 1) * c["nodes"]))
    if c["grammar"]:
        words = c["allowed"].reshape(c["S"], -1, 32)
        packed = (words.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
        kw.update(allowed=torch.from_numpy(packed.view(np.int32)).cuda(), allowed_row=i32(c["allowed_row"]))
    return LogitRules(**kw)


def logits_reference(c, x):
    ref, mag = np.empty_like(x), np.empty_like(x)
    for s in range(c["S"]):
        r = int(c["row_req"][s])
        if r < 0:
            continue
        h = c["hist"][r][:c["lens"][r]]
        out = list(h[c["prompt"][r]:])
        if c["tree"]:
            out += [c["draft"][r * c["nodes"] + t] for t in np.nonzero(c["bits"][r][s % c["nodes"]])[0]]
        ok = None
        if c["grammar"] and c["allowed_row"][s] >= 0:
            ok = c["allowed"][c["allowed_row"][s]][:c["V"]]
        b = slice(c["start"][r], c["start"][r + 1])
        ref[s], mag[s] = R.logit_row(x[s], h[:c["prompt"][r]], out, float(c["rep"][r]),
                                     float(c["freq"][r]), float(c["pres"][r]),
                                     list(zip(c["ids"][b].tolist(), c["vals"][b].tolist())), ok)
    return ref, mag


@pytest.mark.parametrize("V", [1, 31, 1000, 8192, 8193, 32003, 128256])
@pytest.mark.parametrize("reqs,nodes,grammar", [(1, 1, True), (5, 1, False), (3, 11, True)])
def test_process_logits(V, reqs, nodes, grammar):
    rng = np.random.default_rng(V + reqs)
    m = model(vocab=V)
    c = logits_case(rng, V, reqs, nodes, grammar=grammar)
    x = bf16(rng, c["S"], V, scale=4.0)
    ref, mag = logits_reference(c, f64(x))
    rules = rules_of(c)
    live = c["row_req"] >= 0
    for out in (torch.full((c["S"], V), 6.0, device="cuda"),
                torch.full((c["S"], V + 5), 6.0, device="cuda")[:, 1:V + 1],
                torch.full((c["S"], V), 6.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((c["S"], V + 3), 6.0, dtype=torch.bfloat16, device="cuda")[:, 2:V + 2]):
        m.process_logits(x, rules, out=out)
        check_logits(f64(out)[live], ref[live], mag[live], out.dtype == torch.bfloat16)
        assert torch.all(out[~torch.from_numpy(live).cuda()] == 6)
    # strided and misaligned input, in place
    wide = torch.full((c["S"], V + 9), 2.5, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:V + 3] = x
    view = wide[:, 3:V + 3]
    same = m.process_logits(view, rules, out=view)
    check_logits(f64(same)[live], ref[live], mag[live], True)
    assert torch.all(wide[:, :3] == 2.5) and torch.all(wide[:, V + 3:] == 2.5)
    assert torch.equal(view[-1], x[-1])  # row_req -1
    assert m.check_device() == 0


def test_process_logits_long_history_and_paths():
    rng = np.random.default_rng(50)
    V = 20000
    m = model(vocab=V)
    c = logits_case(rng, V, 2, 64, history=9000, biases=300)
    x = bf16(rng, c["S"], V, scale=4.0)
    ref, mag = logits_reference(c, f64(x))
    live = c["row_req"] >= 0
    out = m.process_logits(x, rules_of(c))
    check_logits(f64(out)[live], ref[live], mag[live], False)
    assert torch.equal(out[:-1], m.process_logits(x, rules_of(c))[:-1])


def test_process_logits_rules_one_by_one():
    """Each rule alone, and none."""
    rng = np.random.default_rng(51)
    V, S = 777, 4
    m = model(vocab=V)
    x = bf16(rng, S, V, scale=4.0)
    assert torch.equal(m.process_logits(x, LogitRules(n_reqs=S)), x.float())
    ids = rng.integers(0, V, (S, 20))
    hist = dict(history=i32(ids), history_lens=i32([20, 0, 7, 20]))
    p = torch.tensor([1.3, 0.7, 1.1, 2.0]).cuda()
    for name in ("repetition", "frequency", "presence"):
        out = f64(m.process_logits(x, LogitRules(**hist, **{name: p})))
        for s in range(S):
            n = [20, 0, 7, 20][s]
            kw = {{"repetition": "rep", "frequency": "freq", "presence": "pres"}[name]: float(p[s])}
            ref, mag = R.logit_row(f64(x)[s], (), ids[s][:n], **kw)
            check_logits(out[s], ref, mag, False)
    allowed = torch.zeros((S, 25), dtype=torch.int32, device="cuda")
    allowed[1, 0] = 1 << 5
    out = f64(m.process_logits(x, LogitRules(allowed=allowed)))
    assert np.isneginf(out[0]).all() and np.isneginf(out[2:]).all()  # nothing allowed
    assert np.isneginf(out[1]).sum() == V - 1 and out[1, 5] == f64(x)[1, 5]


def test_process_logits_infinities_and_nan():
    V = 300
    m = model(vocab=V)
    x = torch.zeros((1, V), dtype=torch.bfloat16, device="cuda")
    x[0, :6] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan"), float("inf"),
                             -float("inf")])
    allowed = np.full((1, 10), -1, dtype=np.int32)
    allowed[0, 0] = ~0b111  # 0, 1, 2 not allowed
    out = m.process_logits(x, LogitRules(
        history=i32([[3, 4, 5, 0, 1, 2]]), history_lens=i32([6]), repetition=torch.tensor([1.5]).cuda(),
        frequency=torch.tensor([0.5]).cuda(), presence=torch.tensor([0.25]).cuda(),
        allowed=torch.from_numpy(allowed).cuda()))[0].tolist()
    assert out[:3] == [-float("inf")] * 3
    assert out[3] != out[3] and out[4] == float("inf") and out[5] == -float("inf")
    assert out[6:] == [0.0] * (V - 6)


def test_process_logits_bad_indices():
    rng = np.random.default_rng(53)
    V, S = 500, 3
    m = model(vocab=V)
    x = bf16(rng, S, V)
    plain = x.float()
    hist = i32(rng.integers(0, V, (S, 10)))
    pres = torch.ones(S).cuda()
    full = m.process_logits(x, LogitRules(history=hist, history_lens=i32([10] * 3), presence=pres))
    assert m.check_device() == 0
    # lengths are cut
    out = m.process_logits(x, LogitRules(history=hist, history_lens=i32([11, 10, 10**9]), presence=pres))
    assert m.check_device() == TABLE_RANGE and torch.equal(out, full)
    out = m.process_logits(x, LogitRules(history=hist, history_lens=i32([-1, 10, 10]), presence=pres))
    assert m.check_device() == TABLE_RANGE
    assert torch.equal(out[0], plain[0]) and torch.equal(out[1:], full[1:])
    out = m.process_logits(x, LogitRules(history=hist, history_lens=i32([10] * 3), presence=pres,
                                         prompt_lens=i32([0, 11, -4])))
    assert m.check_device() == TABLE_RANGE
    assert torch.equal(out[0], full[0]) and torch.equal(out[1], plain[1]) and torch.equal(out[2], full[2])
    # requests
    into = torch.full((S, V), 4.0, device="cuda")
    m.process_logits(x, LogitRules(row_req=i32([0, 3, -2]), history=hist, history_lens=i32([10] * 3),
                                   presence=pres), out=into)
    assert m.check_device() == TABLE_RANGE
    assert torch.equal(into[0], full[0]) and torch.all(into[1:] == 4)
    # bias ranges
    ids, vals = i32([1, 2, 3]), torch.ones(3).cuda()
    for start in ([0, 1, 4, 3], [-1, 1, 2, 3], [2, 1, 2, 3]):
        out = m.process_logits(x, LogitRules(bias_start=i32(start), bias_ids=ids, bias_values=vals))
        assert m.check_device() == TABLE_RANGE
        for r in range(3):
            lo, hi = start[r], start[r + 1]
            want = plain[r].clone()
            if 0 <= lo <= hi <= 3:
                want[[1, 2, 3][lo:hi]] += 1
            assert torch.equal(out[r], want), (start, r)
    # paths outside the rows
    mask = torch.ones((S, 1), dtype=torch.int64, device="cuda")
    for start in ([0, 1, 2, 4], [-1, 1, 2, 3], [0, 2, 1, 3]):
        out = m.process_logits(x, LogitRules(draft_tokens=i32([5, 6, 7]), tree_mask=mask,
                                             q_start=i32(start), presence=pres))
        assert m.check_device() == TABLE_RANGE
        for r in range(3):
            want = plain[r].clone()
            if 0 <= start[r] < start[r + 1] <= 3:
                want[5 + start[r]] -= 1
            assert torch.equal(out[r], want), (start, r)
    # grammar rows
    allowed = torch.full((2, 16), -1, dtype=torch.int32, device="cuda")
    out = m.process_logits(x, LogitRules(allowed=allowed, allowed_row=i32([1, 2, -2]), n_reqs=S))
    assert m.check_device() == TABLE_RANGE
    assert torch.equal(out[0], plain[0]) and torch.isneginf(out[1:]).all()
    assert m.check_device() == 0


@pytest.mark.parametrize("V,reqs,nodes,history", [(1000, 3, 5, 40), (8192, 40, 1, 300), (32000, 90, 1, 2500),
                                                  (32000, 12, 16, 700), (20008, 7, 20, 20000)])
def test_process_logits_in_place_aligned(V, reqs, nodes, history):
    rng = np.random.default_rng(V + nodes)
    m = model(vocab=V)
    c = logits_case(rng, V, reqs, nodes, history=history, biases=20)
    x = bf16(rng, c["S"], V, scale=4.0)
    ref, mag = logits_reference(c, f64(x))
    live = c["row_req"] >= 0
    rules = rules_of(c)
    apart = m.process_logits(x, rules, dtype=torch.bfloat16)
    y = x.clone()
    m.process_logits(y, rules, out=y)
    check_logits(f64(y)[live], ref[live], mag[live], True)
    rows = torch.from_numpy(live).cuda()
    assert torch.equal(y[rows], apart[rows]) and torch.equal(y[~rows], x[~rows])
    assert m.check_device() == 0


@pytest.mark.parametrize("start", [[2**31 - 1, 2**31 - 1], [2**31 - 1, 3], [-(2**31), 2**31 - 1], [0, 2**31 - 1]])
def test_process_logits_bias_ranges_outside(start):
    rng = np.random.default_rng(56)
    m = model(8, 2, 64, 2)
    x = bf16(rng, 1, 1000)
    rules = LogitRules(n_reqs=1, bias_start=i32(start), bias_ids=i32([1, 2, 3]),
                       bias_values=torch.ones(3).cuda())
    got = m.process_logits(x, rules)
    bad = start[0] < 0 or start[1] < start[0] or start[1] > 3
    assert m.check_device() == (TABLE_RANGE if bad else 0)
    assert torch.equal(got, x.float())


@pytest.mark.parametrize("n", [40, 300, 700, 2000])
def test_process_logits_many_biases(n):
    """More biases than a CTA's threads keep, tokens named once and several times."""
    rng = np.random.default_rng(57)
    V = 40000
    m = model(8, 2, 64, 2, V)
    x = bf16(rng, 2, V)
    ids = rng.integers(0, V, (2, n))
    ids[1, n // 2:] = ids[1, :n - n // 2]
    vals = rng.standard_normal((2, n)).astype(np.float32)
    rules = LogitRules(n_reqs=2, bias_start=i32([0, n, 2 * n]), bias_ids=i32(ids.reshape(-1)),
                       bias_values=torch.from_numpy(vals.reshape(-1)).cuda())
    got = m.process_logits(x, rules).cpu().numpy()
    for r in range(2):
        add = np.zeros(V, dtype=np.float32)
        for i, y in zip(ids[r], vals[r]):
            add[i] += y  # in the list's order, as documented
        assert np.array_equal(got[r], x[r].float().cpu().numpy() + add)
    assert m.check_device() == 0


@pytest.mark.parametrize("rows", [4, 400])
def test_process_logits_rows_left_alone_are_not_looked_up(rows):
    """A padding row's other indices may hold anything."""
    rng = np.random.default_rng(55)
    V = 40000
    m = model(8, 2, 64, 2, V)
    x = bf16(rng, rows, V)
    req = np.where(np.arange(rows) % 2, -1, 0)
    which = np.where(req < 0, 2**30, 0)
    allowed = torch.full((1, R.ceil_div(V, 32)), -1, dtype=torch.int32, device="cuda")
    rules = LogitRules(row_req=i32(req), n_reqs=1, allowed=allowed, allowed_row=i32(which),
                       presence=torch.ones(1).cuda(), history=i32([[7, 9]]), history_lens=i32([2]))
    out = torch.full((rows, V), 3.0, device="cuda")
    m.process_logits(x, rules, out=out)
    assert torch.all(out[1::2] == 3.0)
    want = x[0::2].float()
    want[:, [7, 9]] -= 1.0
    assert torch.equal(out[0::2], want)
    assert m.check_device() == 0


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_refusals_of_the_c_calls():
    ARG, UNS, WS = (B.STATUS[s] for s in ("TP_ERR_ARG", "TP_ERR_UNSUPPORTED", "TP_ERR_WORKSPACE"))
    rng = np.random.default_rng(60)
    m = model(8, 2, 64, 2)
    c = attn_case(rng, m, [20], [3], 8)
    ws = m.step_workspace(1, 3)
    q, k, v, o = c["q"], c["k"], c["v"], torch.empty_like(c["q"])
    M = q.shape[0]

    def attn(q_=q.data_ptr(), ldq=512, o_=o.data_ptr(), ldo=512, k_=k.data_ptr(), v_=v.data_ptr(),
             w=ws.data_ptr(), wb=ws.numel(), pages={}, step={}):
        p, s = B.tp_pages_t(), B.tp_step_t()
        for dst, src, over in ((p, c["pages"].c, pages), (s, c["step"].c, step)):
            for name, _ in dst._fields_:
                setattr(dst, name, over.get(name, getattr(src, name)))
        return B.tp_tree_attention(m.handle, q_, ldq, o_, ldo, p, s, k_, v_, w, wb, 0)

    assert attn() == 0
    for kw in (dict(q_=0), dict(o_=0), dict(k_=0), dict(v_=0), dict(q_=q.data_ptr() + 2), dict(ldq=504),
               dict(ldo=500), dict(ldq=513), dict(o_=q.data_ptr()), dict(o_=q.data_ptr() + 1024),
               dict(pages=dict(table=0)), dict(pages=dict(ld_table=0)), dict(pages=dict(n_pages=0)),
               dict(pages=dict(page_size=0)), dict(step=dict(n_seqs=0)), dict(step=dict(n_tokens=-1)),
               dict(step=dict(max_new=-1)), dict(step=dict(max_ctx=-1)), dict(step=dict(old_lens=0)),
               dict(step=dict(q_start=0)), dict(step=dict(tree_words=0))):
        assert attn(**kw) == ARG, kw
    for kw in (dict(pages=dict(page_size=12)), dict(pages=dict(page_size=65544)),
               dict(pages=dict(n_pages=2**28)), dict(step=dict(n_seqs=8193)), dict(step=dict(max_new=257)),
               dict(step=dict(n_tokens=2**30 + 1)),
               dict(step=dict(max_new=65)), dict(step=dict(tree_words=5))):
        assert attn(**kw) == UNS, kw
    for kw in (dict(w=0), dict(w=ws.data_ptr() + 8), dict(wb=ws.numel() - 1)):
        assert attn(**kw) == WS, kw
    assert attn(step=dict(n_tokens=0)) == 0 and attn(step=dict(max_new=0)) == 0

    tc = tables_case(rng, 2, 3, 8, 20, True, 0.0)
    pages, step = run_tables(m, tc, 1)

    def tables(w=ws.data_ptr(), wb=ws.numel(), pages_={}, step_={}):
        p, s = B.tp_pages_t(), B.tp_step_t()
        for dst, src, over in ((p, pages.c, pages_), (s, step.c, step_)):
            for name, _ in dst._fields_:
                setattr(dst, name, over.get(name, getattr(src, name)))
        return B.tp_step_tables(m.handle, p, s, w, wb, 0)

    for name in ("table", "free_ring", "free_state", "free_next"):
        assert tables(pages_={name: 0}) == ARG, name
    for name in ("old_lens", "new_lens", "q_start", "slots", "positions", "token_seq", "tree_words",
                 "n_seqs"):
        assert tables(step_={name: 0}) == ARG, name
    for kw in (dict(max_new=65), dict(max_new=257, tree_words=5), dict(n_seqs=8193),
               dict(tree_mask=0, max_new=300), dict(n_tokens=2**30 + 1)):
        assert tables(step_=kw) == UNS, kw
    assert tables(w=0) == WS and tables(wb=8) == WS

    qkv = bf16(rng, 2, 4, m.qkv_rows())
    pos, slots = i32([0, 1, 2, 3]), i32([-1, -1, -1, -1])
    n_r = m.qkv_rows()

    def append(x=qkv.data_ptr(), rs=4 * n_r, n=4, p_=pos.data_ptr(), s_=slots.data_ptr(),
               k_=k.data_ptr(), v_=v.data_ptr(), q_=0, ldq=512, page=8):
        p = B.tp_pages_t()
        p.n_pages, p.page_size = c["pages"].n_pages, page
        return B.tp_cache_append(m.handle, x, rs, n, p_, s_, p, k_, v_, q_, ldq, 0)

    assert append() == 0 and append(n=0) == 0
    for kw in (dict(x=0), dict(rs=4 * n_r - 8), dict(rs=4 * n_r + 4), dict(n=-1), dict(p_=0), dict(s_=0),
               dict(k_=0), dict(v_=0), dict(k_=v.data_ptr()), dict(k_=k.data_ptr() + 8),
               dict(q_=qkv.data_ptr()), dict(q_=k.data_ptr()), dict(q_=o.data_ptr(), ldq=504),
               dict(q_=o.data_ptr() + 2), dict(x=k.data_ptr())):
        assert append(**kw) == ARG, kw
    assert append(page=9) == UNS

    x = bf16(rng, 3, 1000)
    y = torch.empty((3, 1000), device="cuda")
    some = i32([0, 0, 0, 0])

    def logits(x_=x.data_ptr(), ld=1000, S=3, o_=y.data_ptr(), ldo=1000, f=1, **rules):
        r = B.tp_logit_rules_t()
        r.n_reqs = 3
        for name, val in rules.items():
            setattr(r, name, val)
        return B.tp_process_logits(m.handle, x_, ld, S, r, o_, ldo, f, 0)

    p = some.data_ptr()
    assert logits() == 0 and logits(S=0) == 0
    for kw in (dict(x_=0), dict(o_=0), dict(ld=999), dict(ldo=999), dict(S=-1), dict(f=2), dict(n_reqs=2),
               dict(n_reqs=0), dict(x_=x.data_ptr() + 1), dict(o_=y.data_ptr() + 2),
               dict(o_=x.data_ptr()), dict(o_=x.data_ptr() + 2000, f=0), dict(history=p),
               dict(draft_tokens=p), dict(draft_tokens=p, tree_mask=p, q_start=p),
               dict(draft_tokens=p, tree_mask=p, q_start=p, tree_words=5), dict(bias_start=p, n_biases=1),
               dict(allowed=p, n_allowed=3, ld_allowed=31), dict(allowed=p, n_allowed=2, ld_allowed=32),
               dict(allowed=p, allowed_row=p, ld_allowed=32)):
        assert logits(**kw) == ARG, kw
    big = TPModel(make_config(512, 8, 2, 64, 256, 2**30 + 2, 0, 2, max_positions=8), [], max_tokens=1)
    r = B.tp_logit_rules_t()
    r.n_reqs = 1
    far = x.data_ptr() + 2**40  # (refused before anything looks at it)
    assert B.tp_process_logits(big.handle, x.data_ptr(), 2**30 + 2, 1, r, far, 2**30 + 2, 1, 0) == UNS
    assert m.check_device() == 0 and big.check_device() == 0


# ---------------------------------------------------------------------------
# streams, graphs, the run together
# ---------------------------------------------------------------------------
def test_tree_attention_output_in_the_cache_is_refused():
    """o in one buffer with the pages, from the first bytes of K to the last of V."""
    rng = np.random.default_rng(61)
    m = model(8, 2, 64, 2)
    c = attn_case(rng, m, [20], [3], 8, pad=0)
    ref = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    n, row = c["k"].numel(), 3 * 512
    buf = torch.zeros(2 * n + 2 * row, dtype=torch.bfloat16, device="cuda")
    k, v = buf[row:row + n].view_as(c["k"]), buf[row + n:row + 2 * n].view_as(c["v"])
    k.copy_(c["k"])
    v.copy_(c["v"])
    for at in (8, row, row + n - 8, row + n, row + 2 * n - row, row + 2 * n - 8):
        with pytest.raises(B.TPError, match="TP_ERR_ARG"):
            m.tree_attention(c["q"], c["step"], c["pages"], k, v, out=buf[at:at + row].view(3, 512))
    for at in (0, row + 2 * n):  # next to the cache
        out = buf[at:at + row].view(3, 512)
        m.tree_attention(c["q"], c["step"], c["pages"], k, v, out=out)
        assert torch.equal(out, ref)


def test_calls_on_another_stream():
    rng = np.random.default_rng(70)
    m = model(8, 2, 64, 2)
    c = attn_case(rng, m, [90, 5], [6, 11], 16)
    ref = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    x = bf16(rng, 2, 1000)
    want = m.process_logits(x, LogitRules(n_reqs=2))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ws = m.step_workspace(2, 64, stream=st)
    for s in (st, st.cuda_stream):
        got = m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"], ws=ws, stream=s)
        y = m.process_logits(x, LogitRules(n_reqs=2), stream=s)
        st.synchronize()
        assert torch.equal(got[:17], ref[:17]) and torch.equal(y, want)


def weights(rng, m):
    c = m
    H, d = c["hidden"], c["dim"]
    mk = lambda *s: bf16(rng, *s, scale=0.05)  # noqa: E731
    one = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    return dict(attn_norm=one, mlp_norm=one, wq=mk(c["heads"] * d, H), wk=mk(c["kv"] * d, H),
                wv=mk(c["kv"] * d, H), wo=mk(H, c["heads"] * d), wg=mk(256, H), wu=mk(256, H),
                wd=mk(H, 256))


def test_speculative_steps_match_one_token_at_a_time():
    """Two rounds of drafting, verifying and accepting through the paged calls, as captured
    graphs, against the same tokens in 64 bits: the attention block's output of every drafted
    token equals that of its path decoded token by token, the cache ends with the accepted
    tokens, and pages return to the ring."""
    rng = np.random.default_rng(80)
    shape = dict(hidden=512, heads=8, kv=2, dim=64)
    t, page, n_pages, vocab = 4, 8, 60, 1000
    cfg = make_config(512, 8, 2, 64, 256, vocab, 1, t, max_positions=512, plain_column_shards=1)
    w = weights(rng, shape)
    emb = bf16(rng, vocab, 512)
    m = TPModel(cfg, [w], emb, torch.ones(512, dtype=torch.bfloat16, device="cuda"),
                bf16(rng, vocab, 512, scale=0.05), max_tokens=64)
    n, T = 3, 10
    M = n * T + 2
    pages = PageTable.alloc(n, n_pages, page, 200)
    k, v = m.alloc_pages(n_pages, page), m.alloc_pages(n_pages, page)
    k.fill_(float("nan"))
    v.fill_(float("nan"))
    step = Step.alloc(n, M, T, 200, parents=torch.full((M,), -1, dtype=torch.int32, device="cuda"),
                      tree_words=1)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    rules = LogitRules(row_req=step.token_seq, n_reqs=n, presence=torch.full((n,), 2.0).cuda(),
                       draft_tokens=ids, tree_mask=step.tree_mask, q_start=step.q_start)
    buf = {}

    def verify():
        m.step_tables(pages, step)
        h = m.vocab_embed(ids)
        u = m.rmsnorm(h, w["attn_norm"])
        buf["qkv"] = m.column_linear(0, B.TP_QKV, u)
        q = m.cache_append(buf["qkv"], step.positions, step.slots, pages, k, v)
        o = torch.zeros_like(q)
        m.tree_attention(q, step, pages, k, v, out=o)
        buf["h"] = m.row_linear_reduce(0, B.TP_O, o, residual=h)
        buf["raw"] = m.lm_head_gather(buf["h"])
        buf["logits"] = m.process_logits(buf["raw"], rules)

    m.ensure_workspace(M)
    m.ensure_step_workspace(n, T)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # nothing runs yet: the ring is untouched
        verify()
    assert pages.free_state.tolist() == [0, n_pages]

    # 64-bit model of the attention block
    W = {a: f64(w[a]) for a in ("wq", "wk", "wv", "wo")}
    E = f64(emb)

    def block(tokens):
        """h after attention of the last token of a sequence, in 64 bits with the storage roundings
        left out."""
        x = E[np.asarray(tokens)]
        u = x / np.sqrt((x**2).mean(-1, keepdims=True) + cfg.rms_eps)
        L = len(tokens)
        q = R.rotate((u @ W["wq"].T).reshape(L, 8, 64), np.arange(L), cfg.rope_theta)[-1]
        kk = R.rotate((u @ W["wk"].T).reshape(L, 2, 64), np.arange(L), cfg.rope_theta)
        vv = (u @ W["wv"].T).reshape(L, 2, 64)
        o = np.concatenate([R.attention_row(q[h], kk[:, h // 4], vv[:, h // 4],
                                            np.ones(L, dtype=bool))[0] for h in range(8)])
        return x[-1] + W["wo"] @ o

    text = [[] for _ in range(n)]
    for rnd in range(3):
        sizes = [[T, T, 7], [T, 0, T], [1, 4, T]][rnd]
        trees = [list(range(-1, s - 1)) if rnd == 0 else R.random_tree(rng, s) for s in sizes]
        drafted = [rng.integers(0, vocab, s).tolist() for s in sizes]
        flat = sum(drafted, [])
        ids.copy_(i32(flat + [0] * (M - len(flat))))
        step.parents.copy_(i32(sum(trees, []) + [-1] * (M - len(flat))))
        old = [len(x) for x in text]
        step.old_lens.copy_(i32(old))
        step.new_lens.copy_(i32([a + b for a, b in zip(old, sizes)]))
        graph.replay()
        torch.cuda.synchronize()
        assert m.check_device() == 0
        h, raw, logits = f64(buf["h"]), f64(buf["raw"]), f64(buf["logits"])
        start = step.q_start.tolist()
        accepted = []
        for b in range(n):
            bits = R.tree_bits(trees[b])
            best = []
            for i in range(sizes[b]):
                path = np.nonzero(bits[i])[0].tolist()
                ref = block(text[b] + [drafted[b][p] for p in path])
                # bf16 storage of u, q, k, v, o and h: the layer tests' bound
                assert np.abs(h[start[b] + i] - ref).max() <= 2e-2 * np.abs(ref).max()
                for tok in {drafted[b][p] for p in path}:
                    assert logits[start[b] + i, tok] == np.float32(raw[start[b] + i, tok] - 2.0)
                if len(path) > len(best) and (not best or rng.random() < 0.6):
                    best = path
            accepted.append(best)
        # keep the accepted paths: their rows again, into the step's first slots
        slots = step.slots.tolist()
        final = [-1] * M
        for b in range(n):
            for j, p in enumerate(accepted[b]):
                final[start[b] + p] = slots[start[b] + j]
        m.cache_append(buf["qkv"], step.positions, i32(final), pages, k, v, want_q=False)
        for b in range(n):
            text[b] += [drafted[b][p] for p in accepted[b]]
        shrink = Step.alloc(n, 0, T, 200, step.new_lens.clone(), i32([len(x) for x in text]))
        m.step_tables(pages, shrink)
        used = sum(R.ceil_div(len(x), page) for x in text)
        assert pages.free_state.tolist()[1] == n_pages - used
        assert m.check_device() == 0
    assert min(len(x) for x in text) > 3


@pytest.mark.parametrize("t", [1, 4])
def test_a_whole_layer_over_pages_with_trained_norms(t):
    """The chain of calls of a paged layer (the unfolded shards, since its norm weights are not 1;
    SiLU(gate) * up by the caller), a prompt chunk and then single tokens, against the layer in
    64 bits; without the unfolded shards column_linear refuses."""
    rng = np.random.default_rng(82)
    shape, inter, page = dict(hidden=512, heads=8, kv=2, dim=64), 256, 8
    w = weights(rng, shape)
    w["attn_norm"], w["mlp_norm"] = (1 + bf16(rng, 512, scale=0.3) for _ in range(2))
    cfg = make_config(512, 8, 2, 64, inter, 100, 1, t, max_positions=512, plain_column_shards=1)
    m = TPModel(cfg, [w], max_tokens=64)
    folded = TPModel(make_config(512, 8, 2, 64, inter, 100, 1, t, max_positions=512), [w], max_tokens=64)
    with pytest.raises(B.TPError, match="TP_ERR_UNSUPPORTED"):
        folded.column_linear(0, B.TP_QKV, bf16(rng, 3, 512))
    n, prompt = 2, [37, 5]
    pages = PageTable.alloc(n, 40, page, 100)
    k, v = m.alloc_pages(40, page), m.alloc_pages(40, page)
    k.fill_(float("nan"))
    v.fill_(float("nan"))
    x = [bf16(rng, p + 2, 512) for p in prompt]

    W = {a: f64(w[a]) for a in w}

    def norm(h, g):
        return h / np.sqrt((h**2).mean(-1, keepdims=True) + cfg.rms_eps) * g

    def layer(h):  # one sequence in 64 bits
        L = len(h)
        u = norm(h, W["attn_norm"])
        q = R.rotate((u @ W["wq"].T).reshape(L, 8, 64), np.arange(L), cfg.rope_theta)
        kk = R.rotate((u @ W["wk"].T).reshape(L, 2, 64), np.arange(L), cfg.rope_theta)
        vv = (u @ W["wv"].T).reshape(L, 2, 64)
        o = np.stack([np.concatenate([R.attention_row(q[i, j], kk[:, j // 4], vv[:, j // 4], np.arange(L) <= i)[0]
                                      for j in range(8)]) for i in range(L)])
        h = h + o @ W["wo"].T
        u = norm(h, W["mlp_norm"])
        gate, up = u @ W["wg"].T, u @ W["wu"].T
        return h + (gate / (1 + np.exp(-gate)) * up) @ W["wd"].T

    ref = [layer(f64(y)) for y in x]
    lens = [0] * n
    for sizes in (prompt, [1, 1], [1, 1]):
        new = [a + b for a, b in zip(lens, sizes)]
        M = sum(sizes)
        step = Step.alloc(n, M, max(sizes), 100, i32(lens), i32(new))
        h = torch.cat([y[a:b] for y, a, b in zip(x, lens, new)])
        m.step_tables(pages, step)
        qkv = m.column_linear(0, B.TP_QKV, m.rmsnorm(h, w["attn_norm"]))
        q = m.cache_append(qkv, step.positions, step.slots, pages, k, v)
        o = m.tree_attention(q, step, pages, k, v)
        h = m.row_linear_reduce(0, B.TP_O, o, residual=h)
        gate, up = m.column_linear(0, B.TP_GATE_UP, m.rmsnorm(h, w["mlp_norm"])).float().chunk(2, dim=2)
        a = (torch.nn.functional.silu(gate) * up).bfloat16()  # [t, M, inter / t]
        got = f64(m.row_linear_reduce(0, B.TP_DOWN, a.transpose(0, 1).reshape(M, inter), residual=h))
        at = 0
        for b in range(n):
            want = ref[b][lens[b]:new[b]]
            # bf16 storage of every tensor on the way: the layer tests' bound
            assert np.abs(got[at:at + sizes[b]] - want).max() <= 2e-2 * np.abs(want).max()
            at += sizes[b]
        lens = new
    assert m.check_device() == 0


def test_threads_with_steps_of_different_sizes():
    """Four host threads, a stream and a workspace each, steps and rules of different sizes."""
    rng = np.random.default_rng(93)
    m = model(8, 2, 64, 2, 32003)
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                c, rules = cases[i]
                x = torch.zeros((300, 32003), dtype=torch.bfloat16, device="cuda")
                words = 0
                for _ in range(20):
                    pages = PageTable(c["page"], i32(c["table"]), i32(c["ring"]),
                                      i32([c["first"], c["count"]]))
                    step = Step.alloc(len(c["old"]), c["n_tokens"], c["max_new"], c["max_ctx"],
                                      i32(c["old"]), i32(c["new"]), i32(c["parents"]), words)
                    ws = m.step_workspace(len(c["old"]), c["max_new"])
                    m.step_tables(pages, step, ws=ws)
                    m.process_logits(x, rules, dtype=torch.bfloat16)
                    torch.cuda.current_stream().synchronize()
                    check_tables(c, words, pages, step)
        except Exception as e:  # noqa: BLE001 (handed to the test)
            failed.append((i, repr(e)))

    cases = []
    for i, n in enumerate((8000, 3600, 5000, 40)):
        c = tables_case(rng, n, 3, 16, 40, True, 0.2)
        hist = torch.zeros((300, 2100 + i), dtype=torch.int32, device="cuda")
        kw = dict(history=hist, history_lens=torch.zeros(300, dtype=torch.int32, device="cuda"))
        if i % 2:
            kw.update(bias_start=i32([0] * 301), bias_ids=i32([0]), bias_values=torch.ones(1).cuda())
        cases.append((c, LogitRules(**kw)))
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert m.check_device() == 0


def test_two_graphs_with_a_workspace_each():
    """Replayed at the same time on two streams."""
    rng = np.random.default_rng(90)
    m = model(8, 2, 128, 2)
    cases = [attn_case(rng, m, [2500, 300], [5, 40], 16) for _ in range(2)]
    refs = [m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"]).clone() for c in cases]
    graphs, outs, keep = [], [], []
    for c in cases:
        ws = m.step_workspace(2, 64)
        out = torch.zeros_like(c["q"])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"], out=out, ws=ws)
        graphs.append(g)
        outs.append(out)
        keep.append(ws)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, ref in zip(outs, refs):
        assert torch.equal(out[:45], ref[:45])
    assert m.check_device() == 0


def test_one_workspace_for_steps_of_different_sizes():
    """Pieces of a small step lie where no larger step keeps its tickets."""
    rng = np.random.default_rng(92)
    m = model(16, 8, 64, 2)
    ws = m.step_workspace(300, 80)
    small = attn_case(rng, m, [5001], [80], 64)
    large = attn_case(rng, m, rng.integers(100, 900, 300).tolist(), [1] * 300, 16)
    for c, pick in ((small, 13), (large, 3), (small, 13)):
        out = torch.full_like(c["q"], 3.0)
        m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"], out=out, ws=ws)
        check_attn(m, c, out, rows=lambda b, i: (b + i) % pick == 0)
    assert m.check_device() == 0


def test_workspace_does_not_grow_inside_a_capture():
    m = TPModel(make_config(512, 8, 2, 64, 256, 100, 0, 2, max_positions=64), [], max_tokens=1)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError, match="before the graph capture"):
            m.ensure_step_workspace(4, 4)
        torch.zeros(1, device="cuda")
    with pytest.raises(ValueError):
        m.step_workspace(8193, 4)
    first = m.ensure_step_workspace(4, 4)
    assert m.ensure_step_workspace(1, 1) is first
    larger = m.ensure_step_workspace(8000, 256)
    assert larger is not first and larger.numel() == B.tp_step_workspace_bytes(m.handle, 8000, 256)
    assert m.ensure_step_workspace(8000, 256) is larger and m.ensure_step_workspace(2, 7) is larger
    with pytest.raises(ValueError):
        m.ensure_step_workspace(0, 4)


def test_workspaces_held_while_a_batch_grows():
    """A batch that grows by one sequence a step, up to the most a step has: a handful of
    workspaces, and a capture after the first step needs no new one."""
    m = TPModel(make_config(512, 8, 2, 64, 256, 100, 0, 2, max_positions=64), [], max_tokens=1)
    for n in list(range(1, 600)) + [1000, 2000, 5000, 8192]:
        ws = m.ensure_step_workspace(n, 1 + n % 300)
        assert ws.numel() >= B.tp_step_workspace_bytes(m.handle, n, 1 + n % 300)
        if n == 599:
            assert not m._old_step_ws
    held = [m.step_ws] + m._old_step_ws
    most = B.tp_step_workspace_bytes(m.handle, 8192, 256)
    assert len(held) <= 4 and sum(w.numel() for w in held) <= 4 * most
    assert m.ensure_step_workspace(1, 9000) is m.step_ws is ws
    assert not any(w.any() for w in held)
    for bad in ((8193, 4), (0, 4), (-1, 4), (4, -1)):
        with pytest.raises(ValueError):
            m.ensure_step_workspace(*bad)


def test_counters_and_profile_names():
    rng = np.random.default_rng(91)
    m = model(8, 2, 64, 2)
    c = attn_case(rng, m, [9], [2], 8)
    before = m.stats().kernel_launches
    B.tp_profile(m.handle, True)
    m.tree_attention(c["q"], c["step"], c["pages"], c["k"], c["v"])
    m.process_logits(bf16(rng, 1, 1000), LogitRules(n_reqs=1))
    B.tp_profile(m.handle, False)
    t = B.tp_profile_read(m.handle, 0)
    assert set(t) == {"tree_attn", "process_logits"}
    assert m.stats().kernel_launches == before + 2
