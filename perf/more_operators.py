"""Cases of beam search and of shared cache pages: the selection over beams and
vocabulary, the beams' texts behind their parents, forks of page tables, the
copies of pages in every layer, and page tables made dense.

`own` false: plain torch forms.  `own` true: the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # selection: one request with four beams, a small vocabulary: latency
        dict(name="select_one", op="select", reqs=1, width=4, cands=8, vocab=32000, fp32=False, idle=0.0, masked=0.0),
        # selection: a served batch, the logits as the LM head leaves them
        dict(name="select_batch", op="select", reqs=64, width=4, cands=8, vocab=128256, fp32=False, idle=0.0, masked=0.0),
        # selection: wide beams behind the rules on logits (fp32, grammars that leave few tokens), some beams not in use
        dict(name="select_wide", op="select", reqs=13, width=16, cands=32, vocab=152064, fp32=True, idle=0.1, masked=0.3),
        # selection: an odd vocabulary, whose rows begin off 16-byte boundaries
        dict(name="select_odd", op="select", reqs=31, width=7, cands=21, vocab=32003, fp32=False, idle=0.2, masked=0.1),
        # texts: one request's beams: latency
        dict(name="advance_one", op="advance", reqs=1, width=4, room=512, max_len=300, idle=0.0),
        # texts: a full batch with long texts
        dict(name="advance_batch", op="advance", reqs=64, width=8, room=8192, max_len=8000, idle=0.05),
        # forks: two requests' beams a step: latency
        dict(name="fork_small", op="fork", reqs=2, width=4, page=16, max_len=1000, spare=300, done=0.0, cut=0.0),
        # forks: a full batch at long contexts; some requests end, some go back to an earlier token
        dict(name="fork_batch", op="fork", reqs=128, width=8, page=16, max_len=8000, spare=20000, done=0.05, cut=0.1),
        # copies: a step's partly filled pages of one request, few layers
        dict(name="copy_small", op="copy", moves=3, pages=40, page=16, layers=4, kv=8, dim=128, ranks=8, whole=False),
        # copies: the partly filled pages of a full batch, every layer of a 32-layer model
        dict(name="copy_forks", op="copy", moves=150, pages=320, page=16, layers=32, kv=8, dim=128, ranks=4, whole=False),
        # compaction: a small pool with holes, and its whole pages moved
        dict(name="compact_small", op="compact", reqs=5, width=1, page=16, max_len=700, used=0.5, tail=0.0),
        # compaction: a large pool after hours of service, prefixes shared by four rows each
        dict(name="compact_pool", op="compact", reqs=200, width=4, page=16, max_len=8000, used=0.6, tail=0.2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select", "advance", "fork", "copy", "compact"])
    if op == "select":
        width, vocab, fp32 = _log(rng, 1, 32), _log(rng, 40, 152064), rng.random() < 0.4
        reqs = _log(rng, 1, max(1, min(256, 16000000 // (vocab * width))))
        return dict(op="select", reqs=reqs, width=width, cands=min(64, rng.randint(width, 3 * width)), vocab=vocab, fp32=fp32,
                    idle=rng.choice([0.0, 0.3]), masked=rng.choice([0.0, 0.5]))
    if op == "advance":
        width, room = _log(rng, 1, 32), _log(rng, 2, 8192)
        return dict(op="advance", reqs=_log(rng, 1, max(1, min(256, 3000000 // (width * room)))), width=width, room=room,
                    max_len=rng.randint(1, room - 1), idle=rng.choice([0.0, 0.2]))
    if op == "fork":
        width, page, length = _log(rng, 1, 16), 8 * _log(rng, 1, 16), _log(rng, 5, 8000)
        return dict(op="fork", reqs=_log(rng, 1, max(2, min(256, 1000 // width))), width=width, page=page, max_len=length,
                    spare=_log(rng, 10, 20000), done=rng.choice([0.0, 0.2]), cut=rng.choice([0.0, 0.2]))
    if op == "copy":
        kv, dim, ranks = rng.choice([(8, 128, 8), (8, 128, 1), (4, 128, 2), (2, 64, 4), (1, 64, 1), (32, 128, 4)])
        page, layers = 8 * _log(rng, 1, 16), _log(rng, 1, 64)
        room = max(2, int(3e8 // (layers * page * kv * dim * 4)))
        pages = max(2, _log(rng, 2, max(3, min(2000, room))))
        return dict(op="copy", moves=rng.randint(1, max(1, pages // 2)), pages=pages, page=page, layers=layers, kv=kv, dim=dim,
                    ranks=ranks, whole=rng.random() < 0.5)
    width, page, length = _log(rng, 1, 8), 8 * _log(rng, 1, 16), _log(rng, 5, 8000)
    return dict(op="compact", reqs=_log(rng, 1, max(1, min(800, 200000 * page // length) // width)), width=width, page=page,
                max_len=length, used=rng.choice([0.2, 0.5, 0.9]), tail=rng.choice([0.0, 0.3]))


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32).to(DEV)


def _ints(g, lo, hi, n):
    """n whole numbers in [lo, hi], on the host."""
    return torch.randint(lo, hi + 1, (n,), generator=g)


_models = {}


def _model(kv=1, dim=64, ranks=1, vocab=64):
    """The framework's model handle: its shape and status word; these operators read no weights."""
    from megatron_tensor_layers_tp_gb300.runtime import TPModel, make_config

    key = (kv, dim, ranks, vocab)
    if key not in _models:
        heads = max(kv, ranks)
        cfg = make_config(heads * dim, heads, kv, dim, 64 * ranks, vocab, 0, ranks, max_positions=64)
        _models[key] = TPModel(cfg, [], max_tokens=1)
    return _models[key]


def _parents(g, R, W):
    """Parents of R x W beams, as rows: the better a beam, the more often it is continued."""
    w = (W * torch.rand((R, W), generator=g) ** 2).long().clamp(max=W - 1)
    return w + torch.arange(R)[:, None] * W


def _select_state(case, g, gg):
    R, W, K, V = case["reqs"], case["width"], case["cands"], case["vocab"]
    # a request's beams agree on most of what may follow
    x = 2.5 * torch.randn((R, 1, V), generator=gg, device=DEV) + 1.5 * torch.randn((R, W, V), generator=gg, device=DEV)
    ends = torch.randperm(V, generator=g)[: min(2, V - 1)]
    x[:, :, ends.to(DEV)] += 9.0
    x = x.view(R * W, V)
    if case["masked"]:  # grammars that allow one token in a hundred
        rows = (torch.rand(R * W, generator=g) < case["masked"]).to(DEV)
        x.masked_fill_(rows[:, None] & (torch.rand((R * W, V), generator=gg, device=DEV) < 0.99), -math.inf)
    scores = -torch.rand(R * W, generator=g) * 12
    scores[torch.rand(R * W, generator=g) < case["idle"]] = -math.inf
    s = dict(logits=x if case["fp32"] else x.bfloat16(), scores=scores.float().to(DEV), ends=_i32(ends))
    if own:
        from megatron_tensor_layers_tp_gb300.runtime import Beams

        s["model"] = _model(vocab=V)
        s["beams"] = Beams.alloc(R, W, K, ends=s["ends"], scores=s["scores"])
    return s


def _advance_state(case, g, gg):
    R, W, ld = case["reqs"], case["width"], case["room"]
    n = R * W
    lens = _ints(g, max(1, case["max_len"] // 2), case["max_len"], R).repeat_interleave(W)
    parents = _parents(g, R, W).flatten()
    parents[torch.rand(n, generator=g) < case["idle"]] = -1
    return dict(parents=_i32(parents), tokens=_i32(_ints(g, 0, 128255, n)), lens=_i32(lens),
                history=torch.randint(0, 128256, (n, ld), generator=gg, device=DEV, dtype=torch.int32),
                out=torch.zeros((n, ld), dtype=torch.int32, device=DEV), lens_out=torch.zeros(n, dtype=torch.int32, device=DEV),
                **(dict(model=_model()) if own else {}))


def _shared_tables(case, g, spare, idle):
    """Page tables of requests whose beams share their prefix's pages: (lens, table, page numbers not in use, pages in all)."""
    R, W, P, L = case["reqs"], case["width"], case["page"], case["max_len"]
    f = torch.Generator().manual_seed(R + 7 * W + L)  # sizes go by the case
    length = _ints(f, max(1, L // 3), L, R)
    common = (length.float() * (0.3 + 0.7 * torch.rand(R, generator=f))).long() // P  # full pages that all beams hold
    lens = length[:, None].repeat(1, W)
    lens[torch.rand((R, W), generator=f) < idle] = 0
    at = torch.randperm(R, generator=g)  # the requests in another order
    lens, common = lens[at], common[at]
    have, ld = (lens + P - 1) // P, (L + P - 1) // P + 1
    col = torch.arange(ld)[None, None, :]
    shared = (col < common[:, None, None]) & (col < have[:, :, None])
    apart = (col >= common[:, None, None]) & (col < have[:, :, None])
    prefix = shared.any(1)
    n_prefix, n_apart = int(prefix.sum()), int(apart.sum())
    n_pages = n_prefix + n_apart + spare(n_prefix + n_apart)
    perm = torch.randperm(n_pages, generator=g).int()
    pre = torch.zeros((R, ld), dtype=torch.int32)
    pre[prefix] = perm[:n_prefix]
    table = torch.where(shared, pre[:, None, :], torch.zeros((), dtype=torch.int32))
    table[apart] = perm[n_prefix:n_prefix + n_apart]
    return lens.flatten(), table.view(R * W, ld), perm[n_prefix + n_apart:], n_pages


def _ring(g, free, n_pages):
    first = int(_ints(g, 0, n_pages - 1, 1))
    ring = torch.zeros(n_pages, dtype=torch.int32)
    ring[(first + torch.arange(len(free))) % n_pages] = free
    return _i32(ring), _i32([first, len(free)])


def _fork_state(case, g, gg):
    R, W, P = case["reqs"], case["width"], case["page"]
    n = R * W
    lens, table, free, n_pages = _shared_tables(case, g, lambda used: n + case["spare"], 0.02)
    ring, state = _ring(g, free, n_pages)
    src = _parents(g, R, W)
    src[torch.rand(R, generator=g) < case["done"]] = -1
    src = src.flatten()
    keep = torch.where(src >= 0, lens[src.clamp(min=0)], 0)
    back = (torch.rand(R, generator=g) < case["cut"]).repeat_interleave(W)
    keep = torch.where(back, (keep.float() * torch.rand(n, generator=g)).long(), keep)
    s = dict(P=P, n_pages=n_pages, table=_i32(table), ring=ring, free=state, lens=_i32(lens), src=_i32(src), keep=_i32(keep),
             table_out=torch.zeros_like(_i32(table)), max_ctx=case["max_len"])
    if own:
        from megatron_tensor_layers_tp_gb300.runtime import PageFork, PageTable

        s["model"] = _model()
        s["pages"] = PageTable(P, s["table"], s["ring"], s["free"], free_next=torch.empty_like(s["free"]),
                               holders=torch.zeros(n_pages, dtype=torch.int32, device=DEV))
        s["fork"] = PageFork.alloc(s["pages"], s["max_ctx"], s["lens"], s["src"], s["keep"], table=s["table_out"])
    else:
        s["moves"] = torch.zeros((n, 3), dtype=torch.int32, device=DEV)
    return s


def _copies(case):
    """(cache copies, KV heads a copy) of the case's ranks."""
    kv, t = case["kv"], case["ranks"]
    return (t, kv // t) if kv >= t else (kv, 1)


def _copy_state(case, g, gg):
    copies, kvr = _copies(case)
    M, P = case["moves"], case["page"]
    pages = torch.randperm(case["pages"], generator=g)[: 2 * M]
    tokens = torch.full((M,), P) if case["whole"] else _ints(g, 1, P - 1, M)
    pools = torch.randn((2, case["layers"], copies, case["pages"], kvr, P, case["dim"]), generator=gg, device=DEV, dtype=torch.bfloat16)
    # the list has room for more moves than a step makes
    moves = torch.full((M + 5, 3), -1)
    moves[:M] = torch.stack([pages[:M], pages[M:], tokens], 1)
    s = dict(pools=pools, moves=_i32(moves), count=_i32([M]))
    if own:
        from megatron_tensor_layers_tp_gb300.runtime import LayerPages, PageMoves, PageTable

        s["model"] = _model(case["kv"], case["dim"], case["ranks"])
        s["layers"] = LayerPages(list(pools[0]), list(pools[1]))
        s["pages"], s["list"] = PageTable(P, n_pages=case["pages"]), PageMoves(s["moves"], s["count"])
    return s


def _compact_state(case, g, gg):
    lens, table, free, n_pages = _shared_tables(case, g, lambda used: int(used / case["used"]) - used + 1, case["tail"])
    ring, state = _ring(g, free, n_pages)
    s = dict(P=case["page"], n_pages=n_pages, table=_i32(table), ring=ring, free=state, lens=_i32(lens), max_ctx=case["max_len"],
             table_out=torch.zeros_like(_i32(table)))
    if own:
        from megatron_tensor_layers_tp_gb300.runtime import PageMoves, PageTable

        s["model"] = _model()
        s["pages"] = PageTable(s["P"], s["table"], s["ring"], s["free"])
        s["to"] = PageTable(s["P"], s["table_out"], torch.empty_like(s["ring"]), torch.empty_like(s["free"]),
                            holders=torch.zeros(n_pages, dtype=torch.int32, device=DEV))
        s["list"] = PageMoves.alloc(n_pages // 2 + 1)
    else:
        s["moves"] = torch.zeros((n_pages // 2 + 1, 3), dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(select=_select_state, advance=_advance_state, fork=_fork_state, copy=_copy_state,
             compact=_compact_state)[case["op"]](case, g, gg)
    s["op"], s["case"] = case["op"], case
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_select(s):
    c = s["case"]
    R, W, K, V = c["reqs"], c["width"], c["cands"], c["vocab"]
    x = s["logits"].double()  # scores of different beams may lie close together
    top = x.amax(1, keepdim=True)
    d = x - torch.where(top == -math.inf, 0.0, top)
    y = d - d.exp().sum(1, keepdim=True).log() + s["scores"].double()[:, None]
    y = torch.where((x > -math.inf) & (s["scores"] > -math.inf)[:, None], y, -math.inf)
    best, at = y.view(R, W * V).sort(dim=1, descending=True, stable=True)  # equal scores: the lowest index first
    best, at = best[:, :K], at[:, :K]
    if best.shape[1] < K:  # fewer tokens than candidates
        best = torch.cat([best, best.new_full((R, K - best.shape[1]), -math.inf)], 1)
        at = torch.cat([at, at.new_zeros((R, K - at.shape[1]))], 1)
    there = best > -math.inf
    rows = torch.where(there, at // V + torch.arange(R, device=DEV)[:, None] * W, -1)
    tokens = torch.where(there, at % V, -1)
    goes = there & (tokens[:, :, None] != s["ends"].long()[None, None, :]).all(2)
    place = torch.where(goes, goes.long().cumsum(1) - 1, W).clamp(max=W)
    n_scores = best.new_full((R, W + 1), -math.inf).scatter(1, place, best)[:, :W]
    n_rows = rows.new_full((R, W + 1), -1).scatter(1, place, rows)[:, :W]
    n_tokens = tokens.new_zeros((R, W + 1)).scatter(1, place, tokens)[:, :W]
    return dict(cand_scores=best.float(), cand_rows=rows.int(), cand_tokens=tokens.int(), scores=n_scores.float().flatten(),
                parents=n_rows.int().flatten(), tokens=n_tokens.int().flatten())


def _own_select(s):
    b = s["model"].beam_select(s["logits"], s["beams"])
    return dict(cand_scores=b.cand_scores, cand_rows=b.cand_rows, cand_tokens=b.cand_tokens, scores=b.next_scores,
                parents=b.parents, tokens=b.tokens)


def _plain_advance(s):
    p = s["parents"].long()
    n = torch.where(p >= 0, s["lens"][p.clamp(min=0)], 0)
    at = torch.arange(s["history"].shape[1], device=DEV)[None, :]
    end = (p >= 0)[:, None] & (at == n[:, None])
    text = torch.where(end, s["tokens"][:, None], s["history"][p.clamp(min=0)])
    s["out"].copy_(torch.where((at < n[:, None]) | end, text, s["out"]))
    s["lens_out"].copy_(torch.where(p >= 0, n + 1, 0))
    return dict(history=s["out"], lens=s["lens_out"])


def _own_advance(s):
    out, lens = s["model"].beam_advance(s["parents"], s["tokens"], s["history"], s["lens"], out=s["out"], lens_out=s["lens_out"])
    return dict(history=out, lens=lens)


def _plain_fork(s):
    P, N, table = s["P"], s["n_pages"], s["table"].long()
    n, ld = table.shape
    lens, src, keep = s["lens"].long(), s["src"].long(), s["keep"].long()
    keep = torch.where(src >= 0, keep, 0)
    col, row = torch.arange(ld, device=DEV)[None, :], torch.arange(n, device=DEV)
    old = col < ((lens + P - 1) // P)[:, None]
    new = table[src.clamp(min=0)]
    whole, last = col < (keep // P)[:, None], (col == (keep // P)[:, None]) & (keep % P > 0)[:, None]
    full = torch.zeros(N, dtype=torch.long, device=DEV).index_add(0, new[whole], torch.ones_like(new[whole]))
    held = torch.zeros(N, dtype=torch.bool, device=DEV)
    held[table[old]] = True
    open_ = torch.where(keep % P > 0, new.gather(1, (keep // P)[:, None])[:, 0], N)  # the page that the row writes to next
    lowest = torch.full((N + 1,), n, device=DEV).scatter_reduce(0, open_, row, "amin")
    copies = (open_ < N) & ((full[open_.clamp(max=N - 1)] > 0) | (lowest[open_] < row))
    first, count = s["free"][0].long(), s["free"][1].long()
    number = copies.long().cumsum(0) - 1
    fresh = s["ring"].long()[(first + number.clamp(min=0)) % N]
    to = torch.where(copies, fresh, open_)
    s["table_out"].copy_(torch.where(whole, new, torch.where(last, to[:, None], s["table_out"].long())))
    holders = full.clone()
    holders[to[open_ < N]] = 1
    gone = held & (full == 0) & (lowest[:N] == n)
    free = gone.nonzero()[:, 0]
    s["ring"][(first + count + torch.arange(free.numel(), device=DEV)) % N] = free.int()
    taken = copies.sum()
    s["moves"][number[copies]] = torch.stack([open_, to, keep % P], 1)[copies].int()
    return dict(table=s["table_out"], lens=keep.int(), ring=s["ring"], holders=holders.int(), moves=s["moves"],
                count=taken.int().view(1), free=torch.stack([(first + taken) % N, count - taken + free.numel()]).int())


def _own_fork(s):
    f, p = s["model"].fork_pages(s["pages"], s["fork"]), s["pages"]
    return dict(table=f.table, lens=f.new_lens, ring=p.free_ring, holders=p.holders, moves=f.moves.table, count=f.moves.count,
                free=p.free_next)


def _plain_copy(s):
    x, m = s["pools"], s["moves"][: s["case"]["moves"]].long()
    P = x.shape[5]
    there = torch.arange(P, device=DEV)[None, :] < m[:, 2:3]
    which, off = there.nonzero(as_tuple=True)
    x[:, :, :, m[which, 1], :, off] = x[:, :, :, m[which, 0], :, off]
    return x


def _own_copy(s):
    s["model"].copy_pages(s["list"], s["pages"], s["layers"])
    return s["pools"]


def _plain_compact(s):
    P, N, table = s["P"], s["n_pages"], s["table"].long()
    there = torch.arange(table.shape[1], device=DEV)[None, :] < ((s["lens"].long() + P - 1) // P)[:, None]
    holders = torch.zeros(N, dtype=torch.long, device=DEV).index_add(0, table[there], torch.ones_like(table[there]))
    held = holders > 0
    used, page = held.sum(), torch.arange(N, device=DEV)
    movers, holes = (held & (page >= used)).nonzero()[:, 0].flip(0), (~held & (page < used)).nonzero()[:, 0]
    name = page.clone()
    name[movers] = holes
    s["table_out"].copy_(torch.where(there, name[table], s["table_out"].long()))
    after = torch.zeros_like(holders)
    after[name[held]] = holders[held]
    s["moves"][: movers.numel()] = torch.stack([movers, holes, torch.full_like(movers, P)], 1).int()
    return dict(table=s["table_out"], ring=page.int(), free=torch.stack([used % N, N - used]).int(), holders=after.int(),
                moves=s["moves"], count=torch.tensor([movers.numel()], dtype=torch.int32, device=DEV))


def _own_compact(s):
    to = s["to"]
    s["model"].compact_pages(s["pages"], s["lens"], s["max_ctx"], s["list"], out=to)
    return dict(table=to.table, ring=to.free_ring, free=to.free_next, holders=to.holders, moves=s["list"].table, count=s["list"].count)


_plain = dict(select=_plain_select, advance=_plain_advance, fork=_plain_fork, copy=_plain_copy, compact=_plain_compact)
_own = dict(select=_own_select, advance=_own_advance, fork=_own_fork, copy=_own_copy, compact=_own_compact)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "select":
        R, W, K, V = case["reqs"], case["width"], case["cands"], case["vocab"]
        rows = R * W * (1.0 - case["idle"])
        # a logit is read once; its difference, exponential and sum
        return {"bytes": int(rows * V * (4 if case["fp32"] else 2) + R * (12 * K + 16 * W)), "flops": int(3 * rows * V)}
    if op == "advance":
        n = case["reqs"] * case["width"]
        return {"bytes": int(n * (16 + 8 * (1.0 - case["idle"]) * 0.75 * case["max_len"])), "flops": 0}
    if op == "copy":
        tokens = case["moves"] * (case["page"] if case["whole"] else case["page"] / 2)
        return {"bytes": int(2 * 2 * case["layers"] * tokens * case["kv"] * case["dim"] * 2 + 12 * case["moves"]), "flops": 0}
    n, P = case["reqs"] * case["width"], case["page"]
    entries = n * (2 * case["max_len"] / 3 + P / 2) / P  # of the tables
    pages = entries * (0.35 + 0.65 / case["width"])  # two thirds of a row's are its request's
    if op == "fork":
        return {"bytes": int(8 * entries + 4 * (pages + n + case["spare"]) + 28 * n), "flops": 0}
    return {"bytes": int(8 * entries * (1.0 - case["tail"]) + 8 * pages / case["used"] + 4 * n), "flops": 0}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def _exact_select(s):
    c = s["case"]
    R, W, K, V = c["reqs"], c["width"], c["cands"], c["vocab"]
    ends = set(s["ends"].tolist())
    out = dict(cand_scores=[], cand_rows=[], cand_tokens=[], scores=[], parents=[], tokens=[])
    for r in range(R):
        pool = []
        for b in range(r * W, (r + 1) * W):
            score = float(s["scores"][b])
            if score == -math.inf:
                continue
            p = torch.log_softmax(s["logits"][b].double(), 0)
            # the tokens that at most K - 1 others of the row are better than
            edge = p.topk(min(K, V)).values[-1]
            at = (p >= edge).nonzero()[:, 0].tolist() if float(edge) > -math.inf else (p > -math.inf).nonzero()[:, 0].tolist()
            pool += [(-(score + q), b, v) for v, q in zip(at, p[at].tolist())]
        pool = sorted(pool)[:K]
        alive = [x for x in pool if x[2] not in ends][:W]
        pool += [(math.inf, -1, -1)] * (K - len(pool))
        alive += [(math.inf, -1, 0)] * (W - len(alive))
        out["cand_scores"].append([-x[0] for x in pool])
        out["cand_rows"].append([x[1] for x in pool])
        out["cand_tokens"].append([x[2] for x in pool])
        out["scores"] += [-x[0] for x in alive]
        out["parents"] += [x[1] for x in alive]
        out["tokens"] += [x[2] for x in alive]
    return {k: torch.tensor(v, dtype=torch.float64 if "scores" in k else torch.int32) for k, v in out.items()}


def exact(case, seed):
    """The selection's scores; whole numbers have nothing to be off by."""
    if case["op"] != "select" and case["op"] != "copy":
        return None
    s = prepare(case, seed)
    if case["op"] == "select":
        return _exact_select(s)
    x = s["pools"].double()
    for a, b, n in s["moves"].tolist()[: case["moves"]]:
        x[:, :, :, b, :, :n] = x[:, :, :, a, :, :n]
    return x
