"""Cases of the paged-cache serving operators: the step tables, the rotary
embedding with the store into cache pages, attention for trees of drafted
tokens over the pages, and the rules on logits.

`own` false: plain torch forms.  `own` true: the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
THETA = 10000.0


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # tables: a small serving batch verifying 8-token trees every step
        dict(name="tables_small", op="tables", seqs=8, max_new=8, page=16, max_len=1000, tree=True, shrink=0.0),
        # tables: a full batch in the middle of service; a tenth of the requests hand pages back
        dict(name="tables_mixed", op="tables", seqs=512, max_new=64, page=16, max_len=4000, tree=True, shrink=0.1),
        # tables: prompts admitted together, one slot for each of ~64k prompt tokens
        dict(name="tables_prompts", op="tables", seqs=61, max_new=2048, page=32, max_len=2300, tree=False, shrink=0.0),
        # append: one decode step's rows, where latency counts
        dict(name="append_decode", op="append", tokens=8, heads=32, kv=8, dim=128, ranks=8, page=16, holes=0.0),
        # append: a prompt chunk, replicated KV heads (two ranks share one), padded rows among it
        dict(name="append_prompt", op="append", tokens=8191, heads=40, kv=4, dim=128, ranks=8, page=64, holes=0.05),
        # attention: one request, one token, a short context: latency
        dict(name="attn_single", op="attn", seqs=1, min_new=1, max_new=1, min_ctx=700, max_ctx=700, heads=32, kv=8,
             dim=128, ranks=8, page=16, tree=True),
        # attention: a ragged batch of drafted trees, five query heads to a KV head
        dict(name="attn_trees", op="attn", seqs=16, min_new=8, max_new=32, min_ctx=150, max_ctx=2048, heads=40, kv=8,
             dim=128, ranks=8, page=16, tree=True),
        # attention: a full batch at long contexts, small trees: the cache's bytes count
        dict(name="attn_long", op="attn", seqs=64, min_new=2, max_new=8, min_ctx=1500, max_ctx=4096, heads=32, kv=8,
             dim=128, ranks=4, page=64, tree=True),
        # attention: prompt chunks (causal chains) of heads of 64, pages that end inside key tiles
        dict(name="attn_chunks", op="attn", seqs=6, min_new=100, max_new=256, min_ctx=0, max_ctx=8000, heads=32, kv=4,
             dim=64, ranks=2, page=24, tree=False),
        # logits: one request's next token with every rule on
        dict(name="logits_one", op="logits", reqs=1, nodes=1, vocab=128256, history=300, biases=40, grammar=True,
             fp32=True),
        # logits: a batch with long histories, penalties only
        dict(name="logits_batch", op="logits", reqs=64, nodes=1, vocab=128256, history=4096, biases=0, grammar=False,
             fp32=True),
        # logits: every drafted token of sixteen trees, each with its own path and grammar state
        dict(name="logits_trees", op="logits", reqs=16, nodes=16, vocab=152064, history=1500, biases=300, grammar=True,
             fp32=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(32, 8, 128, 1), (32, 8, 128, 8), (40, 8, 128, 8), (40, 4, 128, 8), (28, 4, 128, 2), (16, 2, 64, 2),
          (8, 8, 64, 4), (16, 1, 64, 1), (32, 32, 128, 4)]


def draw(rng):
    op = rng.choice(["tables", "append", "attn", "attn", "logits"])
    if op == "tables":
        tree = rng.random() < 0.6
        seqs = _log(rng, 1, 512)
        top = min(256, 32768 // seqs) if tree else min(2048, 120000 // seqs)
        return dict(op="tables", seqs=seqs, max_new=_log(rng, 1, top), page=8 * _log(rng, 1, 32),
                    max_len=_log(rng, 20, 4000), tree=tree, shrink=rng.choice([0.0, 0.1, 0.5]))
    if op == "append":
        h, k, d, r = rng.choice(_HEADS)
        return dict(op="append", tokens=_log(rng, 1, 8191), heads=h, kv=k, dim=d, ranks=r, page=8 * _log(rng, 1, 32),
                    holes=rng.choice([0.0, 0.05, 0.5]))
    if op == "attn":
        h, k, d, r = rng.choice(_HEADS)
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, min(256, 512 // seqs)))
        ctx = _log(rng, 16, min(32000, int(6.5e8 / (seqs * k * d * 4)), int(3e10 / (seqs * new * h * d * 4))))
        return dict(op="attn", seqs=seqs, min_new=rng.randint(1, new), max_new=new, min_ctx=rng.randint(0, ctx),
                    max_ctx=ctx, heads=h, kv=k, dim=d, ranks=r, page=8 * _log(rng, 1, 32), tree=rng.random() < 0.7)
    reqs, vocab = _log(rng, 1, 64), _log(rng, 1000, 152064)
    nodes = _log(rng, 1, max(1, min(64, 160 // reqs)))
    return dict(op="logits", reqs=reqs, nodes=nodes, vocab=vocab, history=_log(rng, 1, 8000),
                biases=rng.choice([0, 7, 300]), grammar=rng.random() < 0.5, fp32=rng.random() < 0.6)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32).to(DEV)


def _ints(g, lo, hi, n):
    """n whole numbers in [lo, hi], on the host."""
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _shuffled(g, *columns):
    """The same requests in another order: sizes in all stay those of the case."""
    at = torch.randperm(columns[0].numel(), generator=g)
    return [c[at] for c in columns]


def _parents(g, sizes):
    """Parents of random trees, token after token: -1 for a child of the context."""
    out = []
    for t in sizes:
        r = torch.rand(t, generator=g).tolist()
        # half of the tokens continue the one before, as a chain does
        out += [-1 if i == 0 else (i - 1 if r[i] < 0.5 else int(r[i] * 2 * (i + 1) - (i + 1)) - 1) for i in range(t)]
    return torch.tensor(out, dtype=torch.int32)


def _ancestors(parents, sizes, words):
    """Bit masks of each token's path (itself included), and its depth, on the host."""
    rows, depth, at = [], [], 0
    for t in sizes:
        first = len(rows)
        for i in range(t):
            p = int(parents[at + i])
            rows.append((rows[first + p] if p >= 0 else 0) | (1 << i))
            depth.append(depth[first + p] + 1 if p >= 0 else 0)
        at += t
    mask = torch.tensor([[((r >> (64 * w)) & (2**64 - 1)) for w in range(words)] for r in rows], dtype=torch.uint64)
    return mask.view(torch.int64).reshape(-1, words), torch.tensor(depth, dtype=torch.int32)


def _heads(case):
    """(attention ranks, q heads a rank, KV heads a rank, replicas, copies)."""
    t, n = case["ranks"], case["kv"]
    kvr, rep = (n // t, 1) if n >= t else (1, t // n)
    return t, case["heads"] // t, kvr, rep, min(t, n)


_models = {}


def _model(heads=8, kv=8, dim=64, ranks=1, vocab=64):
    """The framework's model handle: its shape, rotary table and status word; these operators read no weights."""
    from megatron_tensor_layers_tp_gb300.runtime import TPModel, make_config

    key = (heads, kv, dim, ranks, vocab)
    if key not in _models:
        cfg = make_config(heads * dim, heads, kv, dim, 64 * ranks, vocab, 0, ranks, rope_theta=THETA,
                          max_positions=40000)
        _models[key] = TPModel(cfg, [], max_tokens=1)
    return _models[key]


def _tables_state(case, g):
    B, T, P = case["seqs"], case["max_new"], case["page"]
    f = torch.Generator().manual_seed(B + T + P)
    old = _ints(f, 0, case["max_len"], B)
    new = old + _ints(f, 1, T, B)
    if not case["tree"]:  # prompts are admitted into empty rows
        old, new = torch.zeros_like(old), _ints(f, max(1, T // 2), T, B)
    gone = torch.rand(B, generator=f) < case["shrink"]
    new = torch.where(gone, (old.float() * torch.rand(B, generator=f)).long(), new)
    old, new = _shuffled(g, old, new)
    have, ld = (old + P - 1) // P, (case["max_len"] + T + P - 1) // P
    used = int(have.sum())
    spare = int(((new + P - 1) // P - have).clamp(min=0).sum())
    n_pages = used + spare + 7
    perm = torch.randperm(n_pages, generator=g).int()
    table = torch.full((B, ld), -1, dtype=torch.int32)
    table[torch.arange(ld)[None, :] < have[:, None]] = perm[:used]
    first = int(_ints(g, 0, n_pages - 1, 1))
    ring = torch.zeros(n_pages, dtype=torch.int32)
    ring[(first + torch.arange(n_pages - used)) % n_pages] = perm[used:]
    sizes = (new - old).clamp(min=0)
    M = int(sizes.sum()) + 5  # a few padded rows behind the last sequence
    parents = None
    if case["tree"]:
        parents = torch.cat([_parents(g, sizes.tolist()), torch.full((5,), -1, dtype=torch.int32)])
    words = (T + 63) // 64 if case["tree"] else 0
    s = dict(P=P, T=T, M=M, n_pages=n_pages, words=words, max_ctx=int(torch.maximum(old, new).max()), old=_i32(old),
             new=_i32(new), table=_i32(table), ring=_i32(ring), free=_i32([first, n_pages - used]),
             parents=None if parents is None else _i32(parents))
    if own:
        from megatron_tensor_layers_tp_gb300.runtime import PageTable, Step

        s["model"] = _model()
        s["pages"] = PageTable(P, s["table"], s["ring"], s["free"], free_next=torch.empty_like(s["free"]))
        s["step"] = Step.alloc(B, M, T, s["max_ctx"], s["old"], s["new"], parents=s["parents"], tree_words=words)
    return s


def _pool(case, n_pages, gg):
    _, _, kvr, _, copies = _heads(case)
    return torch.randn((copies, n_pages, kvr, case["page"], case["dim"]), generator=gg, device=DEV).bfloat16()


def _append_state(case, g, gg):
    t, nq, kvr, _, _ = _heads(case)
    M, P = case["tokens"], case["page"]
    n_pages = (M + P - 1) // P + 3
    qkv = torch.randn((t, M, (nq + 2 * kvr) * case["dim"]), generator=gg, device=DEV).bfloat16()
    slots = torch.randperm(n_pages * P, generator=g)[:M]
    slots[torch.rand(M, generator=g) < case["holes"]] = -1
    s = dict(qkv=qkv, pos=_i32(_ints(g, 0, 39999, M)), slots=_i32(slots), k=_pool(case, n_pages, gg),
             v=_pool(case, n_pages, gg))
    if own:
        from megatron_tensor_layers_tp_gb300.runtime import PageTable

        s["model"] = _model(case["heads"], case["kv"], case["dim"], t)
        s["pages"] = PageTable(P, n_pages=n_pages)
    return s


def _attn_state(case, g, gg):
    B, P = case["seqs"], case["page"]
    f = torch.Generator().manual_seed(B + case["max_ctx"])
    ctx = _ints(f, case["min_ctx"], case["max_ctx"], B)
    T = _ints(f, case["min_new"], case["max_new"], B)
    ctx[0], T[-1] = case["max_ctx"], case["max_new"]
    ctx, T = _shuffled(g, ctx, T)
    M, ln = int(T.sum()), ctx + T
    have = (ln + P - 1) // P
    ld, n_pages = int(have.max()), int(have.sum()) + 3
    table = torch.zeros((B, ld), dtype=torch.int32)
    table[torch.arange(ld)[None, :] < have[:, None]] = torch.randperm(n_pages, generator=g)[: int(have.sum())].int()
    start = torch.cat([torch.zeros(1, dtype=torch.long), T.cumsum(0)])
    mask = None
    words = (case["max_new"] + 63) // 64
    if case["tree"]:
        mask = _ancestors(_parents(g, T.tolist()), T.tolist(), words)[0].to(DEV)
    q = torch.randn((M, case["heads"] * case["dim"]), generator=gg, device=DEV).bfloat16()
    s = dict(q=q, k=_pool(case, n_pages, gg), v=_pool(case, n_pages, gg), table=_i32(table), ctx=_i32(ctx),
             new=_i32(ln), start=_i32(start), mask=mask, P=P, T=case["max_new"], L=int(ln.max()),
             heads=case["heads"], dim=case["dim"])
    if own:
        from megatron_tensor_layers_tp_gb300.runtime import PageTable, Step

        s["model"] = _model(case["heads"], case["kv"], case["dim"], case["ranks"])
        s["pages"] = PageTable(P, s["table"], n_pages=n_pages)
        s["step"] = Step(n_tokens=M, max_new=s["T"], max_ctx=s["L"], old_lens=s["ctx"], new_lens=s["new"],
                         q_start=s["start"], tree_mask=mask)
    return s


def _logits_state(case, g, gg):
    R, N, V, H = case["reqs"], case["nodes"], case["vocab"], case["history"]
    S = R * N
    logits = (3 * torch.randn((S, V), generator=gg, device=DEV)).bfloat16()
    # texts repeat their words: ids fall off as a power of their rank
    ids = (V * torch.rand((R, H), generator=g) ** 3).long().clamp(max=V - 1)
    ln = _ints(g, max(1, H // 2), H, R)
    prompt = (ln.float() * 0.5).long()
    n = min(case["biases"], V)
    count = _ints(g, n // 2, n, R) if n else torch.zeros(R, dtype=torch.long)
    bids = torch.cat([torch.randperm(V, generator=g)[: int(c)] for c in count])
    s = dict(logits=logits, history=_i32(ids), lens=_i32(ln), prompt=_i32(prompt),
             rep=(1 + torch.rand(R, generator=g)).to(DEV), freq=torch.rand(R, generator=g).to(DEV),
             pres=torch.rand(R, generator=g).to(DEV), fp32=case["fp32"], bias_start=None, mask=None, allowed=None,
             row_req=_i32(torch.arange(S) // N))
    if n:
        s.update(bias_start=_i32(torch.cat([torch.zeros(1, dtype=torch.long), count.cumsum(0)])), bias_ids=_i32(bids),
                 bias=torch.randn(len(bids), generator=g).to(DEV), bias_req=torch.arange(R).repeat_interleave(count).to(DEV))
    if N > 1:
        words = (N + 63) // 64
        s.update(mask=_ancestors(_parents(g, [N] * R), [N] * R, words)[0].to(DEV), start=_i32(torch.arange(R + 1) * N),
                 draft=_i32((V * torch.rand(S, generator=g) ** 3).long().clamp(max=V - 1)))
    if case["grammar"]:
        words = (V + 31) // 32
        s["allowed"] = torch.randint(-(2**31), 2**31, (S, words), generator=gg, device=DEV).int()
    if own:
        from megatron_tensor_layers_tp_gb300.runtime import LogitRules

        s["model"] = _model(vocab=V)
        s["rules"] = LogitRules(
            row_req=s["row_req"], history=s["history"], history_lens=s["lens"], prompt_lens=s["prompt"],
            repetition=s["rep"], frequency=s["freq"], presence=s["pres"], draft_tokens=s.get("draft"),
            tree_mask=s["mask"], q_start=s.get("start"), bias_start=s["bias_start"], bias_ids=s.get("bias_ids"),
            bias_values=s.get("bias"), allowed=s["allowed"])
    return s


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op == "tables":
        s = _tables_state(case, g)
    elif op == "append":
        s = _append_state(case, g, gg)
    elif op == "attn":
        s = _attn_state(case, g, gg)
    else:
        s = _logits_state(case, g, gg)
    s["op"], s["case"] = op, case
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_tables(s):
    P, N, T, W = s["P"], s["n_pages"], s["T"], s["words"]
    old, new, table, ring = s["old"].long(), s["new"].long(), s["table"], s["ring"]
    B, ld = table.shape
    have, want = (old + P - 1) // P, (new + P - 1) // P
    pops, push = (want - have).clamp(min=0), (have - want).clamp(min=0)
    first, count = s["free"][0].long(), s["free"][1].long()
    j = torch.arange(ld, device=DEV)[None, :]
    take = (j >= have[:, None]) & (j < want[:, None])
    give = (j >= want[:, None]) & (j < have[:, None])
    at = (first + (pops.cumsum(0) - pops - have)[:, None] + j) % N
    to = (first + count + (push.cumsum(0) - push - want)[:, None] + j) % N
    table[take] = ring[at[take]]
    ring[to[give]] = table[give]
    free = torch.stack([(first + pops.sum()) % N, count - pops.sum() + push.sum()]).int()
    size = (new - old).clamp(min=0)
    end = size.cumsum(0)
    q_start = torch.cat([end.new_zeros(1), end])
    t = torch.arange(s["M"], device=DEV)
    valid = t < end[-1]
    seq = torch.searchsorted(end, t, right=True).clamp(max=B - 1)
    i = t - q_start[seq]
    pos = old[seq] + i
    slots = table[seq, (pos // P).clamp(max=ld - 1)].long() * P + pos % P
    out = {}
    if W:
        # ancestors as the transitive closure of "is the parent of", squared until paths of T are covered
        A = torch.zeros((B * T, T), device=DEV)
        row, par = (seq * T + i)[valid], s["parents"].long()[valid]
        A[row, i[valid]] = 1.0
        A[row[par >= 0], par[par >= 0]] = 1.0
        A = A.view(B, T, T)
        for _ in range(max(1, (T - 1).bit_length())):
            A = (A @ A > 0).float()
        bits = torch.zeros((s["M"], W * 64), dtype=torch.int64, device=DEV)
        bits[valid, :T] = A.view(B * T, T)[row].long()
        pos = old[seq] + bits.sum(1) - 1
        out["mask"] = (bits.view(-1, W, 64) << torch.arange(64, device=DEV)).sum(-1)
    none = torch.tensor(-1, device=DEV)
    out.update(table=table, ring=ring, free=free, q_start=q_start.int(), slots=torch.where(valid, slots, none).int(),
               positions=torch.where(valid, pos, 0).int(), token_seq=torch.where(valid, seq, none).int())
    return out


def _own_tables(s):
    m, st = s["model"], s["step"]
    m.step_tables(s["pages"], st)
    out = dict(table=s["table"], ring=s["ring"], free=s["pages"].free_next, q_start=st.q_start, slots=st.slots,
               positions=st.positions, token_seq=st.token_seq)
    if s["words"]:
        out["mask"] = st.tree_mask
    return out


def _plain_append(s):
    c = s["case"]
    t, nq, kvr, rep, copies = _heads(c)
    d, h, P = c["dim"], c["dim"] // 2, c["page"]
    M = c["tokens"]
    x = s["qkv"].view(t, M, nq + 2 * kvr, d).float()
    ang = s["pos"].double()[:, None] * THETA ** (torch.arange(h, device=DEV).double() * (-2.0 / d))[None, :]
    cos, sin = ang.cos().float()[None, :, None, :], ang.sin().float()[None, :, None, :]
    a, b = x[:, :, : nq + kvr, :h], x[:, :, : nq + kvr, h:]
    r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1).bfloat16()
    q = r[:, :, :nq].transpose(0, 1).reshape(M, t * nq * d)
    ok = s["slots"] >= 0
    page, off = s["slots"][ok].long() // P, s["slots"][ok].long() % P
    s["k"][:, page, :, off] = r[::rep, :, nq:].transpose(0, 1)[ok]
    s["v"][:, page, :, off] = s["qkv"].view(t, M, nq + 2 * kvr, d)[::rep, :, nq + kvr:].transpose(0, 1)[ok]
    return dict(q=q, k=s["k"], v=s["v"])


def _own_append(s):
    q = s["model"].cache_append(s["qkv"], s["pos"], s["slots"], s["pages"], s["k"], s["v"])
    return dict(q=q, k=s["k"], v=s["v"])


def _plain_attn(s):
    d, P, T, L = s["dim"], s["P"], s["T"], s["L"]
    ctx, start = s["ctx"].long(), s["start"].long()
    copies, _, kvr, _, _ = s["k"].shape
    n, B, M = copies * kvr, ctx.numel(), s["q"].shape[0]
    G = s["heads"] // n
    size = start[1:] - start[:-1]
    j = torch.arange(L, device=DEV)
    there = j[None, :] < (ctx + size)[:, None]
    page = torch.where(there, s["table"].long()[:, j // P], 0)
    off = (j % P)[None, :].expand(B, L)
    k = s["k"][:, page, :, off].float().reshape(B, L, n, d).permute(0, 2, 3, 1)
    v = s["v"][:, page, :, off].float().reshape(B, L, n, d).permute(0, 2, 1, 3)
    i = torch.arange(T, device=DEV)
    row = (start[:-1, None] + i).clamp(max=M - 1)
    q = s["q"].float()[row].view(B, T, n, G, d).permute(0, 2, 1, 3, 4).reshape(B, n, T * G, d)
    sc = (q @ k).view(B, n, T, G, L) * (1.0 / math.sqrt(d))
    drafted = (j[None, :] - ctx[:, None])[:, None, :]  # a drafted key's number in its tree
    if s["mask"] is not None:
        w = s["mask"][row]  # [B, T, words]
        word = (drafted // 64).clamp(0, w.shape[2] - 1).expand(B, T, L)
        sees = (w.gather(2, word) >> (drafted % 64)) & 1 == 1
    else:
        sees = drafted <= i[None, :, None]
    sees = (((drafted < 0) | sees) & there[:, None, :])[:, None, :, None, :]
    sc = torch.where(sees, sc, torch.tensor(-math.inf, device=DEV))
    top = sc.amax(-1, keepdim=True)
    e = torch.where(sees, (sc - torch.where(top == -math.inf, 0.0, top)).exp(), 0.0)
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (p.view(B, n, T * G, L) @ v).view(B, n, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, n * G * d)
    return o[i[None, :] < size[:, None]].bfloat16()


def _own_attn(s):
    return s["model"].tree_attention(s["q"], s["step"], s["pages"], s["k"], s["v"])


def _plain_logits(s):
    x = s["logits"].float()
    S, V = x.shape
    req = s["row_req"].long()
    R, H = s["history"].shape
    at = torch.arange(H, device=DEV)[None, :]
    ids = s["history"].long()
    inside = at < s["lens"][:, None]
    written = (inside & (at >= s["prompt"][:, None])).float()
    seen = torch.zeros((R, V), device=DEV).scatter_add_(1, ids, inside.float())[req]
    count = torch.zeros((R, V), device=DEV).scatter_add_(1, ids, written)[req]
    if s["mask"] is not None:
        N = s["case"]["nodes"]
        i = torch.arange(N, device=DEV)
        path = (((s["mask"][:, i // 64] >> (i % 64)) & 1) == 1).float()
        drafted = s["draft"].long()[s["start"].long()[req][:, None] + i[None, :]]
        seen.scatter_add_(1, drafted, path)
        count.scatter_add_(1, drafted, path)
    rep, freq, pres = s["rep"][req][:, None], s["freq"][req][:, None], s["pres"][req][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * count
    x = x - pres * (count > 0).float()
    if s["bias_start"] is not None:
        bias = torch.zeros((R, V), device=DEV)
        bias[s["bias_req"], s["bias_ids"].long()] = s["bias"]
        x = x + bias[req]
    if s["allowed"] is not None:
        v = torch.arange(V, device=DEV)
        ok = (s["allowed"][:, v // 32] >> (v % 32).int()) & 1 == 1
        x = torch.where(ok, x, torch.tensor(-math.inf, device=DEV))
    return x if s["fp32"] else x.bfloat16()


def _own_logits(s):
    return s["model"].process_logits(s["logits"], s["rules"], dtype=torch.float32 if s["fp32"] else torch.bfloat16)


_plain = dict(tables=_plain_tables, append=_plain_append, attn=_plain_attn, logits=_plain_logits)
_own = dict(tables=_own_tables, append=_own_append, attn=_own_attn, logits=_own_logits)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "tables":
        B, T, P = case["seqs"], case["max_new"], case["page"]
        M = B * T // 2 if case["tree"] else B * T * 3 // 4
        words = (T + 63) // 64 if case["tree"] else 0
        # lengths; each new token's slot, position, sequence, parent and mask; new pages from the ring into the table
        return {"bytes": 8 * B + M * (12 + (4 if words else 0) + 8 * words) + 4 * (B + 1) + 8 * (M // P) + 16, "flops": 0}
    if op == "append":
        t, nq, kvr, rep, _ = _heads(case)
        M, d, kept = case["tokens"], case["dim"], 1.0 - case["holes"]
        heads = case["heads"] + 2 * case["kv"] * kept
        return {"bytes": int(2 * M * heads * d * 2 + 8 * M), "flops": int(3 * M * heads * d)}
    if op == "attn":
        B, d = case["seqs"], case["dim"]
        T, C = (case["min_new"] + case["max_new"]) / 2, (case["min_ctx"] + case["max_ctx"]) / 2
        rows = B * T * case["heads"]
        return {"bytes": int(B * (C + T) * case["kv"] * d * 4 + 2 * rows * d * 2), "flops": int(4 * rows * (C + T) * d)}
    S, V, H = case["reqs"] * case["nodes"], case["vocab"], case["history"]
    return {"bytes": int(S * V * (2 + (4 if case["fp32"] else 2)) + (S * V // 8 if case["grammar"] else 0)
                         + case["reqs"] * (3 * H + 6 * case["biases"])), "flops": 0}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def _exact_tables(s):
    P, N, W = s["P"], s["n_pages"], s["words"]
    old, new = s["old"].tolist(), s["new"].tolist()
    table, ring = s["table"].tolist(), s["ring"].tolist()
    first, count = s["free"].tolist()
    parents = s["parents"].tolist() if W else None
    taken, given = 0, 0
    start, slots, pos, seq, mask = [0], [], [], [], []
    returned = []
    for b, (o, n) in enumerate(zip(old, new)):
        have, want = -(-o // P), -(-n // P)
        for p in range(have, want):
            table[b][p] = ring[(first + taken) % N]
            taken += 1
        returned += table[b][want:have]
        here = []
        for i in range(max(n - o, 0)):
            l = o + i
            path = [i]
            while parents and parents[start[-1] + path[-1]] >= 0:
                path.append(parents[start[-1] + path[-1]])
            here.append(sum(1 << p for p in path))
            slots.append(table[b][l // P] * P + l % P)
            pos.append(o + len(path) - 1 if parents else l)
            seq.append(b)
        mask += here
        start.append(start[-1] + max(n - o, 0))
    for p in returned:
        ring[(first + count + given) % N] = p
        given += 1
    pad = s["M"] - len(slots)
    out = dict(table=table, ring=ring, free=[(first + taken) % N, count - taken + given], q_start=start,
               slots=slots + [-1] * pad, positions=pos + [0] * pad, token_seq=seq + [-1] * pad)
    out = {k: torch.tensor(v, dtype=torch.int32) for k, v in out.items()}
    if W:
        rows = [[(m >> (64 * w)) & (2**64 - 1) for w in range(W)] for m in mask + [0] * pad]
        out["mask"] = torch.tensor(rows, dtype=torch.uint64).view(torch.int64)
    return out


def _exact_append(s):
    c = s["case"]
    t, nq, kvr, rep, _ = _heads(c)
    d, P, M = c["dim"], c["page"], c["tokens"]
    half = d // 2
    turn = torch.polar(torch.ones((M, half), dtype=torch.float64, device=DEV), torch.outer(
        s["pos"].double(), torch.tensor([THETA ** (-2.0 * j / d) for j in range(half)], dtype=torch.float64, device=DEV)))
    q = torch.empty((M, c["heads"] * d), dtype=torch.float64, device=DEV)
    k, v = s["k"].double(), s["v"].double()
    rows = (s["slots"] >= 0).nonzero().flatten()
    page, off = s["slots"].long()[rows] // P, s["slots"].long()[rows] % P
    for r in range(t):
        for h in range(nq + 2 * kvr):
            x = s["qkv"][r, :, h * d:(h + 1) * d].double()
            if h < nq + kvr:
                z = torch.complex(x[:, :half], x[:, half:]) * turn
                x = torch.cat([z.real, z.imag], 1)
            if h < nq:
                q[:, (r * nq + h) * d:(r * nq + h + 1) * d] = x
            elif r % rep == 0:
                to, local = (k, h - nq) if h < nq + kvr else (v, h - nq - kvr)
                to[r // rep, page, local, off] = x[rows]
    return dict(q=q, k=k, v=v)


def _exact_attn(s):
    d, P, H = s["dim"], s["P"], s["heads"]
    copies, _, kvr, _, _ = s["k"].shape
    G = H // (copies * kvr)
    ctx, start = s["ctx"].tolist(), s["start"].tolist()
    out = torch.zeros((s["q"].shape[0], H * d), dtype=torch.float64, device=DEV)
    for b, c in enumerate(ctx):
        T = start[b + 1] - start[b]
        if not T:
            continue
        L = c + T
        pages = s["table"][b, : -(-L // P)].long()
        sees = torch.ones((T, L), dtype=torch.bool)
        if s["mask"] is None:
            sees[:, c:] = torch.ones((T, T), dtype=torch.bool).tril()
        else:
            words = s["mask"][start[b]:start[b + 1]].tolist()
            sees[:, c:] = torch.tensor([[bool((w[t // 64] >> (t % 64)) & 1) for t in range(T)] for w in words])
        sees = sees.to(DEV)
        for n in range(copies * kvr):
            k = s["k"][n // kvr, pages, n % kvr].reshape(-1, d)[:L].double()
            v = s["v"][n // kvr, pages, n % kvr].reshape(-1, d)[:L].double()
            for h in range(n * G, (n + 1) * G):
                w = s["q"][start[b]:start[b + 1], h * d:(h + 1) * d].double() @ k.T / math.sqrt(d)
                w = torch.softmax(w.masked_fill(~sees, -math.inf), -1)
                out[start[b]:start[b + 1], h * d:(h + 1) * d] = torch.nan_to_num(w, nan=0.0) @ v
    return out


def _exact_logits(s):
    S, V = s["logits"].shape
    N = s["case"]["nodes"]
    out = torch.empty((S, V), dtype=torch.float64, device=DEV)
    lens, prompt = s["lens"].tolist(), s["prompt"].tolist()
    starts = s["bias_start"].tolist() if s["bias_start"] is not None else None
    paths = s["mask"].tolist() if s["mask"] is not None else None
    for row in range(S):
        r = row // N
        text = s["history"][r].long()
        written = torch.bincount(text[prompt[r]:lens[r]], minlength=V)
        if paths:
            here = [t for t in range(N) if (paths[row][t // 64] >> (t % 64)) & 1]
            written = written + torch.bincount(s["draft"][r * N + torch.tensor(here, device=DEV)].long(), minlength=V)
        seen = (torch.bincount(text[: prompt[r]], minlength=V) + written) > 0
        x = s["logits"][row].double()
        rep = s["rep"][r].double()
        x = torch.where(seen & (x > 0), x / rep, torch.where(seen, x * rep, x))
        x = x - s["freq"][r].double() * written - s["pres"][r].double() * (written > 0)
        if starts:
            x[s["bias_ids"][starts[r]:starts[r + 1]].long()] += s["bias"][starts[r]:starts[r + 1]].double()
        if s["allowed"] is not None:
            bits = (s["allowed"][row].long()[:, None] >> torch.arange(32, device=DEV)[None, :]) & 1
            x[bits.flatten()[:V] == 0] = -math.inf
        out[row] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(tables=_exact_tables, append=_exact_append, attn=_exact_attn, logits=_exact_logits)[case["op"]](s)
