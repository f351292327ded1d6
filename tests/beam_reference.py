"""Plain 64-bit implementations of beam selection, of the texts behind their
parents, and of forks and compaction of page tables (numpy and Python numbers,
one request / row / page at a time)."""
from __future__ import annotations

import numpy as np

from tests.paged_reference import ceil_div


def finite(x):
    """NaN counts as -infinity, +infinity as the largest fp32 number."""
    return np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))


def row_values(x, score):
    """The values of a row's continuations: x [V] float64, -inf where there is none."""
    x = finite(x)
    if not np.isfinite(score) or not (x > -np.inf).any():
        return np.full(len(x), -np.inf)
    top = x.max()
    with np.errstate(under="ignore"):
        d = x - top
        return d - np.log(np.exp(d).sum()) + float(score)


def select(x, scores, W, K, ends=()):
    """x [R*W, V] float64, scores [R*W].  Returns per request its candidates [(value, row, token)],
    at most K, and its next beams, at most W.  Equal values go by row, logit and token."""
    out = []
    for r in range(len(scores) // W):
        pool = []
        for b in range(r * W, (r + 1) * W):
            v = row_values(x[b], scores[b])
            logits = finite(x[b])
            at = np.argsort(-logits, kind="stable")[:K]
            pool += [(v[i], b, int(i), -logits[i]) for i in at if v[i] > -np.inf]
        pool.sort(key=lambda c: (-c[0], c[1], c[3], c[2]))
        pool = [c[:3] for c in pool[:K]]
        out.append((pool, [c for c in pool if c[2] not in ends][:W]))
    return out


def fork(table, lens, src, keep, page, ring, first, count):
    """Rows of pages after the fork, and (moves, ring, first, count, rows a page has)."""
    n_pages, rows = len(ring), range(len(table))
    keep = [0 if src[b] < 0 else lens[src[b]] if keep is None else keep[b] for b in rows]
    was = {p for b in rows for p in table[b][:ceil_div(lens[b], page)]}
    full = {table[src[b]][i] for b in rows if src[b] >= 0 for i in range(keep[b] // page)}
    new, moves, mine = [], [], set()
    for b in rows:
        row = list(table[src[b]][:keep[b] // page]) if src[b] >= 0 else []
        if keep[b] % page:
            p = table[src[b]][keep[b] // page]
            if p in full or p in mine:
                q = ring[(first + len(moves)) % n_pages]
                moves.append((p, q, keep[b] % page))
                p = q
            else:
                mine.add(p)
            row.append(p)
        new.append(row)
    holders = {}
    for row in new:
        for p in row:
            holders[p] = holders.get(p, 0) + 1
    gone = sorted(p for p in was if p not in holders)
    ring = list(ring)
    for i, p in enumerate(gone):
        ring[(first + count + i) % n_pages] = p
    return new, keep, moves, ring, (first + len(moves)) % n_pages, count - len(moves) + len(gone), holders


def compact(table, lens, page, n_pages):
    """Rows of pages by their new names, and (moves, pages held, rows a page has)."""
    holders = {}
    for b, n in enumerate(lens):
        for p in table[b][:ceil_div(n, page)]:
            holders[p] = holders.get(p, 0) + 1
    used = len(holders)
    movers = sorted((p for p in holders if p >= used), reverse=True)
    holes = [p for p in range(used) if p not in holders]
    name = dict(zip(movers, holes))
    rows = [[name.get(p, p) for p in table[b][:ceil_div(n, page)]] for b, n in enumerate(lens)]
    return rows, [(a, b, page) for a, b in zip(movers, holes)], used, \
        {name.get(p, p): c for p, c in holders.items()}


def shared_tables(rng, reqs, width, page, max_len, spare, idle=0.1):
    """Tables of requests whose beams share full pages of a prefix, in shuffled pages."""
    lens, table, at, ld = [], [], 0, ceil_div(max_len, page) + 1
    for _ in range(reqs):
        n = int(rng.integers(0, max_len + 1))
        common = int(rng.integers(0, n // page + 1))
        prefix = list(range(at, at + common))
        at += common
        held = False
        for _ in range(width):
            m = 0 if rng.random() < idle else max(common * page, n - int(rng.integers(0, 3)) * (page // 2))
            own = ceil_div(m, page) - common if m else 0
            table.append((prefix + list(range(at, at + own))) if m else [])
            held |= m > 0
            at += own
            lens.append(m)
        if not held:  # (pages that no row holds are no row's)
            at -= common
    n_pages = at + spare
    perm = rng.permutation(n_pages).tolist()
    rows = [[perm[p] for p in r] + [-5] * (ld - len(r)) for r in table]
    held = {p for r in rows for p in r}
    free = [p for p in range(n_pages) if p not in held]
    rng.shuffle(free)
    first = int(rng.integers(0, n_pages))
    ring = [-9] * n_pages
    for i, p in enumerate(free):
        ring[(first + i) % n_pages] = p
    return dict(lens=lens, table=rows, ring=ring, first=first, count=len(free), page=page, n_pages=n_pages,
                max_ctx=max_len)
