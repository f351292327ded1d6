"""Plain 64-bit implementations of the paged-cache serving calls (numpy and
Python numbers, one sequence / row / token at a time), and the inputs the
tests feed to both sides."""
from __future__ import annotations

import numpy as np


def ceil_div(a: int, b: int) -> int:
    return -(-a // b)


# ---------------------------------------------------------------------------
# step tables
# ---------------------------------------------------------------------------
def step_tables(old, new, table, ring, first, count, page, n_tokens, parents=None, words=0):
    """The tables of a step; `table` and `ring` are changed in place.  Returns
    (first, count, q_start, slots, positions, token_seq, masks)."""
    n_pages = len(ring)
    taken, returned = 0, []
    q_start, slots, pos, seq, masks = [0], [], [], [], []
    for b, (o, n) in enumerate(zip(old, new)):
        have, want = ceil_div(o, page), ceil_div(n, page)
        for p in range(have, want):
            table[b][p] = ring[(first + taken) % n_pages]
            taken += 1
        returned += [table[b][p] for p in range(want, have)]
        for i in range(max(n - o, 0)):
            path = [i]
            if parents is not None:
                while parents[q_start[-1] + path[-1]] >= 0:
                    path.append(parents[q_start[-1] + path[-1]])
                masks.append(sum(1 << t for t in path))
            else:
                masks.append((1 << (i + 1)) - 1)
            pos.append(o + (len(path) - 1 if parents is not None else i))
            slots.append(table[b][(o + i) // page] * page + (o + i) % page)
            seq.append(b)
        q_start.append(q_start[-1] + max(n - o, 0))
    for i, p in enumerate(returned):
        ring[(first + count + i) % n_pages] = p
    pad = n_tokens - len(slots)
    masks = [[(m >> (64 * w)) & (2**64 - 1) for w in range(words)] for m in masks + [0] * pad]
    return ((first + taken) % n_pages, count - taken + len(returned), q_start, slots + [-1] * pad,
            pos + [0] * pad, seq + [-1] * pad, masks)


def random_tree(rng, size):
    """Parents of a random tree of `size` tokens (-1: a child of the old tokens)."""
    return [-1 if i == 0 or rng.random() < 0.15 else
            (i - 1 if rng.random() < 0.5 else int(rng.integers(0, i))) for i in range(size)]


def tree_bits(parents):
    """[T, T] truth values: token t is i or an ancestor of i."""
    T = len(parents)
    m = np.zeros((T, T), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def pack_bits(m, words):
    """[rows, T] truth values -> [rows, words] int64 bit patterns."""
    out = np.zeros((m.shape[0], words), dtype=np.uint64)
    for t in range(m.shape[1]):
        out[:, t // 64] |= m[:, t].astype(np.uint64) << np.uint64(t % 64)
    return out.view(np.int64)


# ---------------------------------------------------------------------------
# rotary embedding, attention
# ---------------------------------------------------------------------------
def rotate(x, pos, theta):
    """x [M, heads, d] in float64, pos [M]."""
    d = x.shape[-1]
    half = d // 2
    out = np.empty_like(x)
    for j in range(half):
        ang = np.asarray(pos, dtype=np.float64) * theta ** (-2.0 * j / d)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        out[:, :, j] = x[:, :, j] * c - x[:, :, j + half] * s
        out[:, :, j + half] = x[:, :, j + half] * c + x[:, :, j] * s
    return out


def attention_row(q, k, v, sees):
    """One row: q [d], k, v [L, d], sees [L].  Returns (o, sum of p |v|, score
    bound |q||k| / sqrt d); zeros when it sees nothing."""
    d = q.shape[0]
    if not sees.any():
        return np.zeros(d), np.zeros(d), 0.0
    k, v = k[sees], v[sees]
    s = k @ q / np.sqrt(d)
    e = np.exp(s - s.max())
    p = e / e.sum()
    bound = float((np.abs(k) @ np.abs(q)).max() / np.sqrt(d))
    return p @ v, p @ np.abs(v), bound


# ---------------------------------------------------------------------------
# logits
# ---------------------------------------------------------------------------
def logit_row(x, prompt=(), output=(), rep=1.0, freq=0.0, pres=0.0, biases=(), allowed=None):
    """One row: x [V] float64.  Returns (row, the sum of its terms' magnitudes)."""
    x = x.copy()
    V = len(x)
    mag = np.abs(x)
    count = {}
    for t in output:
        if 0 <= t < V:
            count[t] = count.get(t, 0) + 1
    for t in set(int(t) for t in prompt if 0 <= t < V) | set(count):
        x[t] = x[t] / rep if x[t] > 0 else x[t] * rep
        mag[t] = abs(x[t])
    for t, c in count.items():
        x[t] = x[t] - freq * c - pres
        mag[t] += abs(freq * c) + abs(pres)
    for t, w in biases:
        if 0 <= t < V:
            x[t] += w
            mag[t] += abs(w)
    if allowed is not None:
        x[~allowed] = -np.inf
        mag[~allowed] = 0.0
    return x, mag
