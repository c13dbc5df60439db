"""Float64 reference of what lies between a block's projections: the norm of each
head with the position rotation and its backward pass, a paged cache written
slot by slot, and the attention over it, row by row.

Written from the formulas, on float64 arrays; what the GPU stores in a narrower
type in between (a rounded key in the cache) is an input here.
"""

from __future__ import annotations

import numpy as np


def _pairs(dim: int, rot: int, interleaved: bool):
    """The channels (a, b) of every turned pair."""
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def turn(x, positions, inv_freq, interleaved=False, sign=1.0):
    """x (tokens x heads x dim) with its first 2 len(inv_freq) channels turned."""
    x = np.array(x, np.float64)
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    if rot == 0:
        return x
    a, b = _pairs(x.shape[2], rot, interleaved)
    angle = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(angle), sign * np.sin(angle)
    xa, xb = x[:, :, a].copy(), x[:, :, b].copy()
    x[:, :, a], x[:, :, b] = xa * c - xb * s, xb * c + xa * s
    return x


def head_norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=2, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rope(x, weight, positions, inv_freq, eps, interleaved=False):
    return turn(head_norm(x, weight, eps), positions, inv_freq, interleaved)


def rope_backward(dy, x, weight, positions, inv_freq, eps, interleaved=False):
    """(dx, dweight); dweight None without a weight."""
    dz = turn(dy, positions, inv_freq, interleaved, -1.0)
    if weight is None:
        return dz, None
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=2, keepdims=True) + eps)
    u = w * dz
    dx = r * u - x * r ** 3 * np.mean(u * x, axis=2, keepdims=True)
    return dx, np.sum(dz * x * r, axis=(0, 1))


def rows(starts, tokens):
    """(sequence, place in it) of each row that belongs to one; others are absent."""
    out = {}
    for i in range(len(starts) - 1):
        for t in range(starts[i], starts[i + 1]):
            if 0 <= t < tokens:
                out[t] = (i, t - starts[i])
    return out


def place(seq, key, table, page_size, pages):
    """(page, slot) of a sequence's key; None where it has none."""
    column = key // page_size
    if key < 0 or column >= table.shape[1] or not 0 <= table[seq, column] < pages:
        return None
    return int(table[seq, column]), key % page_size


def append(k_pages, v_pages, k, v, starts, lens, table):
    """Copies of the pages (pages x heads x slots x dim) with the rows' keys and values in them."""
    k_pages, v_pages = np.array(k_pages), np.array(v_pages)
    for t, (i, n) in rows(starts, len(k)).items():
        at = place(i, lens[i] - (starts[i + 1] - starts[i]) + n, table, k_pages.shape[2], k_pages.shape[0])
        if at is not None:
            k_pages[at[0], :, at[1]], v_pages[at[0], :, at[1]] = k[t], v[t]
    return k_pages, v_pages


def seen(seq, n, starts, lens, tree_word=None):
    """The keys that row n of a sequence sees."""
    count = starts[seq + 1] - starts[seq]
    base = lens[seq] - count
    if tree_word is None:
        return list(range(0, base + n + 1))
    word = int(tree_word) & (2 ** 64 - 1)
    return list(range(0, base)) + [base + j for j in range(min(count, 64)) if word >> j & 1 and base + j >= 0]


def attention(q, k_pages, v_pages, starts, lens, table, scale, tree=None):
    """(out, lse) of every row (tokens x heads x dim, tokens x heads), NaN where a row belongs to no sequence."""
    q, k_pages, v_pages = (np.asarray(a, np.float64) for a in (q, k_pages, v_pages))
    tokens, heads, dim = q.shape
    group = heads // k_pages.shape[1]
    out, lse = np.full(q.shape, np.nan), np.full((tokens, heads), np.nan)
    for t, (i, n) in rows(starts, tokens).items():
        keys = [place(i, j, table, k_pages.shape[2], k_pages.shape[0]) for j in
                seen(i, n, starts, lens, None if tree is None else tree[t])]
        keys = [a for a in keys if a is not None]
        page, slot = np.array([a[0] for a in keys], int), np.array([a[1] for a in keys], int)
        for h in range(heads):
            if not keys:
                out[t, h], lse[t, h] = 0.0, -np.inf
                continue
            s = scale * (k_pages[page, h // group, slot] @ q[t, h])
            m = np.max(s)
            p = np.exp(s - m)
            out[t, h], lse[t, h] = p @ v_pages[page, h // group, slot] / np.sum(p), m + np.log(np.sum(p))
    return out, lse


def accept(pages, path, starts, lens, table):
    """A copy of the pages with every sequence's accepted rows moved together."""
    old, new = np.asarray(pages), np.array(pages)
    for i in range(len(lens)):
        count = starts[i + 1] - starts[i]
        for j, p in enumerate(path[i]):
            if not 0 <= p < count or j >= count:
                continue
            a = place(i, lens[i] - count + p, table, old.shape[2], old.shape[0])
            b = place(i, lens[i] - count + j, table, old.shape[2], old.shape[0])
            if a is not None and b is not None:
                new[b[0], :, b[1]] = old[a[0], :, a[1]]
    return new
