"""Rotary rotation, append to a paged cache, and attention over it (oracle, fp64).

  rotation  for every pair i < rot / 2 of a head, (a, b) = elements (i, i + rot / 2),
            or (2 i, 2 i + 1) when interleaved:
            a' = a c - b s, b' = b c + a s with c, s = table[position][i], [rot / 2 + i]
  append    row r goes to slot = page * page_size + place; negative slots, and those
            past the cache, are left out; E4M3 caches hold codes of v / scale with
            scale = max|v| / 448 of the head
  attention z_j = scale q . k_j over the visible tokens j of a row at position i:
            j <= i and (window == 0 or i - j < window or j < sinks);
            y = sum softmax(z)_j v_j, lse = log sum exp z; nothing visible: 0, -inf
"""

import numpy as np


def rotate(x, positions, table, interleaved):
    """x [m][heads][d], positions [m], table [max_pos][rot] -> fp64."""
    y = np.array(x, np.float64)
    table = np.asarray(table, np.float64)
    rot = table.shape[1]
    half = rot // 2
    for r, pos in enumerate(positions):
        t = table[min(max(int(pos), 0), len(table) - 1)]
        for i in range(half):
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            a, b = y[r, :, ia].copy(), y[r, :, ib].copy()
            y[r, :, ia] = a * t[i] - b * t[half + i]
            y[r, :, ib] = b * t[i] + a * t[half + i]
    return y


def slots_of(slots, pages, page_size):
    """(rows that are stored, their pages, their places)."""
    s = np.asarray(slots, np.int64)
    rows = np.nonzero((s >= 0) & (s < pages * page_size))[0]
    return rows, s[rows] // page_size, s[rows] % page_size


def tokens(cache, table_row, n):
    """The first n tokens of a sequence, [n][kv_heads][d], of a cache [pages][kv_heads]
    [page_size][d]; entries outside the cache are the nearest page."""
    j = np.arange(n)
    size = cache.shape[2]
    page = np.clip(np.asarray(table_row, np.int64)[j // size], 0, cache.shape[0] - 1)
    return cache[page, :, j % size]


def visible(position, n, window, sinks):
    j = np.arange(n)
    seen = j <= position
    if window:
        seen &= (position - j < window) | (j < sinks)
    return seen


def attend(q, k, v, position, scale, window=0, sinks=0):
    """One row: q [heads][d], k and v [n][kv_heads][d] -> (y [heads][d], lse [heads],
    weights [heads][n], what bounds z: sum |q k| scale [heads][n])."""
    heads, d = q.shape
    n, kv = k.shape[:2]
    y, lse = np.zeros((heads, d)), np.full(heads, -np.inf)
    w, mag = np.zeros((heads, n)), np.zeros((heads, n))
    seen = visible(position, n, window, sinks)
    if not seen.any():
        return y, lse, w, mag
    for h in range(heads):
        kh = h // (heads // kv)
        z = k[seen, kh] @ q[h] * scale
        mag[h, seen] = np.abs(k[seen, kh]) @ np.abs(q[h]) * scale
        big = z.max()
        e = np.exp(z - big)
        lse[h] = big + np.log(e.sum())
        w[h, seen] = e / e.sum()
        y[h] = w[h, seen] @ v[seen, kh]
    return y, lse, w, mag
