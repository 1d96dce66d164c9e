"""The paged cache of a ragged batch, written plainly in binary64 (loops over requests).

TEST INFRASTRUCTURE ONLY: the reference the library's cache kernels are checked against.

Request i's rows are cu[i] + i .. cu[i + 1] + i; row j takes slot L_i + j and sits at position
L_i + depth(j): j in a linear draft, the length of node j - 1's path in a tree.  Slot s lies in page
page_table[i][s // page_size]; a page outside [0, n_pages) is no page.
"""
from __future__ import annotations

import numpy as np


def depths(parents) -> list[int] | None:
    """Depth per row of a tree (row 0 the last committed token), None if it is not valid."""
    if len(parents) > 64:
        return None
    d = [0]
    for n, p in enumerate(parents):
        if not -1 <= p < n:
            return None
        d.append(d[p + 1] + 1)
    return d


def fits(length, K) -> bool:
    """Whether positions behind `length` cached slots are 32-bit numbers, with room for a tile."""
    return 0 <= length < 2 ** 31 - 1 - 1024 - K


def requests(cu, cache_len, n_draft_rows, parents=None):
    """(i, first row, K, L, depths, visible rows per row) of the requests that are not passed over."""
    for i in range(len(cu) - 1):
        lo, hi = int(cu[i]), int(cu[i + 1])
        if lo < 0 or hi < lo or hi > n_draft_rows or not fits(int(cache_len[i]), hi - lo):
            continue
        K = hi - lo
        if parents is None:
            yield i, lo + i, K, int(cache_len[i]), list(range(K + 1)), [list(range(j + 1)) for j in range(K + 1)]
            continue
        tree = [int(p) for p in parents[lo:hi]]
        d = depths(tree)
        if d is None:
            continue
        see = [[0]]
        for n, p in enumerate(tree):
            see.append(see[p + 1] + [n + 1])
        yield i, lo + i, K, int(cache_len[i]), d, see


def place(table_row, n_pages, page_size, s):
    """(page, place) of slot s, or None."""
    k = s // page_size
    if k >= len(table_row) or not 0 <= table_row[k] < n_pages:
        return None
    return int(table_row[k]), s % page_size


def rotate(x, position, inv_freq, interleaved):
    """x [heads, D] turned in its first 2 len(inv_freq) values."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    angle = float(position) * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(angle), np.sin(angle)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    x[:, a], x[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return x


def append(keys, values, key_cache, value_cache, table, cache_len, cu, inv_freq=(), interleaved=False, parents=None,
           queries=None):
    """(key_cache, value_cache, queries) after the append, in binary64; queries of rows passed over are NaN."""
    kc, vc = np.array(key_cache, dtype=np.float64), np.array(value_cache, dtype=np.float64)
    n_pages, _, ps, _ = kc.shape
    q = None if queries is None else np.full(queries.shape, np.nan)
    for i, row0, K, L, d, _ in requests(cu, cache_len, keys.shape[0] - len(cu) + 1, parents):
        for j in range(K + 1):
            if queries is not None:
                q[row0 + j] = rotate(queries[row0 + j], L + d[j], inv_freq, interleaved)
            at = place(table[i], n_pages, ps, L + j)
            if at is not None:
                kc[at[0], :, at[1]] = rotate(keys[row0 + j], L + d[j], inv_freq, interleaved)
                vc[at[0], :, at[1]] = values[row0 + j]
    return kc, vc, q


def attend(queries, key_cache, value_cache, table, cache_len, cu, scale, window=0, sinks=0, parents=None):
    """(out, absolute, span) per row and head: the attention, sum p |v|, and the largest sum |q k| scale over
    the visible slots (what rounding errors scale with).  Rows passed over are zeros."""
    rows, Hq, D = queries.shape
    n_pages, H, ps, _ = key_cache.shape
    G = Hq // H
    out, absolute = np.zeros((rows, Hq, D)), np.zeros((rows, Hq, D))
    span = np.zeros((rows, Hq))
    kc, vc = np.asarray(key_cache, dtype=np.float64), np.asarray(value_cache, dtype=np.float64)
    for i, row0, K, L, d, see in requests(cu, cache_len, rows - len(cu) + 1, parents):
        for j in range(K + 1):
            pos = [(s, s) for s in range(L)] + [(L + r, L + d[r]) for r in see[j]]
            slots = [s for s, p in pos if window == 0 or L + d[j] - p < window or s < sinks]
            at = [x for x in (place(table[i], n_pages, ps, s) for s in slots) if x is not None]
            if not at:
                continue
            pg, pl = np.array(at).T
            k, v = kc[pg, :, pl], vc[pg, :, pl]  # [n, H, D]
            for h in range(Hq):
                q = np.asarray(queries[row0 + j, h], dtype=np.float64)
                x = k[:, h // G] @ q * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                out[row0 + j, h] = p @ v[:, h // G]
                absolute[row0 + j, h] = p @ np.abs(v[:, h // G])
                span[row0 + j, h] = (np.abs(k[:, h // G]) @ np.abs(q)).max() * abs(scale)
    return out, absolute, span


def settle(key_cache, value_cache, table, cache_len, cu, accepted_len, accepted_nodes):
    """(key_cache, value_cache, new_len): caches [layers, n_pages, H, page_size, D], values unchanged in type."""
    kc, vc = np.array(key_cache), np.array(value_cache)
    n_pages, ps = kc.shape[1], kc.shape[3]
    new_len = np.array(cache_len, dtype=np.int32)
    for i in range(len(cu) - 1):
        lo, K, a, L = int(cu[i]), int(cu[i + 1] - cu[i]), int(accepted_len[i]), int(cache_len[i])
        if lo < 0 or not 0 <= K <= 64 or int(cu[i + 1]) > len(accepted_nodes) or not 0 <= a <= K or not fits(L, K):
            continue
        path = [int(n) for n in accepted_nodes[lo:lo + a]]
        if any(not b < n < K for b, n in zip([-1] + path, path)):
            continue
        new_len[i] = L + 1 + a
        for dd, n in enumerate(path):
            src, dst = place(table[i], n_pages, ps, L + 1 + n), place(table[i], n_pages, ps, L + 1 + dd)
            if src is not None and dst is not None:
                for c in (kc, vc):
                    c[:, dst[0], :, dst[1]] = c[:, src[0], :, src[1]]
    return kc, vc, new_len
