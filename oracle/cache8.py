"""The paged cache in 8 bits, and a round's pages, written plainly (loops over requests, binary64).

TEST INFRASTRUCTURE ONLY: the reference the library's kernels are checked against.

A cache holds e4m3 codes (uint8) and a byte b for each block of tokens and head: the scale 2^(b - 127), b read within
[10, 246].  Requests, rows, slots and pages are those of oracle/cache.py.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.cache import depths, fits, place, requests, rotate  # noqa: F401

LOW, HIGH = 10, 246
KEY_LIMIT, VALUE_LIMIT = 316.0, 448.0


def _decode(code: int) -> float:
    sign, exponent, mantissa = -1.0 if code & 0x80 else 1.0, (code >> 3) & 15, code & 7
    if exponent == 15 and mantissa == 7:
        return math.nan
    if exponent == 0:
        return sign * mantissa * 2.0 ** -9
    return sign * (1 + mantissa / 8) * 2.0 ** (exponent - 7)


DECODED = np.array([_decode(c) for c in range(256)])
_POSITIVE = DECODED[:127]  # 0 .. 448, ascending


def encode(x):
    """The code nearest to x (ties to the even code, the largest beyond 448, NaN of what is not finite)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    below, above = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isfinite(x), code, 0x7f).astype(np.uint8)


def scale_byte(b):
    return np.clip(np.asarray(b, dtype=np.int64), LOW, HIGH)


def scales(b):
    return 2.0 ** (scale_byte(b) - 127.0)


def values(codes, bytes_, block):
    """The numbers that a cache [.., page_size, D] of codes stands for."""
    by = np.repeat(scales(bytes_), block, axis=-1)
    return DECODED[codes] * by[..., None]


def least_byte(top, limit):
    """The byte of the least scale with top <= limit * scale."""
    if top == 0:
        return LOW
    m, e = math.frexp(top / limit)  # m in [0.5, 1): exact enough, checked below
    e -= m == 0.5
    while top > limit * 2.0 ** e:
        e += 1
    while top <= limit * 2.0 ** (e - 1):
        e -= 1
    return int(np.clip(e + 127, LOW, HIGH))


def shifted(codes, shift):
    """Codes times 2^-shift; NaN stays as it is."""
    if shift == 0:
        return codes
    return np.where(np.isnan(DECODED[codes]), codes, encode(np.nan_to_num(DECODED[codes]) * 2.0 ** -float(shift)))


def append8(keys, values_, kc, vc, ks, vs, block, table, cache_len, cu, inv_freq=(), interleaved=False, parents=None,
            queries=None):
    """(key codes, value codes, key bytes, value bytes, queries, exact key values over their scales; NaN where no row is written).
    Codes of rotated keys are those of the binary64 rotation: a kernel's may lie beside them."""
    out = [np.array(x) for x in (kc, vc, ks, vs)]
    n_pages, H, ps, D = kc.shape
    q = None if queries is None else np.full(queries.shape, np.nan)
    exact = np.full(kc.shape, np.nan)
    for i, row0, K, L, d, _ in requests(cu, cache_len, keys.shape[0] - len(cu) + 1, parents):
        if queries is not None:
            for j in range(K + 1):
                q[row0 + j] = rotate(queries[row0 + j], L + d[j], inv_freq, interleaved)
        for first in range(L // block * block, L + K + 1, block):
            at = place(table[i], n_pages, ps, first)
            if at is None:
                continue
            page, where = at
            lo, hi = max(first, L), min(first + block, L + K + 1)
            rows = slice(row0 + lo - L, row0 + hi - L)
            for c, b, x, limit, is_key in ((out[0], out[2], keys, KEY_LIMIT, True), (out[1], out[3], values_, VALUE_LIMIT, False)):
                for h in range(H):
                    raw = np.abs(np.asarray(x[rows, h], dtype=np.float64))
                    byte = least_byte(raw[np.isfinite(raw)].max(initial=0.0), limit)
                    if first < L:
                        old = int(scale_byte(b[page, h, where // block]))
                        held = slice(where, where + L - first)
                        c[page, h, held] = shifted(c[page, h, held], max(byte - old, 0))
                        byte = max(byte, old)
                    b[page, h, where // block] = byte
                    for s in range(lo, hi):
                        v = np.asarray(x[row0 + s - L, h], dtype=np.float64)
                        if is_key:
                            with np.errstate(invalid="ignore"):
                                v = rotate(v[None], L + d[s - L], inv_freq, interleaved)[0]
                        v = v * 2.0 ** (127.0 - byte)
                        c[page, h, s % ps] = encode(v)
                        if is_key:
                            exact[page, h, s % ps] = v
    return out + [q, exact]


def settle8(kc, vc, ks, vs, block, table, cache_len, cu, accepted_len, accepted_nodes):
    """(key codes, value codes, key bytes, value bytes, new_len): caches [layers, n_pages, H, page_size, D]."""
    out = [np.array(x) for x in (kc, vc, ks, vs)]
    layers, n_pages, H, ps, _ = kc.shape
    new_len = np.array(cache_len, dtype=np.int32)
    for i in range(len(cu) - 1):
        lo, K, a, L = int(cu[i]), int(cu[i + 1]) - int(cu[i]), int(accepted_len[i]), int(cache_len[i])
        if lo < 0 or not 0 <= K <= 64 or int(cu[i + 1]) > len(accepted_nodes) or not 0 <= a <= K or not fits(L, K):
            continue
        path = [int(n) for n in accepted_nodes[lo:lo + a]]
        if any(not b < n < K for b, n in zip([-1] + path, path)):
            continue
        new_len[i] = L + 1 + a
        for c, b in ((out[0], out[2]), (out[1], out[3])):
            for layer in range(layers):
                for h in range(H):
                    took = {}  # slot: codes and byte
                    for d, n in enumerate(path):
                        to = place(table[i], n_pages, ps, L + 1 + d)
                        at = place(table[i], n_pages, ps, L + 1 + n) or to
                        if to is not None:
                            took[L + 1 + d] = (c[layer, at[0], h, at[1]].copy(), int(scale_byte(b[layer, at[0], h, at[1] // block])))
                    for first in sorted({s // block * block for s in took}):
                        page, where = place(table[i], n_pages, ps, first)
                        old = int(scale_byte(b[layer, page, h, where // block]))
                        mine = [s for s in took if first <= s < first + block]
                        byte = max([took[s][1] for s in mine] + ([old] if first <= L else []))
                        if first <= L:
                            for s in range(first, min(L + 1, first + block)):
                                c[layer, page, h, s % ps] = shifted(c[layer, page, h, s % ps], byte - old)
                        for s in mine:
                            c[layer, page, h, s % ps] = shifted(took[s][0], byte - took[s][1])
                        b[layer, page, h, where // block] = byte
    return out + [new_len]


def pages(table, page_size, cache_len, n_draft_rows, cu, ring, state, window=0, sinks=0):
    """(table, ring, state, placed, slots) after a round's pages."""
    table, ring, state = (np.array(x) for x in (table, ring, state))
    B, width = table.shape
    n_pages = len(ring)
    placed, slots = np.full(B, -1, dtype=np.int32), np.full(n_draft_rows + B, -1, dtype=np.int64)
    first, count = int(state[0]), int(state[1])
    if not (0 <= first < n_pages and 0 <= count <= n_pages):
        return table, ring, state, placed, slots
    free = [int(ring[(first + x) % n_pages]) for x in range(count)]
    taken, returned, wanted = 0, [], 0
    for i in range(B):
        lo, hi, L = int(cu[i]), int(cu[i + 1]), int(cache_len[i])
        if lo < 0 or hi < lo or hi > n_draft_rows or not (L == -1 or fits(L, hi - lo)):
            continue
        K = hi - lo
        is_page = [0 <= int(p) < n_pages for p in table[i]]
        last = (L + K) // page_size  # of its rows
        needed = set()
        if L >= 0:
            if window == 0:
                needed = set(range(min(last + 1, width)))
            else:
                needed = {k for k in range(min(last + 1, width))
                          if k * page_size < sinks or (k + 1) * page_size - 1 > L - window}
        back = [k for k in range(width) if is_page[k] and k not in needed]
        returned += [int(table[i, k]) for k in back]
        want = []
        placed[i] = 0
        if L >= 0:
            if last < width:
                want = [k for k in range(L // page_size, last + 1) if not is_page[k]]
                wanted += len(want)
                if not want or wanted <= count:
                    placed[i] = 1
        table[i, back] = -1
        if placed[i] == 1:
            for k in want:
                table[i, k] = free[taken]
                taken += 1
            for j in range(K + 1):
                p = int(table[i, (L + j) // page_size])
                if 0 <= p < n_pages:
                    slots[lo + i + j] = p * page_size + (L + j) % page_size
    for x, p in enumerate(returned[:n_pages - count]):
        ring[(first + count + x) % n_pages] = p
    state[0] = (first + taken) % n_pages
    state[1] = count - taken + min(len(returned), n_pages - count)
    return table, ring, state, placed, slots
