"""Paged cache in float64 numpy: attention over pages, and the bookkeeping of
pages, from the definitions (one request, one slot, one page at a time).

Pools are float64 arrays of the values that the cache holds, in the library's
layout: keys [layers][pages][Hkv][page][D], values [layers][pages][Hkv][page/8][D][8].
"""
from __future__ import annotations

import numpy as np

F8_MAX = 448.0


def f8_values() -> np.ndarray:
    """The 127 non-negative finite e4m3 values (no infinities; 0x7f is NaN)."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0**-9, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def round_f8(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to the even code, past +-448 saturated, NaN kept."""
    table = f8_values()
    a = np.minimum(np.abs(np.asarray(x, np.float64)), F8_MAX)
    hi = np.clip(np.searchsorted(table, a), 1, 126)
    lo = hi - 1
    d_lo, d_hi = a - table[lo], table[hi] - a
    pick = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), np.nan, np.copysign(table[pick], x))


def held(tokens: int, page: int) -> int:
    return -(-int(tokens) // page)


def sequence(pool, layer, pages, tokens, head, page, values):
    """The first `tokens` keys or values of a sequence, [tokens][D]."""
    rows = []
    for j in range(tokens):
        p = pages[j // page]
        off = j % page
        rows.append(pool[layer, p, head, off // 8, :, off % 8] if values else pool[layer, p, head, off])
    D = pool.shape[4]
    return np.array(rows).reshape(tokens, D)


def attend(q, n_new, row_start, length, table, k_pool, v_pool, *, layer, page, scale, causal=True, window=0):
    """out, lse [rows][Hq], and per output element the sum of w |v| / sum of w and per (row, head) the largest
    |scale * sum_d |q_d k_d|| over the visible positions (for error bounds); rows of no request are NaN."""
    rows, Hq, D = q.shape
    Hkv = k_pool.shape[2]
    G = Hq // Hkv
    out, mag = np.full((2, rows, Hq, D), np.nan)
    lse, span = np.full((2, rows, Hq), np.nan)
    for b in range(len(length)):
        n, s = int(n_new[b]), int(length[b])
        for h in range(Hkv):
            if n == 0:
                continue
            k = sequence(k_pool, layer, table[b], s, h, page, False)
            v = sequence(v_pool, layer, table[b], s, h, page, True)
            for i in range(n):
                pos = s - n + i
                lo = max(0, pos - window + 1) if window else 0
                hi = min(s, pos + 1) if causal else s
                lo, hi = min(lo, s), max(hi, 0)
                r = int(row_start[b]) + i
                for g in range(G):
                    x = q[r, h * G + g]
                    if hi <= lo:
                        out[r, h * G + g], mag[r, h * G + g], span[r, h * G + g] = 0.0, 0.0, 0.0
                        lse[r, h * G + g] = -np.inf
                        continue
                    t = scale * (k[lo:hi] @ x)
                    top = t.max()
                    w = np.exp(t - top)
                    z = w.sum()
                    out[r, h * G + g] = (w @ v[lo:hi]) / z
                    mag[r, h * G + g] = (w @ np.abs(v[lo:hi])) / z
                    lse[r, h * G + g] = top + np.log(z)
                    span[r, h * G + g] = scale * (np.abs(k[lo:hi]) @ np.abs(x)).max()
    return out, lse, mag, span


def append(k_pool, v_pool, k, v, n_new, row_start, length, table, *, layer, page):
    """The pools with the new tokens written (k, v [rows][Hkv][D]: the values to be stored)."""
    k_pool, v_pool = k_pool.copy(), v_pool.copy()
    for b in range(len(length)):
        n, s = int(n_new[b]), int(length[b])
        for i in range(n):
            pos, r = s - n + i, int(row_start[b]) + i
            if pos < 0 or not 0 <= r < len(k):
                continue
            p, off = table[b][pos // page], pos % page
            if not 0 <= p < k_pool.shape[1]:
                continue
            k_pool[layer, p, :, off] = k[r]
            v_pool[layer, p, :, off // 8, :, off % 8] = v[r]
    return k_pool, v_pool


def update(parent, new_len, table, length, ref, *, page):
    """table, length, ref, n_short and the page copies [(from, to)] of the next sequences."""
    B, width = table.shape
    n_pages = len(ref)
    ref = [int(x) for x in ref]
    rows, keep, want = [], [], []
    for b in range(B):
        w = min(max(int(new_len[b]), 0), width * page)
        p = int(parent[b]) if parent is not None else b
        m = min(min(max(int(length[p]), 0), width * page), w) if 0 <= p < B else 0
        rows.append([int(x) for x in table[p][:held(m, page)]] if m else [])
        keep.append(m)
        want.append(w)
    for b in range(B):
        for x in table[b][:held(min(max(int(length[b]), 0), width * page), page)]:
            if 0 <= x < n_pages:
                ref[x] -= 1
    for r in rows:
        for x in r:
            if 0 <= x < n_pages:
                ref[x] += 1
    shared = list(ref)
    free = [x for x in range(n_pages) if ref[x] == 0]
    given, copies, out_len = 0, [], []
    for b, r in enumerate(rows):
        if want[b] == keep[b]:
            out_len.append(keep[b])
            continue
        copy = keep[b] % page != 0 and 0 <= r[-1] < n_pages and shared[r[-1]] > 1
        need = held(want[b], page) - len(r) + copy
        if need and given + need > len(free):
            out_len.append(keep[b])
            given += need
            continue
        mine = free[given:given + need]
        given += need
        if copy:
            copies.append((r[-1], mine[0]))
            ref[r[-1]] -= 1
            r[-1] = mine[0]
        r.extend(mine[copy:])
        for x in mine:
            ref[x] = 1
        out_len.append(want[b])
    out = np.full((B, width), -1, np.int64)
    for b, r in enumerate(rows):
        out[b, :len(r)] = r
    return out, np.array(out_len), np.array(ref), max(0, given - len(free)), copies


def compact(table, length, ref, *, page):
    """table, ref, n_live and the page moves [(from, to)] that leave the live pages below n_live."""
    n_live = int((ref > 0).sum())
    high = [p for p in range(n_live, len(ref)) if ref[p] > 0]
    holes = [p for p in range(n_live) if ref[p] <= 0]
    to = dict(zip(high, holes))
    out = np.full(table.shape, -1, np.int64)
    for b in range(len(table)):
        for i in range(held(min(max(int(length[b]), 0), table.shape[1] * page), page)):
            p = int(table[b, i])
            if 0 <= p < len(ref) and ref[p] > 0:
                out[b, i] = to.get(p, p)
    new = np.zeros(len(ref), np.int64)
    for p in range(len(ref)):
        if ref[p] > 0:
            new[to.get(p, p)] = ref[p]
    return out, new, n_live, list(to.items())
