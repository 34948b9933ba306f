"""Trees of drafted tokens over a paged cache, and a cache whose tokens carry their own
scales, from the definitions (one node, one token at a time)."""
from __future__ import annotations

import numpy as np

from .cache import F8_MAX, round_f8, sequence


def ancestors(parent):
    """Per node of one tree (parent[i] outside [0, i): none) the list of itself and its ancestors, nearest first."""
    chains = []
    for i, p in enumerate(parent):
        chains.append([i] + (chains[int(p)] if 0 <= int(p) < i else []))
    return chains


def mask(parent, n_new, row_start, n_rows, max_new, window=0):
    """Words [n_rows][ceil(max_new / 32)] (uint32) and depths [n_rows]; rows of no request are 0xFFFFFFFF and -7."""
    words = np.full((n_rows, -(-max_new // 32)), 0xFFFFFFFF, np.uint32)
    depth = np.full(n_rows, -7, np.int64)
    for b in range(len(n_new)):
        n, r0 = min(max(int(n_new[b]), 0), max_new), int(row_start[b])
        rows = [r0 + i for i in range(n)]
        there = [0 <= r < n_rows for r in rows]
        for i, chain in enumerate(ancestors([parent[r] if t else -1 for r, t in zip(rows, there)])):
            if not there[i]:
                continue
            words[rows[i]] = 0
            depth[rows[i]] = len(chain) - 1
            for k, a in enumerate(chain):
                if window == 0 or k < window:
                    words[rows[i], a // 32] |= np.uint32(1 << a % 32)
    return words, depth


def sees(words, i, base, length, depth, window):
    """Positions that node i of a request sees, its nodes starting at position `base`."""
    first = max(0, base + depth - window + 1) if window else 0
    context = [j for j in range(first, max(base, 0))]
    nodes = [base + k for k in range(i + 1) if int(words[k // 32]) >> (k % 32) & 1 and 0 <= base + k < length]
    return np.array(context + nodes, np.int64)


def attend(q, words, depth, n_new, row_start, length, table, k_pool, v_pool, *, layer, page, scale, window=0):
    """As cache.attend, for the nodes of trees."""
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
                r = int(row_start[b]) + i
                if not 0 <= r < rows:
                    continue
                d = min(max(int(depth[r]), 0), i)
                at = sees(words[r], i, s - n, s, d, window)
                for g in range(G):
                    x = q[r, h * G + g]
                    if len(at) == 0:
                        out[r, h * G + g] = mag[r, h * G + g] = span[r, h * G + g] = 0.0
                        lse[r, h * G + g] = -np.inf
                        continue
                    t = scale * (k[at] @ x)
                    top = t.max()
                    w = np.exp(t - top)
                    z = w.sum()
                    out[r, h * G + g] = (w @ v[at]) / z
                    mag[r, h * G + g] = (w @ np.abs(v[at])) / z
                    lse[r, h * G + g] = top + np.log(z)
                    span[r, h * G + g] = scale * (np.abs(k[at]) @ np.abs(x)).max()
    return out, lse, mag, span


def keep(pools, path, n_keep, n_new, length, table, *, page, places):
    """length_out; each pool's tokens moved in place.  places(pool, page id, offset) is the view of a token in all layers."""
    out = []
    for b in range(len(length)):
        n, s = int(n_new[b]), int(length[b])
        base = s - n
        m = min(max(int(n_keep[b]), 0), path.shape[1], n)
        out.append(max(0, base + m))
        for i in range(m):
            src = base + int(path[b, i])
            if not 0 <= int(path[b, i]) < n or src < 0 or base + i < 0:
                continue
            for p in pools:
                places(p, table[b][(base + i) // page], (base + i) % page)[...] = places(p, table[b][src // page], src % page)
    return np.array(out)


def quantise_token(x):
    """Entries and scale of rows [..][D] (float32 values) with a scale of their own, in the arithmetic of the cache: a
    float32 scale, a float32 quotient, the nearest e4m3 value."""
    x = np.asarray(x, np.float32)
    size = np.where(np.isfinite(x), np.abs(x), np.float32(0))
    top = size.max(-1)
    scale = np.where(top > 0, np.maximum(top / np.float32(F8_MAX), np.float32(2.0**-126)), np.float32(1))
    return round_f8((x / scale[..., None]).astype(np.float64)), scale.astype(np.float64)
