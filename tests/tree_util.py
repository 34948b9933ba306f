"""Inputs of the tests of drafted trees and of caches whose tokens carry their own scales."""
from __future__ import annotations

import numpy as np
import torch

from oracle import tree as ot
from tests import cache_util as cu

TYPES = ["bf16", "f32", "f8", "f8t"]


class Case(cu.Case):
    """A cache with sequences; "f8t" has k_tok and v_tok [layers][pages][Hkv][page] besides the entries."""
    k_tok = v_tok = None

    def values(self):
        if self.dtype != "f8t":
            return super().values()
        k, v = self.k_pool.float().double().numpy(), self.v_pool.float().double().numpy()
        v_tok = self.v_tok.double().numpy()
        return (k * self.k_tok.double().numpy()[..., None],
                v * v_tok.reshape(*v_tok.shape[:3], -1, 1, 8))

    def pools(self, device="cuda"):
        """The pools as the library takes them."""
        if self.dtype != "f8t":
            return self.k_pool.to(device), self.v_pool.to(device)
        return tuple(join(x, s).to(device) for x, s in ((self.k_pool, self.k_tok), (self.v_pool, self.v_tok)))

    def scales(self, device="cuda"):
        return (self.k_scale.to(device), self.v_scale.to(device)) if self.dtype == "f8" else (None, None)


def join(entries, scales):
    """A pool of bytes from its entries and scales."""
    layers, pages, Hkv = entries.shape[:3]
    return torch.cat([entries.contiguous().view(torch.uint8).reshape(layers, pages, Hkv, -1),
                      scales.contiguous().view(torch.uint8).reshape(layers, pages, Hkv, -1)], 3)


def make(seed, dtype, page, D, Hq, Hkv, n_new, length, **kw):
    c = cu.make(seed, "f8" if dtype == "f8t" else dtype, page, D, Hq, Hkv, n_new, length, **kw)
    c = Case(**{**vars(c), "dtype": dtype})
    if dtype == "f8t":
        gen = torch.Generator().manual_seed(seed + 1)
        layers, pages = c.k_pool.shape[:2]
        c.k_tok, c.v_tok = ((torch.randn((layers, pages, Hkv, page), generator=gen) * 0.5).exp() * 0.025 for _ in range(2))
        if kw.get("poison", True):  # places of no token: scales that are not finite
            used = np.zeros((pages, page), bool)
            for b, s in enumerate(c.length):
                for j in range(s):
                    used[c.table[b, j // page], j % page] = True
            free = torch.from_numpy(~used)[:, None]
            for x, bad in ((c.k_tok, float("nan")), (c.v_tok, float("inf"))):
                x.masked_fill_(free, bad)
    return c


def handle(ds, c, max_new, layers=1):
    B, width = c.table.shape
    C = ds.Cache.make(B, c.k_pool.shape[1], c.page, width, layers, c.q.shape[1], c.k_pool.shape[2], c.q.shape[2],
                      q="f32" if c.dtype == "f32" else "bf16", cache=c.dtype)
    return C, torch.empty(ds.cache_workspace_bytes(C, max_new), dtype=torch.uint8, device="cuda").fill_(255)


def parents(rng, n, wide=3):
    """A tree of n nodes: node 0 hangs from the context, node i from one of the earlier ones, mostly near i / wide."""
    return [-1 if i == 0 else int(rng.integers(i // wide, i)) for i in range(n)]


def trees(seed, c, max_new=None, window=0):
    """Parents [rows], and the oracle's words and depths, of a tree for each request."""
    rng = np.random.default_rng(seed)
    max_new = max(1, int(c.n_new.max())) if max_new is None else max_new
    parent = np.full(len(c.q), -1, np.int64)
    for n, r in zip(c.n_new, c.row_start):
        parent[r:r + n] = parents(rng, int(n))
    return (parent, *ot.mask(parent, c.n_new, c.row_start, len(parent), max_new, window))


def words_i32(words, device="cuda"):
    return torch.from_numpy(words.view(np.int32).copy()).to(device)


def oracle_tree(c, words, depth, layer=0, scale=None, window=0):
    k, v = c.values()
    return ot.attend(c.q.double().numpy(), words, depth, c.n_new, c.row_start, c.length, c.table, k, v, layer=layer,
                     page=c.page, scale=c.q.shape[2] ** -0.5 if scale is None else scale, window=window)


def gpu_tree(ds, c, words, depth, layer=0, scale=None, window=0, with_lse=True, max_new=None, layers=1):
    max_new = max(1, int(c.n_new.max())) if max_new is None else max_new
    C, ws = handle(ds, c, max_new, layers)
    q = c.q.cuda()
    out = torch.full_like(q, 77.0)
    lse = torch.full(q.shape[:2], 77.0, device="cuda") if with_lse else None
    print(f"[gpu] tree {c.dtype} page={c.page} D={q.shape[2]} Hq={q.shape[1]} Hkv={C.Hkv} n_new={c.n_new.tolist()[:6]} "
          f"length={c.length.tolist()[:6]} window={window}", flush=True)
    ds.tree_attend(C, layer, q, cu.i32(c.n_new), cu.i32(c.row_start), max_new, words_i32(words),
                   None if depth is None else cu.i32(depth), cu.i32(c.length), cu.i32(c.table), *c.pools(), *c.scales(), out,
                   lse, ws, scale=scale, window=window)
    torch.cuda.synchronize()
    return out.cpu(), None if lse is None else lse.cpu()


def gpu_attend(ds, c, layer=0, causal=True, window=0, max_new=None, layers=1):
    max_new = max(1, int(c.n_new.max())) if max_new is None else max_new
    C, ws = handle(ds, c, max_new, layers)
    q = c.q.cuda()
    out, lse = torch.full_like(q, 77.0), torch.full(q.shape[:2], 77.0, device="cuda")
    print(f"[gpu] attend {c.dtype} page={c.page} D={q.shape[2]} Hq={q.shape[1]} Hkv={C.Hkv} n_new={c.n_new.tolist()[:6]} "
          f"length={c.length.tolist()[:6]} causal={causal} window={window}", flush=True)
    ds.cache_attend(C, layer, q, cu.i32(c.n_new), cu.i32(c.row_start), max_new, cu.i32(c.length), cu.i32(c.table),
                    *c.pools(), *c.scales(), out, lse, ws, causal=causal, window=window)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check(c, out, lse, ref):
    """Against the oracle, within cache_util.attend_bound: a token's scale is one more factor of a score, one more rounding
    (the bound takes D + 12 of them for a product of D terms), and one of its weight (8 u)."""
    want, want_lse, mag, span = ref
    got = out.double().numpy()
    none = np.isnan(want_lse)
    assert (got[none] == 77.0).all(), "rows of no request were written"
    keep = ~none
    tol, tol_lse = cu.attend_bound(c.dtype, want[keep], want_lse[keep], mag[keep], span[keep], int(c.length.max()))
    bad = ~(np.abs(got[keep] - want[keep]) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got[keep] - want[keep]) / tol):.3g} "
                           f"bounds, first at {np.argwhere(bad)[:3].tolist()}")
    if lse is not None:
        g = lse.double().numpy()
        assert (g[none] == 77.0).all()
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(g), empty)
        k2 = keep & ~empty
        assert (np.abs(g[k2] - want_lse[k2]) <= tol_lse[~empty[keep]]).all()
