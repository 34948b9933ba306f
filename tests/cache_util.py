"""Inputs of the paged-cache tests: sequences dealt over a shuffled pool, with
NaN in every place that no sequence holds."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from oracle import cache as oc

DATA = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.bfloat16}
STORE = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}
U = 2.0**-24           # half a step of fp32, relative
HALF = {"f32": U, "bf16": 2.0**-8}  # of the data types


@dataclass
class Case:
    """Host tensors of a cache with sequences in it and rows of new tokens."""
    dtype: str
    page: int
    n_new: np.ndarray
    row_start: np.ndarray
    length: np.ndarray
    table: np.ndarray
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor

    def values(self):
        """The pools' values in float64 (scaled)."""
        k, v = self.k_pool.float().double().numpy(), self.v_pool.float().double().numpy()
        if self.dtype == "f8":
            k = k * self.k_scale.double().numpy()[:, None, None]
            v = v * self.v_scale.double().numpy()[:, None, None, None]
        return k, v


def make(seed, dtype, page, D, Hq, Hkv, n_new, length, *, layers=1, layer=0, spare=2, width=None, gap=0, poison=True,
         q_std=1.5, slots=None):
    """Requests with `length` cached tokens of which n_new are new; `gap` unused rows between requests' rows."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    n_new, length = np.asarray(n_new, np.int64), np.asarray(length, np.int64)
    need = -(-length // page)
    n_pages = int(need.sum()) + spare
    width = int(max(1, need.max())) if width is None else width
    order = rng.permutation(n_pages)
    table = np.full((len(length), width), -1, np.int64)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    k_pool = torch.randn((layers, n_pages, Hkv, page, D), generator=gen)
    v_pool = torch.randn((layers, n_pages, Hkv, page // 8, D, 8), generator=gen)
    if dtype == "f8":
        k_pool, v_pool = (x.mul_(40).clamp_(-448, 448) for x in (k_pool, v_pool))
    if poison:
        used = np.zeros((n_pages, page), bool)
        for b, s in enumerate(length):
            for j in range(s):
                used[table[b, j // page], j % page] = True
        free = torch.from_numpy(~used)
        k_pool.masked_fill_(free[:, None, :, None], float("nan"))
        v_pool.masked_fill_(free.view(n_pages, page // 8, 8)[:, None, :, None, :], float("nan"))
    k_pool, v_pool = k_pool.to(STORE[dtype]), v_pool.to(STORE[dtype])
    row_start = np.cumsum(n_new + gap) - (n_new + gap)
    rows = int((n_new + gap).sum())
    data = DATA[dtype]
    return Case(dtype, page, n_new, row_start, length, table, k_pool, v_pool,
                torch.rand(Hkv, generator=gen) * 0.02 + 0.02, torch.rand(Hkv, generator=gen) * 0.02 + 0.02,
                (torch.randn((rows, Hq, D), generator=gen) * q_std).to(data),
                torch.randn((rows, Hkv, D), generator=gen).to(data), torch.randn((rows, Hkv, D), generator=gen).to(data))


def i32(a, device="cuda"):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=device)


def attend_bound(dtype, out, lse, mag, span, n_keys):
    """How far out and lse may be from the float64 values.

    u = 2^-24.  A score is a product sum of D terms in fp32 and some factors: off by at most (D + 8) u times
    the sum of the terms' sizes (`span`, its largest value; D <= 256: 264 u).  exp2 of a difference of scores
    adds the rounding of its argument (|t| <= 2 span, log2(e) included: 4 span u) and 4 u of its own; the running
    maximum's corrections multiply at most one such factor per position.  With e the relative error of a weight,
    out (a quotient of two sums of n terms) is off by at most mag (2 e + (2 n + 64) u), to which a bf16 call adds half a
    step for the weights' rounding (2^-8 mag) and half a step for its own (2^-8 |out|)."""
    e = np.expm1(268 * U * span) + 8 * U
    n = n_keys + 32
    tol = mag * (2 * e + 6 * n * U)[..., None] + np.abs(out) * U
    if dtype != "f32":
        tol = tol + 2.0**-8 * mag + 2.0**-8 * (np.abs(out) + tol)
    tol_lse = e + 6 * n * U + 4 * U * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return tol + 1e-37, tol_lse


def oracle_attend(c: Case, layer=0, scale=None, causal=True, window=0):
    k, v = c.values()
    return oc.attend(c.q.double().numpy(), c.n_new, c.row_start, c.length, c.table, k, v, layer=layer, page=c.page,
                     scale=c.q.shape[2] ** -0.5 if scale is None else scale, causal=causal, window=window)
