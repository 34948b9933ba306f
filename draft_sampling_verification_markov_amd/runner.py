"""Device buffers for one cycle and the three library calls in order.

Plumbing around the binding: uploads host arrays (bf16 given as raw uint16
bit patterns, fp32 as float32), allocates the caller-owned outputs and the
workspace with torch, and issues dspark_draft -> dspark_schedule ->
dspark_verify on the current stream.

PagedCache owns the buffers of the paged key/value cache, and run_cached_cycle
is the cycle with the target's forward pass over that cache between the schedule
and the verification.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass

import numpy as np
import torch

from . import dspark


def to_device(a: np.ndarray, device="cuda") -> torch.Tensor:
    """Upload a host array; uint16 arrays are bf16 bit patterns."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    if a.dtype == np.float32:
        return torch.from_numpy(a).to(device)
    if a.dtype in (np.int32, np.int64):
        return torch.from_numpy(a.astype(np.int32)).to(device)
    raise TypeError(a.dtype)


@dataclass
class CycleInputs:
    Z: torch.Tensor
    Zt: torch.Tensor
    E: torch.Tensor
    Wt: torch.Tensor
    h: torch.Tensor
    w_c: torch.Tensor
    b_c: float
    tau: torch.Tensor
    anchor: torch.Tensor
    T: torch.Tensor

    @classmethod
    def upload(cls, inp: dict, device="cuda") -> "CycleInputs":
        return cls(Z=to_device(inp["Z"], device), Zt=to_device(inp["Zt"], device), E=to_device(inp["E"], device),
                   Wt=to_device(inp["Wt"], device), h=to_device(inp["h"], device), w_c=to_device(inp["w_c"], device),
                   b_c=float(inp["b_c"]), tau=to_device(inp["tau"], device), anchor=to_device(inp["anchor"], device),
                   T=to_device(inp["T"], device))


class CycleOutputs:
    """Caller-owned outputs of the three calls plus the shared workspace."""

    def __init__(self, P: dspark.Problem, device="cuda"):
        B, K = P.B, P.K
        f32, i32 = torch.float32, torch.int32
        self.tok = torch.empty((B, K), dtype=i32, device=device)
        self.logq = torch.empty((B, K), dtype=f32, device=device)
        self.lse = torch.empty((B, K), dtype=f32, device=device)
        self.conf = torch.empty((B, K), dtype=f32, device=device)
        self.surv = torch.empty((B, K), dtype=f32, device=device)
        self.n_sched = torch.empty((B,), dtype=i32, device=device)
        self.n_total = torch.empty((1,), dtype=i32, device=device)
        self.out_tok = torch.empty((B, K + 1), dtype=i32, device=device)
        self.n_acc = torch.empty((B,), dtype=i32, device=device)
        self.next_anchor = torch.empty((B,), dtype=i32, device=device)
        self.logp = torch.empty((B, K), dtype=f32, device=device)
        self.resid_mass = torch.empty((B,), dtype=f32, device=device)
        nbytes = dspark.workspace_bytes(P)
        if nbytes == 0:
            raise ValueError("invalid problem")
        self.workspace = torch.empty((nbytes,), dtype=torch.uint8, device=device)

    def host(self) -> dict:
        return {k: v.cpu().numpy() for k, v in vars(self).items() if k != "workspace"}


def draft(P, x: CycleInputs, o: CycleOutputs, stream=None, path: int = dspark.DRAFT_AUTO):
    if path == dspark.DRAFT_AUTO:
        dspark.draft(P, x.Z, x.E, x.Wt, x.h, x.w_c, x.b_c, x.tau, x.anchor,
                     o.tok, o.logq, o.lse, o.conf, o.surv, o.workspace, stream)
    else:
        dspark.draft_timed(P, x.Z, x.E, x.Wt, x.h, x.w_c, x.b_c, x.tau, x.anchor,
                           o.tok, o.logq, o.lse, o.conf, o.surv, o.workspace, None, stream, path=path)


def schedule(P, x: CycleInputs, o: CycleOutputs, stream=None):
    dspark.schedule(P, o.surv, x.T, o.n_sched, o.n_total, o.workspace, stream)


def verify(P, x: CycleInputs, o: CycleOutputs, stream=None, n_sched=None):
    """n_sched: the drafts to judge, the schedule's unless others are given."""
    dspark.verify(P, x.Zt, x.Z, x.E, x.Wt, x.anchor, o.tok, o.logq, o.lse, o.n_sched if n_sched is None else n_sched,
                  o.out_tok, o.n_acc, o.next_anchor, o.logp, o.resid_mass, o.workspace, stream)


def run_cycle(P, x: CycleInputs, o: CycleOutputs, stream=None, path: int = dspark.DRAFT_AUTO):
    draft(P, x, o, stream, path)
    schedule(P, x, o, stream)
    verify(P, x, o, stream)


def _on(stream):
    """torch's operations on `stream`, or on the current one."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class PagedCache:
    """Pools, page tables, lengths and references of a paged cache, and its calls.

    table, length and ref are the present sequences; update writes the other set of
    them and swaps the two, compact those of table and ref (so a captured graph holds an even
    number of updates, grow's and keep's among them, and of compactions).

    New tokens, a tree's nodes among them, lie at the end of a sequence, and the calls over them take their number, n_new.
    A pool without room, or the end of a row of the page table, leaves a slot fewer than were asked for: n_new is then what
    the slot got (grow), since a larger count would take tokens that the sequence holds already for new ones.

    max_new, of the cache, is the most new tokens of a slot in a call (its workspace is made for them).  Work is planned
    for it, and without row_start slot b's rows begin at b * max_new, so that calls of fewer (trees, which have up to 1024
    nodes, or single tokens, in a cache made for prompts) take a max_new of their own, the same in all that belong together."""

    def __init__(self, C: dspark.Cache, max_new: int, device="cuda", k_scale=None, v_scale=None):
        self.C, self.max_new = C, int(max_new)
        i32 = torch.int32
        self.k = torch.zeros(C.k_shape, dtype=torch.uint8, device=device).to(C.cache_type) if C.cache_dtype == dspark.F8E4M3 \
            else torch.zeros(C.k_shape, dtype=C.cache_type, device=device)
        self.v = torch.zeros_like(self.k).view(C.v_shape)
        self.k_scale, self.v_scale = k_scale, v_scale
        if C.cache_dtype == dspark.F8E4M3:
            one = torch.ones(C.Hkv, dtype=torch.float32, device=device)
            self.k_scale = one if k_scale is None else k_scale
            self.v_scale = one if v_scale is None else v_scale
        self._sets = [(torch.full((C.B, C.max_pages), -1, dtype=i32, device=device),
                       torch.zeros(C.B, dtype=i32, device=device), torch.zeros(C.n_pages, dtype=i32, device=device))
                      for _ in range(2)]
        self.n_short = torch.zeros(1, dtype=i32, device=device)
        self._none_short = torch.zeros_like(self.n_short)
        self.n_live = torch.zeros(1, dtype=i32, device=device)
        self._kept = torch.zeros(C.B, dtype=i32, device=device)
        nbytes = dspark.cache_workspace_bytes(C, self.max_new)
        if nbytes == 0:
            raise ValueError("invalid cache")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)

    table = property(lambda self: self._sets[0][0])
    length = property(lambda self: self._sets[0][1])
    ref = property(lambda self: self._sets[0][2])

    def update(self, new_len, parent=None, stream=None, n_short=None):
        """Every slot's next sequence (dspark_cache_update); n_short (the cache's own, unless another is given) tells
        the pages that were missing."""
        now, new = self._sets
        dspark.cache_update(self.C, parent, new_len, *now, *new, self.n_short if n_short is None else n_short, self.k,
                            self.v, self.workspace, stream)
        self._sets.reverse()

    def _most(self, max_new):
        """A call's max_new: the cache's, or a smaller one."""
        if max_new is None:
            return self.max_new
        if not 1 <= max_new <= self.max_new:
            raise ValueError(f"max_new {max_new} of a cache made for up to {self.max_new} new tokens a slot")
        return max_new

    def grow(self, n_new, stream=None, max_new=None):
        """Every slot longer by n_new [B] rows (clamped to [0, max_new]) as far as there is room.  Returns the rows that each
        got, the n_new of the calls that follow, without reading anything back: none where the pool has no room (n_short
        tells the pages that were missing), at the end of its row of the page table those that fit."""
        self._ints(n_new=n_new)
        with _on(stream):
            before = self.length
            self.update(before + n_new.clamp(0, self._most(max_new)), stream=stream)
            return self.length - before

    def compact(self, stream=None):
        """Live pages to the lowest ids (dspark_cache_compact); n_live tells how many there are."""
        now, new = self._sets
        dspark.cache_compact(self.C, *now, new[0], new[2], self.n_live, self.k, self.v, self.workspace, stream)
        self._sets = [(new[0], now[1], new[2]), (now[0], new[1], now[2])]

    def append(self, layer: int, k, v, n_new=None, row_start=None, stream=None, max_new=None):
        dspark.cache_append(self.C, layer, k, v, n_new, row_start, self._most(max_new), self.length, self.table,
                            self.k_scale, self.v_scale, self.k, self.v, stream)

    def attend(self, layer: int, q, out, lse=None, n_new=None, row_start=None, scale=None, causal=True, window=0,
               stream=None, max_new=None):
        dspark.cache_attend(self.C, layer, q, n_new, row_start, self._most(max_new), self.length, self.table, self.k,
                            self.v, self.k_scale, self.v_scale, out, lse, self.workspace, scale, causal, window, stream)

    def _ints(self, **tensors):
        """Refuses what is no tensor of one int32 a slot (and would be broadcast or converted)."""
        for name, t in tensors.items():
            dspark._dev(t, torch.int32, (self.C.B,), self.n_short.get_device(), name)

    # ---- drafts that form trees (dspark_tree.h); nodes are the new tokens
    def mask(self, parent, mask, depth=None, n_new=None, row_start=None, window=0, stream=None, max_new=None):
        """Ancestor bits and depths of the trees with these parents [rows] (dspark_tree_mask: max_new up to 1024)."""
        max_new = self._most(max_new)
        if n_new is None and row_start is None and parent.numel() != self.C.B * max_new:
            raise ValueError(f"{parent.numel()} parents for {self.C.B} trees of {max_new} nodes")
        dspark.tree_mask(parent, n_new, row_start, max_new, mask, depth, window, stream)

    def tree_attend(self, layer: int, q, mask, out, lse=None, depth=None, n_new=None, row_start=None, scale=None, window=0,
                    stream=None, max_new=None):
        dspark.tree_attend(self.C, layer, q, n_new, row_start, self._most(max_new), mask, depth, self.length, self.table,
                           self.k, self.v, self.k_scale, self.v_scale, out, lse, self.workspace, scale, window, stream)

    def keep(self, path, n_keep, n_new=None, stream=None, max_new=None):
        """The accepted nodes path[b][: n_keep[b]] (ascending), and nothing else of the new tokens, stay: their keys and
        values move to the first new places (dspark_tree_keep), and the sequences end behind them (update).  With n_new a
        path ends before the first node that is not among them: one that lost its place to a lack of room (17 us of the
        call's 47, 256 slots)."""
        max_new = self._most(max_new)
        if n_new is not None:
            if isinstance(path, torch.Tensor) and path.dim() != 2:
                raise ValueError(f"path has shape {tuple(path.shape)}, expected [{self.C.B}][nodes]")
            self._ints(n_keep=n_keep, n_new=n_new)
            dspark._dev(path, torch.int32, (self.C.B, *getattr(path, "shape", ())[1:]), self.n_short.get_device(), "path")
            with _on(stream):
                n_keep = torch.minimum(n_keep, (path < n_new[:, None]).sum(1, dtype=torch.int32))
        dspark.tree_keep(self.C, path, n_keep, n_new, max_new, self.length, self.table, self._kept, self.k, self.v, stream)
        self.update(self._kept, stream=stream, n_short=self._none_short)


def run_cached_cycle(P, x: CycleInputs, o: CycleOutputs, cache: PagedCache, forward, path: int = dspark.DRAFT_AUTO):
    """One cycle over a paged cache, on the current stream, without reading anything back.

    After the schedule the cache grows by the n_sched + 1 rows of every request (the anchor and its
    drafts); forward(tokens [B][K + 1], n_new [B]) runs the target over them (cache.append and
    cache.attend per layer, rows b * (K + 1) ..) and leaves its logits in x.Zt; after the verification
    the cache keeps the anchor and the accepted drafts.

    Returns n_new [B], the rows that each request got.  Where the pool cannot hold a request's rows it gets none
    (n_new 0), and cache.n_short tells the pages that were missing; at the end of its row of the page table it gets those
    that fit.  Of n_new rows the first n_new - 1 drafts are judged (o.n_sched stays the schedule's).  A request without
    rows emits nothing: its out_tok is -1 throughout, n_acc -1, its next_anchor its anchor, and its sequence stays as
    it was.

    The cache's slots are the problem's requests, and its max_new is K + 1; with a larger one (ValueError for a smaller)
    forward has to pass row_start, since without it request b's rows begin at b * max_new."""
    if cache.C.B != P.B or cache.max_new < P.K + 1:
        raise ValueError(f"a cache of {cache.C.B} slots and up to {cache.max_new} new rows a slot for {P.B} requests of "
                         f"up to {P.K + 1}")
    draft(P, x, o, path=path)
    schedule(P, x, o)
    before = cache.length
    cache.update(before + o.n_sched + 1)
    n_new = cache.length - before
    forward(torch.cat([x.anchor[:, None], o.tok], 1), n_new)
    verify(P, x, o, n_sched=(n_new - 1).clamp(min=0))
    # what verify made of logits that no forward pass wrote
    none = n_new == 0
    o.n_acc.masked_fill_(none, -1)
    o.out_tok.masked_fill_(none[:, None], -1)
    o.logp.masked_fill_(none[:, None], float("nan"))
    o.resid_mass.masked_fill_(none, float("nan"))
    o.next_anchor.copy_(torch.where(none, x.anchor, o.next_anchor))
    cache.update(before + o.n_acc + 1, n_short=cache._none_short)  # (this one only shrinks)
    return n_new
