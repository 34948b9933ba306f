"""The paged cache's oracle against what its definitions imply."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests import cache_util as cu


def test_f8_rounding_matches_the_type():
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    want = x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oc.round_f8(x.numpy()), want)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 5), (False, 5)])
def test_attend_against_a_dense_softmax(causal, window):
    c = cu.make(0, "f32", 16, 64, 4, 2, [3, 2], [20, 33], poison=False)
    out, lse, mag, span = cu.oracle_attend(c, causal=causal, window=window)
    k, v = c.values()
    for b in range(2):
        n, s = int(c.n_new[b]), int(c.length[b])
        pos = torch.arange(s - n, s)[:, None]
        j = torch.arange(s)
        hide = (j > pos) if causal else torch.zeros(n, s, dtype=torch.bool)
        if window:
            hide = hide | (j <= pos - window)
        for hq in range(4):
            kk = torch.from_numpy(oc.sequence(k, 0, c.table[b], s, hq // 2, 16, False))
            vv = torch.from_numpy(oc.sequence(v, 0, c.table[b], s, hq // 2, 16, True))
            r = int(c.row_start[b])
            x = (c.q[r:r + n, hq].double() @ kk.T / 8.0).masked_fill(hide, -float("inf"))
            np.testing.assert_allclose(out[r:r + n, hq], (x.softmax(-1) @ vv).numpy(), rtol=1e-12, atol=1e-13)
            np.testing.assert_allclose(lse[r:r + n, hq], x.logsumexp(-1).numpy(), rtol=1e-12)


def holders(table, length, page, n_pages):
    n = np.zeros(n_pages, np.int64)
    for r, s in zip(table, length):
        for x in r[:oc.held(s, page)]:
            n[x] += 1
    return n


def test_update_keeps_references_and_contents():
    rng = np.random.default_rng(0)
    B, n_pages, page, width = 7, 24, 16, 9
    table, length, ref = np.full((B, width), -1), np.zeros(B, np.int64), np.zeros(n_pages, np.int64)
    content = np.full((n_pages, page), -1)
    seqs = [[] for _ in range(B)]
    shortages = 0
    for _ in range(200):
        parent = np.where(rng.random(B) < 0.6, np.arange(B), rng.integers(0, B, B))
        new = np.clip(length[parent] + rng.integers(-25, 30, B), 0, width * page)
        before = length
        table, length, ref, short, copies = oc.update(parent, new, table, length, ref, page=page)
        shortages += short > 0
        np.testing.assert_array_equal(ref, holders(table, length, page, n_pages))
        for a, b in copies:
            content[b] = content[a]
        kept = [seqs[p][:min(before[p], w)] for p, w in zip(parent, new)]
        seqs = []
        for b in range(B):
            s = kept[b]
            for j in range(len(s), length[b]):  # write the growth: the page must be this slot's alone
                assert ref[table[b, j // page]] == 1
                content[table[b, j // page], j % page] = tok = int(rng.integers(1 << 30))
                s = s + [tok]
            seqs.append(s[:length[b]])
        if rng.random() < 0.3:
            table, ref, n_live, moves = oc.compact(table, length, ref, page=page)
            old = content.copy()
            for a, b in moves:
                content[b] = old[a]
            assert (ref[:n_live] > 0).all() and (ref[n_live:] == 0).all()
        for b in range(B):
            got = [content[table[b, j // page], j % page] for j in range(length[b])]
            assert got == seqs[b]
    assert shortages
