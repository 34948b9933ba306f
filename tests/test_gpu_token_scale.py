"""A paged cache whose tokens carry their own scales, on the GPU against the float64 oracle: appended entries and scales
bit for bit, attention (types of layout, pages, row counts, masks, places of no token full of NaN), and the
bookkeeping that moves whole pages."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache as oc  # noqa: E402
from oracle import tree as ot  # noqa: E402
from tests import cache_util as cu  # noqa: E402
from tests import tree_util as tu  # noqa: E402
from tests.test_gpu_cache import ds  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8)


# ------------------------------------------------------------------ append
def append_and_check(ds, c, k, v, layer=0, max_new=None):  # noqa: F811
    """k, v [rows][Hkv][D]; every byte of both pools against the oracle's."""
    max_new = max(1, int(c.n_new.max())) if max_new is None else max_new
    C, _ = tu.handle(ds, c, max_new, c.k_pool.shape[0])
    kp, vp = c.pools()
    before = kp.clone(), vp.clone()
    ds.cache_append(C, layer, k, v, cu.i32(c.n_new), cu.i32(c.row_start), max_new, cu.i32(c.length), cu.i32(c.table), None,
                    None, kp, vp)
    torch.cuda.synchronize()
    for pool, old, x, values in ((kp, before[0], k, False), (vp, before[1], v, True)):
        (e, s), (e0, s0) = C.token_views(pool.cpu(), values), C.token_views(old.cpu(), values)
        want, scale = ot.quantise_token(x.float().cpu().numpy())
        e1, s1 = e0.float().numpy().copy(), s0.numpy().copy()
        written = np.zeros(s1.shape, bool)
        for b in range(len(c.length)):
            for i in range(int(c.n_new[b])):
                pos, r = int(c.length[b]) - int(c.n_new[b]) + i, int(c.row_start[b]) + i
                if pos < 0 or not 0 <= r < len(want):
                    continue
                p, off = c.table[b, pos // c.page], pos % c.page
                if not 0 <= p < e1.shape[1]:
                    continue
                if values:
                    e1[layer, p, :, off // 8, :, off % 8] = want[r]
                else:
                    e1[layer, p, :, off] = want[r]
                s1[layer, p, :, off] = scale[r]
                written[layer, p, :, off] = True
        assert np.array_equal(e.float().numpy(), e1, equal_nan=True)
        assert np.array_equal(s.numpy(), s1, equal_nan=True)
        keep = ~written.reshape(*written.shape[:3], c.page // 8, 1, 8) if values else ~written[..., None]
        keep = torch.from_numpy(np.broadcast_to(keep, e1.shape).copy())
        assert torch.equal(bits(e)[keep], bits(e0)[keep])  # (NaN too, as it was)


@pytest.mark.parametrize("D,Hkv", [(64, 1), (64, 9), (128, 2), (128, 5), (256, 1), (256, 3)])
@pytest.mark.parametrize("page", [16, 128])
def test_append(ds, D, Hkv, page):  # noqa: F811
    c = tu.make(1, "f8t", page, D, Hkv, Hkv, [1, 7, 0, 16, 9, 3], [1, 30, 20, 16, 47, 250], gap=1, layers=2)
    spread = torch.logspace(-12, 12, len(c.k))[:, None, None]
    append_and_check(ds, c, (c.k * spread).bfloat16().cuda(), (c.v * spread.flip(0)).bfloat16().cuda(), layer=1)


def test_append_values_that_are_not_finite(ds):  # noqa: F811
    c = tu.make(2, "f8t", 16, 64, 2, 2, [6, 2], [20, 2])
    inf = float("inf")
    k, v = c.k.clone(), c.v.clone()
    k[0, 0, 3], k[1, 1, :], k[2, 0, :], k[3, 1, 5] = float("nan"), float("nan"), 0.0, -inf
    v[0, 1, 63], v[4, 0, :], v[5, 1, 0], v[6, 0, :] = float("nan"), inf, inf, 0.0
    k[7, 0, :] = 1e-38
    append_and_check(ds, c, k.cuda(), v.cuda())


def test_append_strided_rows_and_bad_places(ds):  # noqa: F811
    # rows of one projection; a page id out of range, positions before 0, rows outside the array
    c = tu.make(3, "f8t", 16, 128, 3, 3, [5, 9, 4], [40, 3, 20])
    c.table[0, 2] = 10 ** 6
    c.row_start = np.array([0, 5, len(c.k) - 2])
    kv = torch.cat([c.k, c.v], 1).cuda()
    append_and_check(ds, c, kv[:, :3], kv[:, 3:])
    append_and_check(ds, c, kv[:, :3], kv[:, 3:], max_new=300)


def test_append_many_requests(ds):  # noqa: F811
    i = np.arange(700)
    c = tu.make(4, "f8t", 16, 64, 1, 1, np.where(i % 3 == 0, 0, 1 + i % 4), 4 + i % 30, poison=False)
    append_and_check(ds, c, c.k.cuda(), c.v.cuda())


# ------------------------------------------------------------------ attend
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 8, 2), (256, 6, 2), (128, 5, 1), (64, 12, 1)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_attend_ragged(ds, D, Hq, Hkv, page):  # noqa: F811
    c = tu.make(11, "f8t", page, D, Hq, Hkv, [1, 5, 0, 3, 2], [1, 37, 20, 3, 130], gap=1)
    tu.check(c, *tu.gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("causal,window", [(True, 1), (True, 33), (False, 0), (False, 7), (True, 2000)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("G", [2, 8])
def test_attend_masks(ds, causal, window, wide, G):  # noqa: F811
    c = tu.make(12, "f8t", 32, 128, 2 * G, 2, [9, 1, 17, 0], [100, 260, 17, 40], width=200 if wide else None)
    tu.check(c, *tu.gpu_attend(ds, c, causal=causal, window=window), cu.oracle_attend(c, causal=causal, window=window))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 257])
@pytest.mark.parametrize("D", [64, 256])
def test_attend_every_length(ds, n, D):  # noqa: F811
    c = tu.make(10 + n, "f8t", 16, D, 4, 2, [1, 2, min(n, 40)], [n, n + 1, n])
    tu.check(c, *tu.gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("D,page", [(64, 32), (128, 16), (128, 256), (256, 16), (256, 64)])
@pytest.mark.parametrize("rows,G", [(1, 3), (17, 4), (40, 2), (150, 2), (301, 1)])
@pytest.mark.parametrize("wide", [False, True])
def test_attend_row_counts(ds, D, page, rows, G, wide):  # noqa: F811
    c = tu.make(20 + rows, "f8t", page, D, 2 * G, 2, [rows, 1, rows // 2], [rows + 333, 700, rows // 2],
                width=5000 // page if wide else None)
    tu.check(c, *tu.gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("rows", [3, 40])
def test_attend_values_that_are_not_finite(ds, rows):  # noqa: F811
    # a NaN among the entries of a key or of a value reaches the rows that see it and no other
    c = tu.make(31, "f8t", 16, 128, 4, 2, [rows, 2], [rows + 50, 30])
    clean = cu.oracle_attend(c)
    nan = float("nan")
    pos = rows + 50 - rows // 2  # among the new tokens: seen by the rows from there on
    p, off = c.table[0, pos // 16], pos % 16
    for which in ("k", "v"):
        d = tu.make(31, "f8t", 16, 128, 4, 2, [rows, 2], [rows + 50, 30])
        if which == "k":
            d.k_pool[0, p, 0, off, 5] = nan
        else:
            d.v_pool[0, p, 0, off // 8, 5, off % 8] = nan
        out, lse = tu.gpu_attend(ds, d)
        first = pos - 50
        assert torch.isfinite(out[:first]).all() and torch.isfinite(out[rows:]).all()
        seen = out[first:rows]
        assert torch.isfinite(seen[:, 2:]).all()  # the other kv head
        if which == "k":
            assert torch.isnan(seen[:, :2]).all() and torch.isnan(lse[first:rows, :2]).all()
        else:
            assert torch.isnan(seen[:, :2, 5]).all() and torch.isfinite(seen[:, :2, :5]).all()
        for r in list(range(first)) + [rows, rows + 1]:
            assert np.allclose(out[r].double().numpy(), clean[0][r], rtol=2e-2, atol=2e-2)


def test_attend_scales_far_apart(ds):  # noqa: F811
    # a token many orders of magnitude above the others, in its key and in its value, and scales of the smallest numbers
    c = tu.make(41, "f8t", 16, 64, 4, 2, [4, 20], [60, 90])
    c.k_tok[0, c.table[0, 1], :, 3] *= 1e3
    c.v_tok[0, c.table[0, 2], :, 7] *= 1e20
    c.v_tok[0, c.table[1, 0], :, :] = 2.0 ** -126
    c.k_tok[0, c.table[1, 0], :, 1] = 1e-38
    tu.check(c, *tu.gpu_attend(ds, c), cu.oracle_attend(c))


def test_tokens_written_and_read(ds):  # noqa: F811
    # what append stores is what attend reads, and near what was given
    B, Hq, Hkv, D, page, T = 3, 8, 2, 128, 16, 40
    c = tu.make(51, "f8t", page, D, Hq, Hkv, [T] * B, [T, T, T])
    C, ws = tu.handle(ds, c, T)
    kp, vp = c.pools()
    n, rs, le, ta = cu.i32(c.n_new), cu.i32(c.row_start), cu.i32(c.length), cu.i32(c.table)
    ds.cache_append(C, 0, c.k.cuda(), c.v.cuda(), n, rs, T, le, ta, None, None, kp, vp)
    out, lse = torch.zeros_like(c.q, device="cuda"), torch.zeros(c.q.shape[:2], device="cuda")
    ds.cache_attend(C, 0, c.q.cuda(), n, rs, T, le, ta, kp, vp, None, None, out, lse, ws)
    c.k_pool, c.k_tok = (x.cpu().contiguous() for x in C.token_views(kp))
    c.v_pool, c.v_tok = (x.cpu().contiguous() for x in C.token_views(vp, True))
    tu.check(c, out.cpu(), lse.cpu(), cu.oracle_attend(c))
    exact = tu.make(51, "f32", page, D, Hq, Hkv, [T] * B, [T, T, T])
    for r in range(len(c.k)):
        b, i = r // T, r % T
        p = exact.table[b, i // page]
        exact.k_pool[0, p, :, i % page], exact.v_pool[0, p, :, i % page // 8, :, i % 8] = c.k[r].float(), c.v[r].float()
    exact.q = c.q.float()
    want = cu.oracle_attend(exact)[0]
    # entries are off by 2^-4 of their value at most; scores by 2^-4 of theirs: a loose check of the whole
    assert np.abs(out.cpu().double().numpy() - want).mean() < 0.06


# ------------------------------------------------------------------ whole pages
@pytest.mark.parametrize("n_pages", [40, 9000])
def test_update_and_compact_move_scales(ds, n_pages):  # noqa: F811
    B, Hkv, D, page, width, layers = 4, 3, 64, 16, 8, 2
    C = ds.Cache.make(B, n_pages, page, width, layers, Hkv, Hkv, D, cache="f8t")
    rng = np.random.default_rng(60)
    length = np.array([37, 90, 16, 5])
    table, ref, order, at = np.full((B, width), -1), np.zeros(n_pages, np.int64), rng.permutation(n_pages), 0
    for b, s in enumerate(length):
        table[b, :oc.held(s, page)] = order[at:at + oc.held(s, page)]
        at += oc.held(s, page)
    ref[table[table >= 0]] = 1
    kp, vp = (torch.randint(0, 256, C.k_shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    k0, v0 = kp.cpu().numpy(), vp.cpu().numpy()
    ws = torch.empty(ds.cache_workspace_bytes(C, 8), dtype=torch.uint8, device="cuda")
    parent, new = np.array([0, 0, 2, 0]), np.array([40, 37, 20, 42])
    t1, l1, r1 = torch.empty(B, width, dtype=torch.int32, device="cuda"), cu.i32(length), cu.i32(ref)
    l2, r2, short = torch.empty_like(l1), torch.empty_like(r1), torch.empty(1, dtype=torch.int32, device="cuda")
    ds.cache_update(C, cu.i32(parent), cu.i32(new), cu.i32(table), l1, r1, t1, l2, r2, short, kp, vp, ws)
    want_t, want_l, want_r, _, copies = oc.update(parent, new, table, length, ref, page=page)
    assert copies and np.array_equal(t1.cpu().numpy(), want_t) and np.array_equal(r2.cpu().numpy(), want_r)
    for a, b in copies:
        k0[:, b], v0[:, b] = k0[:, a], v0[:, a]
    assert np.array_equal(kp.cpu().numpy(), k0) and np.array_equal(vp.cpu().numpy(), v0)
    t2, r3, live = torch.empty_like(t1), torch.empty_like(r2), torch.empty_like(short)
    ds.cache_compact(C, t1, l2, r2, t2, r3, live, kp, vp, ws)
    t_want, r_want, n_live, moves = oc.compact(want_t, want_l, want_r, page=page)
    for a, b in moves:
        k0[:, b], v0[:, b] = k0[:, a], v0[:, a]
    assert np.array_equal(t2.cpu().numpy(), t_want) and int(live) == n_live
    assert np.array_equal(kp.cpu().numpy(), k0) and np.array_equal(vp.cpu().numpy(), v0)
