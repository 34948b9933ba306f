"""Trees and tokens' own scales where they can go wrong on the GPU: pools past 2^32 bytes, page ids and rows out of range,
more requests than a workgroup has threads, larger max_new than any tree, queries that are not finite, no counts at
all, rows of other requests left as they were."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import tree as ot  # noqa: E402
from tests import cache_util as cu  # noqa: E402
from tests import tree_util as tu  # noqa: E402
from tests.test_gpu_cache import ds  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [2, 40])
def test_pools_past_32_bits(ds, rows):  # noqa: F811
    # 17000 pages of 270336 bytes a pool: the sequences lie in the last ones; append, both attentions and keep
    c = tu.make(1, "f8t", 256, 128, 16, 8, [rows, 3], [rows + 300, 20], poison=False)
    n_pages, few = 17000, c.k_pool.shape[1]
    C = ds.Cache.make(2, n_pages, 256, c.table.shape[1], 1, 16, 8, 128, cache="f8t")
    small = c.pools()
    pools = [torch.empty(C.k_shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert pools[0].numel() > 2 ** 32
    for p, s in zip(pools, small):
        p[:, n_pages - few:] = s
    table = np.where(c.table >= 0, c.table + n_pages - few, -1)
    ws = torch.empty(ds.cache_workspace_bytes(C, rows), dtype=torch.uint8, device="cuda")
    n, rs, le, ta = cu.i32(c.n_new), cu.i32(c.row_start), cu.i32(c.length), cu.i32(table)
    print("[gpu] pools past 2^32 bytes, rows", rows, flush=True)
    # the same calls on the small pools
    D, _ = tu.handle(ds, c, rows)
    parent, words, _ = tu.trees(2, c)
    mask = tu.words_i32(words)
    path, m = cu.i32([[0, 1], [1, 2]]), cu.i32([2, 2])
    results = []
    for H, (kp, vp), t in ((C, pools, ta), (D, small, cu.i32(c.table))):
        got = []
        ds.cache_append(H, 0, c.k.cuda(), c.v.cuda(), n, rs, rows, le, t, None, None, kp, vp)
        for tree in (False, True):
            out, lse = torch.zeros_like(c.q, device="cuda"), torch.zeros(c.q.shape[:2], device="cuda")
            if tree:
                ds.tree_attend(H, 0, c.q.cuda(), n, rs, rows, mask, None, le, t, kp, vp, None, None, out, lse, ws)
            else:
                ds.cache_attend(H, 0, c.q.cuda(), n, rs, rows, le, t, kp, vp, None, None, out, lse, ws)
            got += [out, lse]
        cut = torch.zeros(2, dtype=torch.int32, device="cuda")
        ds.tree_keep(H, path, m, n, rows, le, t, cut, kp, vp)
        results.append(got + [cut, kp[:, -few:].clone(), vp[:, -few:].clone()])
        torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", tu.TYPES)
@pytest.mark.parametrize("rows", [3, 40])
def test_page_ids_and_rows_out_of_range(ds, dtype, rows):  # noqa: F811
    # results of those rows are unspecified; the others are as ever, and nothing else is written
    c = tu.make(3, dtype, 16, 64, 4, 2, [rows, rows, 4, rows], [rows + 30, rows, 40, rows + 7], gap=1)
    _, words, depth = tu.trees(4, c)
    ref = tu.oracle_tree(c, words, depth)
    bad = tu.make(3, dtype, 16, 64, 4, 2, [rows, rows, 4, rows], [rows + 30, rows, 40, rows + 7], gap=1)
    bad.table[0, 0], bad.table[0, 1] = -7, 10 ** 9
    r0 = int(bad.row_start[1])
    bad.row_start[1], bad.row_start[3] = -5, len(bad.q) - 2  # rows before and behind the array
    out, lse = tu.gpu_tree(ds, bad, words, depth)
    good = np.arange(int(c.row_start[2]), int(c.row_start[2]) + 4)
    tol, _ = cu.attend_bound(dtype, ref[0][good], ref[1][good], ref[2][good], ref[3][good], 100)
    assert (np.abs(out[good].double().numpy() - ref[0][good]) <= tol).all()
    mine = np.zeros(len(out), bool)  # rows that a request has
    for b in range(4):
        for i in range(int(bad.n_new[b])):
            if 0 <= bad.row_start[b] + i < len(out):
                mine[bad.row_start[b] + i] = True
    assert not mine[r0 + rows - 1] and (out[~torch.from_numpy(mine)] == 77.0).all() and (lse[~torch.from_numpy(mine)] == 77.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f8t", "f32"])
@pytest.mark.parametrize("wide", [False, True])
def test_many_requests(ds, dtype, wide):  # noqa: F811
    i = np.arange(600)
    length = np.where(i % 9 == 5, 0, 6 + (i * 13) % 80)
    length[[3, 255, 256, 511]] = 1500, 90, 7, 1300
    n_new = np.where(i % 5 == 4, 0, np.minimum(length, 1 + i % 11))
    c = tu.make(5, dtype, 16, 64, 4, 1, n_new, length, width=150 if wide else None, poison=False)
    _, words, depth = tu.trees(6, c)
    tu.check(c, *tu.gpu_tree(ds, c, words, depth), tu.oracle_tree(c, words, depth))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f8t", 64), ("f8t", 256), ("f32", 64)])
@pytest.mark.parametrize("max_new", [12, 70, 3000])
def test_larger_max_new_than_any_tree(ds, dtype, D, max_new):  # noqa: F811
    c = tu.make(7, dtype, 16, D, 4, 2, [12, 0, 5], [70, 3, 200])
    parent, _, _ = tu.trees(8, c)
    words, depth = ot.mask(parent, c.n_new, c.row_start, len(parent), max_new, 2)
    tu.check(c, *tu.gpu_tree(ds, c, words, depth, window=2, max_new=max_new),
             tu.oracle_tree(c, words, depth, window=2))


def test_no_counts(ds):  # noqa: F811
    # n_new and row_start left out: max_new nodes a request, one behind the other
    n, B = 18, 3
    c = tu.make(9, "bf16", 16, 64, 4, 2, [n] * B, [n + 5, n, n + 100])
    parent, words, depth = tu.trees(10, c)
    C, ws = tu.handle(ds, c, n)
    mask, d = torch.zeros(n * B, 1, dtype=torch.int32, device="cuda"), torch.zeros(n * B, dtype=torch.int32, device="cuda")
    ds.tree_mask(cu.i32(parent), None, None, n, mask, d)
    assert np.array_equal(mask.cpu().numpy().view(np.uint32), words) and np.array_equal(d.cpu().numpy(), depth)
    out, lse = torch.zeros_like(c.q, device="cuda"), torch.zeros(c.q.shape[:2], device="cuda")
    kp, vp = c.pools()
    ds.tree_attend(C, 0, c.q.cuda(), None, None, n, mask, None, cu.i32(c.length), cu.i32(c.table), kp, vp, None, None, out,
                   lse, ws, scale=0.2)
    tu.check(c, out.cpu(), lse.cpu(), tu.oracle_tree(c, words, depth, scale=0.2))
    cut, path = torch.zeros(B, dtype=torch.int32, device="cuda"), cu.i32([[3, 17]] * B)
    ds.tree_keep(C, path, cu.i32([2, 1, 0]), None, n, cu.i32(c.length), cu.i32(c.table), cut, kp, vp)
    assert cut.cpu().tolist() == [7, 1, 100]


@pytest.mark.parametrize("dtype", tu.TYPES)
@pytest.mark.parametrize("rows", [4, 30])
def test_a_query_that_is_not_finite(ds, dtype, rows):  # noqa: F811
    c = tu.make(11, dtype, 16, 64, 4, 2, [rows], [rows + 40])
    _, words, depth = tu.trees(12, c)
    want = tu.oracle_tree(c, words, depth)
    c.q[1, 2, 7] = float("nan")
    out, lse = tu.gpu_tree(ds, c, words, depth)
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])
    other = torch.ones(rows, 4, dtype=torch.bool)
    other[1, 2] = False
    tol, _ = cu.attend_bound(dtype, want[0], want[1], want[2], want[3], rows + 40)
    assert (np.abs(out.double().numpy() - want[0]) <= tol)[other.numpy()].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8t"])
def test_scores_far_apart(ds, dtype):  # noqa: F811
    # an ancestor that takes all the weight, and one whose weight is nothing
    c = tu.make(13, dtype, 16, 64, 2, 2, [20], [60], q_std=20.0)
    _, words, depth = tu.trees(14, c)
    tu.check(c, *tu.gpu_tree(ds, c, words, depth), tu.oracle_tree(c, words, depth))


@pytest.mark.parametrize("dtype", ["bf16", "f8t"])
def test_one_request_and_one_node(ds, dtype):  # noqa: F811
    for length in (1, 2, 17, 300):
        c = tu.make(15, dtype, 16, 64, 1, 1, [1], [length])
        words, depth = ot.mask([-1], [1], [0], 1, 1)
        tu.check(c, *tu.gpu_tree(ds, c, words, depth), tu.oracle_tree(c, words, depth))


def test_results_repeat_bit_for_bit(ds):  # noqa: F811
    for dtype in tu.TYPES:
        c = tu.make(16, dtype, 16, 64, 8, 2, [60, 20, 7], [900, 300, 2000], width=300)
        _, words, depth = tu.trees(17, c)
        a, b = (tu.gpu_tree(ds, c, words, depth) for _ in range(2))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["bf16", "f8t"])
@pytest.mark.parametrize("max_pages", [96, 1 << 16])
def test_longest_requests_first(ds, dtype, max_pages):  # noqa: F811
    # whole segments taken in the order of their lengths, many of them equal, some of requests without new tokens; and rows
    # of the page table as wide as they may be (2^24 tokens)
    B, page = (256, 16) if max_pages == 96 else (130, 256)
    i = np.arange(B)
    length = np.where(i % 5 == 0, 40, 20 + (i * 29) % 90)
    length[[7, B - 1]] = 1500, 1400
    c = tu.make(18, dtype, page, 64, 16, 8 if B == 130 else 4, np.where(i % 6 == 1, 0, 1 + i % 3), length, poison=False,
                width=max_pages)
    _, words, depth = tu.trees(19, c)
    tu.check(c, *tu.gpu_attend(ds, c), cu.oracle_attend(c))
    tu.check(c, *tu.gpu_tree(ds, c, words, depth), tu.oracle_tree(c, words, depth))
