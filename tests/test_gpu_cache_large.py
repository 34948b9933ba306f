"""Pools whose offsets pass 32 bits, in bytes and in elements: the calls on pages at their far
end.  Also the attention kernels that read with the streaming policy, which they do where a
call may read more than the last-level cache holds."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache as oc  # noqa: E402
from tests import cache_util as cu  # noqa: E402
from tests.test_gpu_cache import bits, check_attend, ds  # noqa: E402,F401

pytestmark = pytest.mark.gpu

PAGE, HKV, D = 16, 2, 128
N_PAGES = (1 << 20) + 600  # of 4096 elements: beyond 2^32


@pytest.fixture(scope="module", params=["bf16", "f8", "f32"])
def pools(request, ds):  # noqa: F811
    C = ds.Cache.make(1, N_PAGES, PAGE, 1, 1, HKV, HKV, D, q="f32" if request.param == "f32" else "bf16", cache=request.param)
    k, v = (torch.empty(s, dtype=C.cache_type, device="cuda") for s in (C.k_shape, C.v_shape))
    yield request.param, k, v
    del k, v
    torch.cuda.empty_cache()


def far_ids(n, seed=0):
    """n page ids: the last one, the ones around 2^20, others beyond it, and a few at the pool's start."""
    rng = np.random.default_rng(seed)
    ids = np.concatenate([[N_PAGES - 1, (1 << 20) - 1, 1 << 20, 0, 3], (1 << 20) + 1 + rng.permutation(500)])
    return rng.permutation(ids[:n]) if n > 5 else ids[:n]


def place(c, k, v):
    """The case's pages, at far ids of the large pools."""
    ids = far_ids(c.k_pool.shape[1])
    at = torch.from_numpy(ids).cuda()
    for pool, x in ((k, c.k_pool), (v, c.v_pool)):
        raw = pool.view(torch.uint8) if c.dtype == "f8" else pool
        raw[0, at] = (x.view(torch.uint8) if c.dtype == "f8" else x)[0].cuda()
    return np.where(c.table >= 0, ids[c.table], -1), ids


@pytest.mark.parametrize("G,n_new", [(1, [1, 3, 2]), (8, [1, 2, 1]), (3, [20, 1, 9]), (8, [40, 9, 17])])
@pytest.mark.parametrize("width", [None, 11000])  # 11000: the keys are dealt out, and read with the streaming policy
@pytest.mark.parametrize("window", [0, 50])
def test_attend_at_the_far_end(ds, pools, G, n_new, width, window):  # noqa: F811
    dtype, k, v = pools
    c = cu.make(100, dtype, PAGE, D, G * HKV, HKV, n_new, [700, 333, 41], width=width)
    table, _ = place(c, k, v)
    T = max(n_new)
    C = ds.Cache.make(3, N_PAGES, PAGE, table.shape[1], 1, G * HKV, HKV, D, q="f32" if dtype == "f32" else "bf16", cache=dtype)
    ws = torch.empty(ds.cache_workspace_bytes(C, T), dtype=torch.uint8, device="cuda").fill_(255)
    q = c.q.cuda()
    out, lse = torch.full_like(q, 77.0), torch.full(q.shape[:2], 77.0, device="cuda")
    print(f"[gpu] attend {dtype} G={G} {n_new} in {N_PAGES} pages, rows of {table.shape[1]}, window {window}", flush=True)
    ds.cache_attend(C, 0, q, cu.i32(c.n_new), cu.i32(c.row_start), T, cu.i32(c.length), cu.i32(table), k, v,
                    c.k_scale.cuda(), c.v_scale.cuda(), out, lse, ws, window=window)
    check_attend(c, out.cpu(), lse.cpu(), cu.oracle_attend(c, window=window))


def test_append_at_the_far_end(ds, pools):  # noqa: F811
    dtype, k, v = pools
    c = cu.make(101, dtype, PAGE, D, HKV, HKV, [17, 1, 33], [40, 9, 70], gap=1, poison=False)
    table, ids = place(c, k, v)
    C = ds.Cache.make(3, N_PAGES, PAGE, table.shape[1], 1, HKV, HKV, D, q="f32" if dtype == "f32" else "bf16", cache=dtype)
    print(f"[gpu] append {dtype} in {N_PAGES} pages", flush=True)
    ds.cache_append(C, 0, c.k.cuda(), c.v.cuda(), cu.i32(c.n_new), cu.i32(c.row_start), 33, cu.i32(c.length), cu.i32(table),
                    c.k_scale.cuda(), c.v_scale.cuda(), k, v)
    kk, vv = c.k.double().numpy(), c.v.double().numpy()
    if dtype == "f8":
        kk, vv = (oc.round_f8((x.astype(np.float32) / s.numpy()[:, None]).astype(np.float64))
                  for x, s in ((kk, c.k_scale), (vv, c.v_scale)))
    want = oc.append(c.k_pool.double().numpy(), c.v_pool.double().numpy(), kk, vv, c.n_new, c.row_start, c.length, c.table,
                     layer=0, page=PAGE)
    at = torch.from_numpy(ids).cuda()
    for pool, ref in zip((k, v), want):
        got = (pool.view(torch.uint8)[:, at].view(pool.dtype) if dtype == "f8" else pool[:, at]).cpu().double().numpy()
        np.testing.assert_array_equal(got, ref)


def test_pages_are_copied_and_moved_at_the_far_end(ds, pools):  # noqa: F811
    # all low ids but a few are held by nobody and marked as in use, so that copies and new pages go to far ids; then a
    # compaction brings the far pages of a pool without such marks to the front
    dtype, k, v = pools
    C = ds.Cache.make(4, N_PAGES, PAGE, 4, 1, HKV, HKV, D, q="f32" if dtype == "f32" else "bf16", cache=dtype)
    ws = torch.empty(ds.cache_workspace_bytes(C, 1), dtype=torch.uint8, device="cuda").fill_(255)
    c = cu.make(102, dtype, PAGE, D, HKV, HKV, [1, 1], [40, 20], poison=False, spare=0)
    table, ids = place(c, k, v)
    full = np.full((4, 4), -1)
    full[:2, :3] = table
    length = np.array([40, 20, 0, 0])
    ref = np.ones(N_PAGES, np.int64)
    ref[(1 << 20) + 520:] = 0
    ref[N_PAGES - 1] = 1
    ref[ids] = 0
    ref[full[full >= 0]] += 1
    to = [torch.full((4, 4), 99, dtype=torch.int32, device="cuda"), cu.i32([99] * 4), cu.i32(np.full(N_PAGES, 99)), cu.i32([99])]
    print(f"[gpu] update {dtype} in {N_PAGES} pages", flush=True)
    parent, new = np.array([0, 1, 0, 1]), np.array([41, 20, 45, 36])
    want = oc.update(parent, new, full, length, ref, page=PAGE)
    assert len(want[4]) == 3 and all(b >= 1 << 20 for _, b in want[4])

    def page(pool, p):
        return bits(pool[0, p:p + 1])

    before = [[page(x, a).copy() for a, _ in want[4]] for x in (k, v)]
    ds.cache_update(C, cu.i32(parent), cu.i32(new), cu.i32(full), cu.i32(length), cu.i32(ref), *to, k, v, ws)
    for got, x in zip(to, want):
        np.testing.assert_array_equal(got.cpu().numpy(), x)
    for x, old in zip((k, v), before):
        for (_, b), y in zip(want[4], old):
            np.testing.assert_array_equal(page(x, b), y)
    table, length = want[:2]
    ref = np.zeros(N_PAGES, np.int64)
    np.add.at(ref, table[table >= 0], 1)
    packed = oc.compact(table, length, ref, page=PAGE)
    assert packed[2] < 20 and any(a >= 1 << 20 for a, _ in packed[3])
    before = [[page(x, a).copy() for a, _ in packed[3]] for x in (k, v)]
    to = [to[0].fill_(99), to[2].fill_(99), to[3].fill_(99)]
    ds.cache_compact(C, cu.i32(table), cu.i32(length), cu.i32(ref), *to, k, v, ws)
    for got, x in zip(to, packed):
        np.testing.assert_array_equal(got.cpu().numpy(), x)
    for x, old in zip((k, v), before):
        for (_, b), y in zip(packed[3], old):
            np.testing.assert_array_equal(page(x, b), y)
