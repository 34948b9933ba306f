"""Attention over caches that hold values which are not finite: in places that weigh nothing,
and in places that no row sees."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import cache_util as cu  # noqa: E402
from tests.test_gpu_cache import check_attend, ds, gpu_attend, handle  # noqa: E402,F401

pytestmark = pytest.mark.gpu

PAGE = 16


def put(c, b, j, key=None, value=None):
    """Position j of request b: its key and its value, all coordinates."""
    p, off = c.table[b][j // PAGE], j % PAGE
    if key is not None:
        c.k_pool[:, p, :, off] = key
    if value is not None:
        c.v_pool[:, p, :, off // 8, :, off % 8] = value


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,rows", [(2, 6), (24, 6), (2, 40), (1, 150)])
@pytest.mark.parametrize("width", [None, 100])
def test_rows_whose_weights_are_all_zero(ds, dtype, G, rows, width):  # noqa: F811
    # every score of request 0 is -inf: its rows get 0 and -inf, also where a value is NaN (next to the diagonal, where
    # some rows do not see it, and far from it, where all do); request 1 is as ever
    c = cu.make(60, dtype, PAGE, 64, 2 * G, 2, [rows, 3], [170 + rows, 40], width=width)
    c.q[:rows] = c.q[:rows].abs() + 0.5
    ref = cu.oracle_attend(c)
    for j in range(170 + rows):
        put(c, 0, j, key=-float("inf"))
    for j in (3, 66, 170, 170 + rows - 1):
        put(c, 0, j, value=float("nan"))
    out, lse = gpu_attend(ds, c)
    assert torch.isneginf(lse[:rows]).all()
    assert (out[:rows] == 0).all(), f"{torch.isnan(out[:rows]).sum()} NaN of {out[:rows].numel()}"
    want, want_lse, mag, span = (x[rows:] for x in ref)
    tol, tol_lse = cu.attend_bound(dtype, want, want_lse, mag, span, 40)
    assert (np.abs(out[rows:].double().numpy() - want) <= tol).all()
    assert (np.abs(lse[rows:].double().numpy() - want_lse) <= tol_lse).all()


def timed(ds, C, q, n, length, table, kp, vp, T):  # noqa: F811
    """Results and the time of a call in ms, the smallest of a few."""
    ws = torch.empty(ds.cache_workspace_bytes(C, T), dtype=torch.uint8, device="cuda")
    one = torch.ones(C.Hkv, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    times = []
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        ds.cache_attend(C, 0, q, n, None, T, length, table, kp, vp, one, one, out, lse, ws)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return out, lse, min(times)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
@pytest.mark.parametrize("T,G", [(1, 4), (9, 4), (40, 8)])
@pytest.mark.parametrize("wide", [False, True])
def test_what_no_row_sees_costs_little(ds, dtype, T, G, wide):  # noqa: F811
    # NaN, as a pool's unused offsets may hold, behind the end of every sequence: the results are bit for bit those
    # over zeros there, in about the same time (with a walk over the keys that the rows do see it is ten times as long)
    B, keys, Hkv, D = 8, 4000, 2, 128
    pages = -(-keys // PAGE)
    width = 4 * pages if wide else pages
    C = ds.Cache.make(B, B * pages, PAGE, width, 1, G * Hkv, Hkv, D, q="f32" if dtype == "f32" else "bf16", cache=dtype)
    gen = torch.Generator(device="cuda").manual_seed(61)
    pools = [torch.randn(s, device="cuda", generator=gen) for s in (C.k_shape, C.v_shape)]
    length = cu.i32([keys - 1 - b for b in range(B)])
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[:, :pages] = torch.arange(B * pages, device="cuda", dtype=torch.int32).view(B, pages)
    q = torch.randn((B * T, G * Hkv, D), device="cuda", generator=gen).to(C.data_type)
    n = cu.i32([T] * B)
    got = []
    for hidden in (0.0, float("nan")):
        for b in range(B):
            for j in range(keys - 1 - b, pages * PAGE):
                p, off = b * pages + j // PAGE, j % PAGE
                pools[0][0, p, :, off] = hidden
                pools[1][0, p, :, off // 8, :, off % 8] = hidden
        got.append(timed(ds, C, q, n, length, table, *(x.to(C.cache_type) for x in pools), T))
    print(f"[gpu] {dtype} T={T} G={G}: {1e3 * got[0][2]:.0f} us, with NaN behind the sequences {1e3 * got[1][2]:.0f}")
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[1][2] < 1.5 * got[0][2] + 0.01


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
@pytest.mark.parametrize("rows,G", [(7, 2), (20, 3)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 11), (False, 0), (False, 9)])
@pytest.mark.parametrize("width", [None, 100])
def test_a_value_reaches_the_rows_that_see_it(ds, dtype, rows, G, causal, window, width):  # noqa: F811
    # request b's value of coordinate 7 at its b-th last position but one is NaN; all other results are as without it
    B, length = 40, [90 + 3 * b for b in range(40)]
    c = cu.make(62, dtype, PAGE, 64, G, 1, [rows] * B, length, width=width)
    ref = gpu_attend(ds, c, causal=causal, window=window)
    place = [length[b] - 1 - b for b in range(B)]
    for b, j in enumerate(place):
        p, off = c.table[b][j // PAGE], j % PAGE
        c.v_pool[0, p, 0, off // 8, 7, off % 8] = float("nan")
    out, lse = gpu_attend(ds, c, causal=causal, window=window)
    sees = np.zeros((B, rows), bool)
    for b, j in enumerate(place):
        for i in range(rows):
            pos = length[b] - rows + i
            sees[b, i] = (not causal or j <= pos) and (window == 0 or j > pos - window)
    assert sees.any() and not sees.all() if causal or window else sees.all()
    want = ref[0].clone()
    want.view(B, rows, G, 64)[torch.from_numpy(sees)[..., None].expand(-1, -1, G)] = \
        want.view(B, rows, G, 64)[torch.from_numpy(sees)[..., None].expand(-1, -1, G)].index_fill(1, torch.tensor([7]), float("nan"))
    torch.testing.assert_close(out, want, rtol=0, atol=0, equal_nan=True)
    assert torch.equal(lse, ref[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
@pytest.mark.parametrize("rows,G", [(5, 3), (40, 2)])
@pytest.mark.parametrize("width", [None, 100])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_a_query_row_stays_by_itself(ds, dtype, rows, G, width, bad):  # noqa: F811
    # one head of one row of q is not finite: that result is NaN (or empty), all others are as without it
    c = cu.make(63, dtype, PAGE, 64, 2 * G, 2, [rows, 2], [300 + rows, 50], width=width)
    ref = gpu_attend(ds, c)
    c.q[rows // 2, 1] = float(bad)
    out, lse = gpu_attend(ds, c)
    keep = torch.ones(out.shape[:2], dtype=torch.bool)
    keep[rows // 2, 1] = False
    assert torch.equal(out[keep], ref[0][keep]) and torch.equal(lse[keep], ref[1][keep])
    assert torch.isnan(out[rows // 2, 1]).all()
