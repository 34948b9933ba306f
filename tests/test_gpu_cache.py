"""The paged cache on the GPU against the float64 oracle, through the C ABI:
attention (types, head layouts, pages, lengths from zero, masks that leave rows
empty, NaN in places that are not visible), appended tokens bit for bit, the
bookkeeping of pages exactly, and whole cycles of them."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache as oc  # noqa: E402
from tests import cache_util as cu  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from draft_sampling_verification_markov_amd import dspark
    dspark.load()
    return dspark


def handle(ds, c: cu.Case, max_new, layers=1):
    B, width = c.table.shape
    C = ds.Cache.make(B, c.k_pool.shape[1], c.page, width, layers, c.q.shape[1], c.k_pool.shape[2], c.q.shape[2],
                      q="f32" if c.dtype == "f32" else "bf16", cache=c.dtype)
    return C, torch.empty(ds.cache_workspace_bytes(C, max_new), dtype=torch.uint8, device="cuda").fill_(255)


def gpu_attend(ds, c: cu.Case, layer=0, scale=None, causal=True, window=0, with_lse=True, max_new=None, layers=1):
    max_new = max(1, int(c.n_new.max())) if max_new is None else max_new
    C, ws = handle(ds, c, max_new, layers)
    q = c.q.cuda()
    out = torch.full_like(q, 77.0)
    lse = torch.full(q.shape[:2], 77.0, device="cuda") if with_lse else None
    print(f"[gpu] attend {c.dtype} page={c.page} D={q.shape[2]} Hq={q.shape[1]} Hkv={C.Hkv} n_new={c.n_new.tolist()[:6]} "
          f"length={c.length.tolist()[:6]} causal={causal} window={window}", flush=True)
    ds.cache_attend(C, layer, q, cu.i32(c.n_new), cu.i32(c.row_start), max_new, cu.i32(c.length), cu.i32(c.table),
                    c.k_pool.cuda(), c.v_pool.cuda(), c.k_scale.cuda(), c.v_scale.cuda(), out, lse, ws, scale=scale,
                    causal=causal, window=window)
    torch.cuda.synchronize()
    return out.cpu(), None if lse is None else lse.cpu()


def check_attend(c: cu.Case, out, lse, ref):
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


RAGGED = ([1, 5, 0, 3, 2], [1, 37, 20, 3, 130])


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 8, 2), (256, 6, 2), (128, 5, 1), (64, 12, 1)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_attend_ragged(ds, dtype, D, Hq, Hkv, page):
    c = cu.make(1, dtype, page, D, Hq, Hkv, *RAGGED, gap=1)
    check_attend(c, *gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 16), (True, 33), (False, 0), (False, 7), (True, 2000)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("G", [2, 8])
def test_attend_masks(ds, dtype, causal, window, wide, G):
    c = cu.make(2, dtype, 32, 128, 2 * G, 2, [9, 1, 17, 0], [100, 260, 17, 40], width=200 if wide else None)
    check_attend(c, *gpu_attend(ds, c, causal=causal, window=window), cu.oracle_attend(c, causal=causal, window=window))


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
def test_attend_rows_that_see_nothing(ds, dtype):
    # more new rows than cached tokens: the first rows lie before position 0; and a request without tokens
    c = cu.make(3, dtype, 16, 64, 2, 1, [5, 3, 4], [2, 0, 4])
    ref = cu.oracle_attend(c)
    assert np.isneginf(ref[1][:3]).all() and np.isneginf(ref[1][5:8]).all()
    out, lse = gpu_attend(ds, c)
    check_attend(c, out, lse, ref)
    assert (out[:3] == 0).all() and (out[5:8] == 0).all()
    c = cu.make(4, dtype, 16, 64, 2, 1, [3, 2], [0, 40])
    check_attend(c, *gpu_attend(ds, c, causal=False), cu.oracle_attend(c, causal=False))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 257])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_every_length(ds, dtype, n):
    c = cu.make(10 + n, dtype, 16, 64, 4, 2, [1, 2, min(n, 40)], [n, n + 1, n])
    check_attend(c, *gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 16), ("bf16", 128, 64), ("f8", 128, 128), ("f32", 64, 32),
                                          ("bf16", 256, 16), ("f8", 256, 32), ("f32", 256, 16), ("f32", 128, 64)])
@pytest.mark.parametrize("rows,G", [(1, 3), (17, 4), (40, 2), (150, 2), (301, 1)])
@pytest.mark.parametrize("wide", [False, True])
def test_attend_row_counts(ds, dtype, D, page, rows, G, wide):
    # every arrangement of rows: a few, some row blocks, several row tiles, over contexts that need several key tiles;
    # with a wide page table the keys are dealt out over the chip and joined
    c = cu.make(20 + rows, dtype, page, D, 2 * G, 2, [rows, 1, rows // 2], [rows + 333, 700, rows // 2],
                width=5000 // page if wide else None)
    check_attend(c, *gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f8", 128), ("f32", 64), ("f32", 256)])
@pytest.mark.parametrize("n_new,length,Hkv", [([600], [700], 1), ([257, 0, 90, 300, 129], [257, 8, 95, 310, 129], 1),
                                              ([150, 33], [200, 700], 3)])
def test_attend_row_tiles_of_few_heads(ds, dtype, D, n_new, length, Hkv):
    # many row tiles of fewer (request, head) pairs than the chip's parts, and of numbers that these do not divide
    c = cu.make(33, dtype, 32, D, 4 * Hkv, Hkv, n_new, length, gap=1)
    check_attend(c, *gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("dtype", ["bf16", "f8", "f32"])
@pytest.mark.parametrize("rows", [1, 9])
def test_attend_many_requests_dealt(ds, dtype, rows):
    # more requests than a workgroup has threads, ragged, some without new tokens or without any, in a wide page table
    i = np.arange(620)
    length = np.where(i % 7 == 3, 0, 1 + (i * 37) % 90)
    length[[0, 255, 256, 511, 619]] = 2100, 70, 1, 0, 1300
    n_new = np.where(i % 5 == 4, 0, np.minimum(1 + i % rows, np.maximum(length, 1)))
    c = cu.make(34, dtype, 32, 64, 4, 1, n_new, length, width=100, poison=False)
    check_attend(c, *gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("dtype", ["bf16", "f8", "f32"])
@pytest.mark.parametrize("B,Hkv", [(70, 8), (256, 3), (257, 2)])
def test_attend_many_ragged_segments(ds, dtype, B, Hkv):
    # more segments than run at once, of unequal and of equal lengths, over more keys than a few
    i = np.arange(B)
    length = 30 + (i * 53) % 200
    length[[1, 5, B - 1]] = 1100, 1100, 900
    length[[0, 7]] = 0, 0
    n_new = np.where(i % 4 == 2, 0, np.minimum(2 + (i * 5) % 8, length))
    n_new[1] = 40
    c = cu.make(36, dtype, 32, 64, 2 * Hkv, Hkv, n_new, length, width=40, poison=False)
    check_attend(c, *gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("dtype,D,n", [("f32", 256, 530), ("bf16", 64, 4200)])
def test_attend_many_row_tiles_dealt(ds, dtype, D, n):
    # more row tiles of a request than a workgroup has threads; the page table's width has the keys dealt
    c = cu.make(35, dtype, 64, D, 8, 1, [n], [n + 70], width=6000 // 64, poison=False)
    check_attend(c, *gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("causal", [True, False])
def test_attend_window_of_any_size(ds, causal):
    # fewer cached tokens than rows, and windows up to the largest integer: the same as none
    c = cu.make(31, "bf16", 16, 64, 4, 2, [9, 2], [5, 40])
    ref = cu.oracle_attend(c, causal=causal)
    for window in (1 << 20, 2**31 - 1):
        check_attend(c, *gpu_attend(ds, c, causal=causal, window=window), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
@pytest.mark.parametrize("G", [2, 20])
def test_attend_scale_of_almost_nothing(ds, dtype, G):
    # the smallest softmax scale (with an e4m3 key scale its product is 0 in fp32): what a row sees weighs the same,
    # what it does not see still nothing
    c = cu.make(32, dtype, 16, 64, 2 * G, 2, [3, 1], [37, 5])
    c.k_scale.fill_(1e-3)
    scale = float(np.float32(1e-45))
    check_attend(c, *gpu_attend(ds, c, scale=scale), cu.oracle_attend(c, scale=scale))


def test_attend_long_context(ds):
    c = cu.make(30, "bf16", 64, 64, 2, 1, [1, 2], [20000, 9], poison=False)
    check_attend(c, *gpu_attend(ds, c), cu.oracle_attend(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("G", [2, 24])
def test_attend_ignores_what_a_row_does_not_see(ds, dtype, bad, G):
    # the keys and values of later new tokens (causal) and before the window hold NaN or infinities: the rows that
    # do not see them stay exact, the rows that do become NaN
    page, D = 16, 64
    if dtype == "f8" and bad == "inf":
        bad = "nan"  # the type has no infinities
    c = cu.make(5, dtype, page, D, G, 1, [6], [75])
    clean_k, clean_v = c.k_pool.clone(), c.v_pool.clone()
    for j in (60, 72):  # 60: before the window of rows 70.. of width 10; 72: seen from row 72 on
        p, off = c.table[0][j // page], j % page
        c.k_pool[0, p, :, off] = float(bad)
        c.v_pool[0, p, :, off // 8, :, off % 8] = float(bad)
    out, lse = gpu_attend(ds, c, window=10)
    d = cu.Case(**{**vars(c), "k_pool": clean_k, "v_pool": clean_v})
    ref = cu.oracle_attend(d, window=10)
    rows = [1, 2]  # positions 70, 71 see neither 60 nor 72
    want, want_lse, mag, span = (x[rows] for x in ref)
    tol, tol_lse = cu.attend_bound(dtype, want, want_lse, mag, span, 75)
    assert (np.abs(out[rows].double().numpy() - want) <= tol).all()
    assert (np.abs(lse[rows].double().numpy() - want_lse) <= tol_lse).all()
    if bad == "nan":
        assert torch.isnan(out[0]).all() and torch.isnan(out[3:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
@pytest.mark.parametrize("G,rows", [(2, 6), (24, 6), (2, 40)])
def test_attend_nan_that_every_row_sees(ds, dtype, G, rows):
    # next to the diagonal, where some keys are hidden, and far from it; keys in one part and dealt out
    page, D = 16, 64
    for j, width in ((66, None), (3, None), (66, 100), (3, 100)):
        c = cu.make(5, dtype, page, D, G, 1, [rows], [70 + rows - 1], width=width)
        p, off = c.table[0][j // page], j % page
        c.v_pool[0, p, :, off // 8, 5, off % 8] = float("nan")
        out, lse = gpu_attend(ds, c)
        assert torch.isnan(out[:, :, 5]).all() and not torch.isnan(lse).any()
        assert not torch.isnan(torch.cat([out[:, :, :5], out[:, :, 6:]], 2)).any()


def test_attend_layers_strides_and_no_lse(ds):
    # the second of three layers; q and out are column slices of wider arrays
    page, D, Hq, Hkv = 16, 64, 4, 2
    c = cu.make(6, "bf16", page, D, Hq, Hkv, [3, 1], [40, 20], layers=3)
    C, ws = handle(ds, c, 3, 3)
    wide = torch.zeros(4, 3 * Hq, D, dtype=torch.bfloat16, device="cuda")
    wide[:, Hq:2 * Hq] = c.q.cuda()
    res = torch.full((4, 2 * Hq, D), 77.0, dtype=torch.bfloat16, device="cuda")
    ds.cache_attend(C, 1, wide[:, Hq:2 * Hq], cu.i32(c.n_new), cu.i32(c.row_start), 3, cu.i32(c.length), cu.i32(c.table),
                    c.k_pool.cuda(), c.v_pool.cuda(), None, None, res[:, Hq:], None, ws, scale=0.3)
    check_attend(c, res[:, Hq:].cpu(), None, cu.oracle_attend(c, layer=1, scale=0.3))
    assert (res[:, :Hq] == 77.0).all()


def test_attend_padded_rows_without_arrays(ds):
    # n_new and row_start NULL: max_new rows for every request, one after the other
    c = cu.make(7, "bf16", 32, 128, 8, 2, [4, 4, 4], [4, 33, 70])
    C, ws = handle(ds, c, 4)
    out = torch.zeros_like(c.q, device="cuda")
    lse = torch.zeros(c.q.shape[:2], device="cuda")
    ds.cache_attend(C, 0, c.q.cuda(), None, None, 4, cu.i32(c.length), cu.i32(c.table), c.k_pool.cuda(),
                    c.v_pool.cuda(), None, None, out, lse, ws)
    check_attend(c, out.cpu(), lse.cpu(), cu.oracle_attend(c))


def test_attend_bad_ids_and_counts_stay_in_bounds(ds):
    # ids outside the pool, lengths past the table, rows past the array: no fault, and the sound request is exact
    c = cu.make(8, "bf16", 16, 64, 2, 1, [2, 2], [40, 40])
    good = cu.oracle_attend(c)
    c.table[1] = [-5, 1 << 30, 7000]
    big = cu.Case(**{**vars(c), "length": np.array([40, 1 << 20]), "n_new": np.array([2, 999]),
                     "row_start": np.array([0, 2])})
    out, lse = gpu_attend(ds, big, max_new=2)
    out, lse = out[:2], lse[:2]
    check_attend(cu.Case(**{**vars(c), "length": c.length[:1]}), out, lse, tuple(x[:2] for x in good))
    big.row_start = np.array([0, 1 << 20])
    gpu_attend(ds, big, max_new=2)
    big.row_start = np.array([0, -7])
    gpu_attend(ds, big, max_new=2)


def test_attend_is_reproducible_and_stream_ordered(ds):
    c = cu.make(9, "bf16", 16, 128, 8, 2, [17] * 6, [500, 17, 900, 64, 65, 300])
    a = gpu_attend(ds, c)
    b = gpu_attend(ds, c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    C, ws = handle(ds, c, 17)
    side = torch.cuda.Stream()
    args = [c.q.cuda(), cu.i32(c.n_new), cu.i32(c.row_start)]
    more = [cu.i32(c.length), cu.i32(c.table), c.k_pool.cuda(), c.v_pool.cuda(), None, None]
    out, lse = torch.empty_like(args[0]), torch.empty(args[0].shape[:2], device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    ds.cache_attend(C, 0, *args, 17, *more, out, lse, ws, stream=side)
    side.synchronize()
    assert torch.equal(out.cpu(), a[0]) and torch.equal(lse.cpu(), a[1])


def bits(t):
    t = t.cpu().contiguous()
    return t.view(torch.uint8).numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f8"])
@pytest.mark.parametrize("D,page,n_new,length", [
    (64, 16, [1], [1]), (128, 16, [1, 1, 1], [8, 9, 16]), (128, 32, [17, 0, 5, 33], [17, 9, 70, 100]),
    (256, 256, [40, 1], [300, 257]), (64, 64, [6, 9], [4, 9]), (128, 16, [200], [333])])
def test_append(ds, dtype, D, page, n_new, length):
    Hkv = 3
    c = cu.make(40, dtype, page, D, Hkv, Hkv, n_new, length, layers=2, gap=1, poison=False)
    C, _ = handle(ds, c, max(n_new), 2)
    kv = torch.cat([c.v, c.k], 1).cuda()  # strided rows
    if dtype == "f8":
        kv[:, :, 0] *= 1e4  # past 448
        c.k, c.v = kv[:, Hkv:].cpu(), kv[:, :Hkv].cpu()
    kp, vp = c.k_pool.cuda(), c.v_pool.cuda()
    print(f"[gpu] append {dtype} D={D} page={page} n_new={n_new} length={length}", flush=True)
    ds.cache_append(C, 1, kv[:, Hkv:], kv[:, :Hkv], cu.i32(c.n_new), cu.i32(c.row_start), max(n_new), cu.i32(c.length),
                    cu.i32(c.table), c.k_scale.cuda(), c.v_scale.cuda(), kp, vp)
    k, v = c.k.double().numpy(), c.v.double().numpy()
    if dtype == "f8":
        # the quotient is an fp32 quotient, then rounded to e4m3
        k, v = (oc.round_f8((x.astype(np.float32) / s.numpy()[:, None]).astype(np.float64))
                for x, s in ((k, c.k_scale), (v, c.v_scale)))
    want_k, want_v = oc.append(c.k_pool.double().numpy(), c.v_pool.double().numpy(), k, v, c.n_new, c.row_start,
                               c.length, c.table, layer=1, page=page)
    np.testing.assert_array_equal(kp.cpu().double().numpy(), want_k)
    np.testing.assert_array_equal(vp.cpu().double().numpy(), want_v)


def test_append_f8_rounds_every_value_as_defined(ds):
    # all bf16 values, as keys of one-token requests with scale 1: nearest e4m3, ties to even, saturated, NaN kept
    D, B = 256, 256
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(B, 1, D)
    C = ds.Cache.make(B, B, 16, 1, 1, 1, 1, D, cache="f8")
    kp = torch.zeros(C.k_shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vp = torch.zeros(C.v_shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    one = torch.ones(1, device="cuda")
    ds.cache_append(C, 0, x.cuda(), x.cuda(), None, None, 1, cu.i32(np.full(B, 3)), cu.i32(np.arange(B)[:, None]), one, one,
                    kp, vp)
    want = oc.round_f8(x.double().numpy()[:, 0])
    np.testing.assert_array_equal(kp.cpu()[0, :, 0, 2].double().numpy(), want)
    np.testing.assert_array_equal(vp.cpu()[0, :, 0, 0, :, 2].double().numpy(), want)


@pytest.mark.parametrize("scale", [0.02, 1.0 / 3.0, 0.03999999, 7.7e-3, 1e3, 3e-20, 2e-39])
def test_append_f8_quotients(ds, scale):
    # all bf16 values over several scales: the e4m3 value of the rounded fp32 quotient, bit for bit
    D, B = 256, 256
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(B, 1, D)
    C = ds.Cache.make(B, B, 16, 1, 1, 1, 1, D, cache="f8")
    kp = torch.zeros(C.k_shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vp = torch.zeros(C.v_shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((1,), scale, device="cuda")
    ds.cache_append(C, 0, x.cuda(), x.cuda(), None, None, 1, cu.i32(np.full(B, 6)), cu.i32(np.arange(B)[:, None]), s, s,
                    kp, vp)
    with np.errstate(over="ignore", invalid="ignore"):
        q = x.float().numpy()[:, 0] / np.float32(scale)
    want = oc.round_f8(q.astype(np.float64))
    np.testing.assert_array_equal(kp.cpu()[0, :, 0, 5].double().numpy(), want)
    np.testing.assert_array_equal(vp.cpu()[0, :, 0, 0, :, 5].double().numpy(), want)


def test_append_leaves_out_bad_ids(ds):
    c = cu.make(41, "bf16", 16, 64, 1, 1, [3, 3], [20, 20], poison=False)
    c.table[1] = [c.k_pool.shape[1], -1]
    C, _ = handle(ds, c, 3)
    kp, vp = c.k_pool.cuda(), c.v_pool.cuda()
    ds.cache_append(C, 0, c.k.cuda(), c.v.cuda(), cu.i32(c.n_new), cu.i32(c.row_start), 3, cu.i32(c.length),
                    cu.i32(c.table), None, None, kp, vp)
    k, v = oc.append(c.k_pool.double().numpy(), c.v_pool.double().numpy(), c.k.double().numpy(), c.v.double().numpy(),
                     c.n_new, c.row_start, c.length, c.table, layer=0, page=16)
    np.testing.assert_array_equal(kp.cpu().double().numpy(), k)
    np.testing.assert_array_equal(vp.cpu().double().numpy(), v)


class Pages:
    """A pool with its tables on the GPU, and the same in numpy."""

    def __init__(self, ds, B, n_pages, page, width, layers=1, Hkv=1, D=64, cache="bf16", seed=0):
        self.ds, self.page = ds, page
        self.C = ds.Cache.make(B, n_pages, page, width, layers, Hkv, Hkv, D, q="f32" if cache == "f32" else "bf16",
                               cache=cache)
        g = torch.Generator().manual_seed(seed)
        t = self.C.cache_type
        self.k = torch.randn(self.C.k_shape, generator=g).to(t).cuda()
        self.v = torch.randn(self.C.v_shape, generator=g).to(t).cuda()
        self.ws = torch.empty(ds.cache_workspace_bytes(self.C, 1), dtype=torch.uint8, device="cuda").fill_(255)
        self.table = np.full((B, width), -1, np.int64)
        self.length = np.zeros(B, np.int64)
        self.ref = np.zeros(n_pages, np.int64)

    def pools_with(self, moves):
        k, v = bits(self.k).copy(), bits(self.v).copy()
        for x in (k, v):
            old = x.copy()
            for a, b in moves:
                x[:, b] = old[:, a]
        return k, v

    def update(self, new_len, parent=None):
        want = oc.update(parent, new_len, self.table, self.length, self.ref, page=self.page)
        k, v = self.pools_with(want[4])
        B, width = self.table.shape
        to = [torch.full((B, width), 99, dtype=torch.int32, device="cuda"), cu.i32(np.full(B, 99)),
              cu.i32(np.full(len(self.ref), 99)), cu.i32([99])]
        self.ds.cache_update(self.C, None if parent is None else cu.i32(parent), cu.i32(new_len), cu.i32(self.table),
                             cu.i32(self.length), cu.i32(self.ref), *to, self.k, self.v, self.ws)
        for got, ref in zip(to, want):
            np.testing.assert_array_equal(got.cpu().numpy(), ref)
        np.testing.assert_array_equal(bits(self.k), k)
        np.testing.assert_array_equal(bits(self.v), v)
        self.table, self.length, self.ref = want[:3]
        return want

    def compact(self):
        want = oc.compact(self.table, self.length, self.ref, page=self.page)
        k, v = self.pools_with(want[3])
        to = [torch.full(self.table.shape, 99, dtype=torch.int32, device="cuda"), cu.i32(np.full(len(self.ref), 99)),
              cu.i32([99])]
        self.ds.cache_compact(self.C, cu.i32(self.table), cu.i32(self.length), cu.i32(self.ref), *to, self.k, self.v,
                              self.ws)
        for got, ref in zip(to, want):
            np.testing.assert_array_equal(got.cpu().numpy(), ref)
        np.testing.assert_array_equal(bits(self.k), k)
        np.testing.assert_array_equal(bits(self.v), v)
        self.table, self.ref = want[:2]
        return want


@pytest.mark.parametrize("cache,page,layers,Hkv,D", [("bf16", 16, 1, 1, 64), ("f8", 16, 3, 2, 64), ("f32", 64, 2, 3, 128)])
def test_update_and_compact_of_random_sequences(ds, cache, page, layers, Hkv, D):
    B, n_pages, width = 13, 40, 12
    p = Pages(ds, B, n_pages, page, width, layers, Hkv, D, cache)
    rng = np.random.default_rng(3)
    short = 0
    for step in range(14):
        parent = None if step % 3 == 0 else np.where(rng.random(B) < 0.5, np.arange(B), rng.integers(-1, B + 1, B))
        base = p.length if parent is None else np.where((parent >= 0) & (parent < B), p.length[np.clip(parent, 0, B - 1)], 0)
        new = base + rng.integers(-3 * page, 4 * page, B)
        print(f"[gpu] update step {step} {cache}", flush=True)
        short += p.update(new, parent)[3] > 0
        if step % 4 == 3:
            p.compact()
    assert short  # the pool ran out at least once
    p.update(np.zeros(B, np.int64))
    assert (p.ref == 0).all()
    p.compact()


@pytest.mark.parametrize("n_pages", [1, 4095, 4096, 4097, 9000, 9216, 32768, 32769])
def test_pages_around_the_scan_blocks(ds, n_pages):
    B = 5
    p = Pages(ds, B, n_pages, 16, max(1, n_pages // 3), seed=1)
    p.update(np.array([16 * (n_pages // 3), 16 * (n_pages // 4), 1, 0, 40]))
    p.update(np.array([16 * (n_pages // 3) - 17, 0, 1, 5, 0]))
    p.compact()
    p.update(np.array([0, 16, 0, 5, 0]))
    p.compact()
    p.update(np.array([1, 16, 1, 5, 1]))


@pytest.mark.parametrize("B", [700, 1024, 1100])
def test_update_many_slots(ds, B):
    p = Pages(ds, B, 3000, 16, 9, seed=2)
    rng = np.random.default_rng(4)
    p.update(rng.integers(0, 100, B))
    parent = rng.integers(0, B, B)
    p.update(p.length[parent] + rng.integers(-20, 30, B), parent)
    p.compact()
    p.update(p.length - 1)


def test_update_forks_share_until_they_write(ds):
    # 20 tokens, forked into 4: the full page stays shared, every fork that writes gets its own partial page
    p = Pages(ds, 4, 12, 16, 4)
    p.update([20, 0, 0, 0])
    p.update([20] * 4, [0, 0, 0, 0])
    assert p.ref.tolist()[:2] == [4, 4]
    got = p.update([21, 20, 25, 36])
    assert len(got[4]) == 3 and p.ref[0] == 4
    assert len({int(p.table[b, 1]) for b in range(4)}) == 4


def test_update_of_a_request_for_more_than_exists(ds):
    p = Pages(ds, 3, 5, 16, 100)
    got = p.update([100 * 16, 16, 2**31 - 1])
    assert got[3] == 100 + 1 + 100 - 5 and p.length.tolist() == [0, 0, 0]


def test_cycle_of_cache_calls_matches_the_oracle(ds):
    """Grow, append and attend, drop rejected tokens, fork, compact: several cycles, the pool's content checked
    against sequences kept in numpy."""
    B, Hq, Hkv, D, page, width, layers = 6, 4, 2, 64, 16, 8, 2
    p = Pages(ds, B, 60, page, width, layers, Hkv, D)
    p.k.fill_(float("nan"))
    p.v.fill_(float("nan"))
    rng = np.random.default_rng(8)
    T = 9
    C = ds.Cache.make(B, 60, page, width, layers, Hq, Hkv, D)
    p.ws = torch.empty(ds.cache_workspace_bytes(C, T), dtype=torch.uint8, device="cuda")
    keys = [np.zeros((layers, 0, Hkv, D)) for _ in range(B)]
    for cycle in range(7):
        n = rng.integers(0 if cycle else 1, T + 1, B)
        p.update(p.length + n)
        start = np.cumsum(n) - n
        rows = max(1, int(n.sum()))
        for layer in range(layers):
            k, v = (torch.randn(rows, Hkv, D).bfloat16() for _ in range(2))
            q = torch.randn(rows, Hq, D).bfloat16()
            common = (cu.i32(n), cu.i32(start), T, cu.i32(p.length), cu.i32(p.table))
            print(f"[gpu] cycle {cycle} layer {layer}", flush=True)
            ds.cache_append(C, layer, k.cuda(), v.cuda(), *common, None, None, p.k, p.v)
            out, lse = torch.full((rows, Hq, D), 77.0, dtype=torch.bfloat16, device="cuda"), torch.full((rows, Hq), 77.0, device="cuda")
            ds.cache_attend(C, layer, q.cuda(), *common, p.k, p.v, None, None, out, lse, p.ws)
            c = cu.Case("bf16", page, n, start, p.length, p.table, p.k.cpu(), p.v.cpu(), None, None, q, None, None)
            check_attend(c, out.cpu(), lse.cpu(), cu.oracle_attend(c, layer=layer))
            for b in range(B):
                s = keys[b]
                if layer == 0:
                    keys[b] = s = np.concatenate([s, np.zeros((layers, n[b], Hkv, D))], 1)
                s[layer, s.shape[1] - n[b]:] = k[start[b]:start[b] + n[b]].double().numpy()
        drop = np.minimum(rng.integers(0, T, B), n)
        p.update(p.length - drop)
        keys = [s[:, :m] for s, m in zip(keys, p.length)]
        if cycle % 2:
            parent = rng.integers(0, B, B)
            p.update(p.length[parent], parent)
            keys = [keys[a] for a in parent]
        if cycle % 3 == 2:
            p.compact()
        pool = p.k.cpu().double().numpy()
        for b in range(B):
            for layer in range(layers):
                for h in range(Hkv):
                    got = oc.sequence(pool, layer, p.table[b], int(p.length[b]), h, page, False)
                    np.testing.assert_array_equal(got, keys[b][layer, :, h])


def test_graph_replays(ds):
    """Update, append and attend captured once; replayed with eager work and other inputs between."""
    B, Hq, Hkv, D, page, width = 4, 8, 2, 128, 16, 40
    T = 5
    p = Pages(ds, B, 170, page, width, 1, Hkv, D)
    C = ds.Cache.make(B, 170, page, width, 1, Hq, Hkv, D)
    ws = torch.empty(ds.cache_workspace_bytes(C, T), dtype=torch.uint8, device="cuda")
    p.update(np.array([300, 17, 64, 600]))
    t0, l0, r0 = cu.i32(p.table), cu.i32(p.length), cu.i32(p.ref)
    t1, l1, r1, short = torch.empty_like(t0), torch.empty_like(l0), torch.empty_like(r0), cu.i32([0])
    new, n = cu.i32(p.length + T), cu.i32(np.full(B, T))
    k, v, q = (torch.randn(B * T, h, D, device="cuda").bfloat16() for h in (Hkv, Hkv, Hq))
    out, lse = torch.zeros_like(q), torch.zeros(B * T, Hq, device="cuda")
    kp, vp = p.k.clone(), p.v.clone()

    def step(out, lse, kp, vp):
        ds.cache_update(C, None, new, t0, l0, r0, t1, l1, r1, short, kp, vp, ws)
        ds.cache_append(C, 0, k, v, n, None, T, l1, t1, None, None, kp, vp)
        ds.cache_attend(C, 0, q, n, None, T, l1, t1, kp, vp, None, None, out, lse, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out, lse, kp, vp)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out, lse, kp, vp)
    for i in range(4):
        q.copy_(torch.randn_like(q))
        k.copy_(torch.randn_like(k))
        if i == 2:
            new.copy_(cu.i32(p.length + np.array([0, 5, 2, 1])))
            n.copy_(cu.i32([0, 5, 2, 1]))
        eo, el, ek, ev = torch.zeros_like(q), torch.zeros_like(lse), p.k.clone(), p.v.clone()
        step(eo, el, ek, ev)
        torch.cuda.synchronize()
        out.zero_()
        lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eo) and torch.equal(lse, el), i
