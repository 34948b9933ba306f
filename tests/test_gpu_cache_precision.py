"""Attention of up to 16 rows of a kv head: its weights carry 16 bits into the product with
the values, so with bf16 data the result is off by its own rounding and little more."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import cache_util as cu  # noqa: E402
from tests.test_gpu_cache import ds, gpu_attend  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f8"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (256, 64)])
@pytest.mark.parametrize("G,n_new", [(1, [1, 1, 1]), (4, [4, 1, 3]), (8, [2, 2, 0]), (1, [16, 9, 1])])
@pytest.mark.parametrize("width,window", [(None, 0), (6000, 0), (None, 100)])
def test_few_rows_are_exact_but_for_their_rounding(ds, dtype, D, page, G, n_new, width, window):  # noqa: F811
    """The bound is cache_util.attend_bound's, but for the weights' rounding: a weight w goes into the product as
    y = bf16(w) and z = bf16(w - y).  w - y is exact in fp32 and at most half a step of y, 2^-8 |w|; z is off by half a
    step of that: 2^-16 |w|.  The product has twice the terms.  (z below bf16's normal range is lost: 2^-126 of a sum
    whose largest weight is 1 or more, within the bound's 1e-37 for values below 8.)"""
    c = cu.make(90, dtype, page, D, 2 * G, 2, n_new, [700, 333, 41], width=None if width is None else width // page)
    want, want_lse, mag, span = cu.oracle_attend(c, window=window)
    out, lse = gpu_attend(ds, c, window=window)
    e = np.expm1(268 * cu.U * span) + 8 * cu.U
    n = 700 + 32
    tol = mag * (2 * e + 12 * n * cu.U + 2.0**-16)[..., None] + np.abs(want) * cu.U
    tol = tol + 2.0**-8 * (np.abs(want) + tol) + 1e-36
    off = np.abs(out.double().numpy() - want)
    assert (off <= tol).all(), f"{(off > tol).sum()} of {off.size} off, worst {np.max(off / tol):.3g} bounds"
    _, tol_lse = cu.attend_bound(dtype, want, want_lse, mag, span, 700)
    assert (np.abs(lse.double().numpy() - want_lse) <= tol_lse).all()
