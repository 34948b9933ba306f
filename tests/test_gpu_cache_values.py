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
