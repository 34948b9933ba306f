"""Cache calls on rows that are laid out otherwise than a projection leaves them."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache as oc  # noqa: E402
from tests import cache_util as cu  # noqa: E402
from tests.test_gpu_cache import check_attend, ds, handle  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_one_head_stored_head_first(ds):  # noqa: F811
    # [1][rows][D] seen as [rows][1][D]: dense rows, whatever the stride of the one head
    c = cu.make(70, "bf16", 16, 64, 1, 1, [3, 6], [20, 41])
    C, ws = handle(ds, c, 6)
    q, k, v = (torch.empty(1, 9, 64, dtype=torch.bfloat16, device="cuda").copy_(x[:, 0]).transpose(0, 1)
               for x in (c.q, c.k, c.v))
    assert q.stride(1) != 64
    out = torch.full((1, 9, 64), 77.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    lse = torch.full((9, 1), 77.0, device="cuda")
    kp, vp = c.k_pool.cuda(), c.v_pool.cuda()
    at = (cu.i32(c.n_new), cu.i32(c.row_start), 6, cu.i32(c.length), cu.i32(c.table))
    print("[gpu] one head, stored head first", flush=True)
    ds.cache_attend(C, 0, q, *at, kp, vp, None, None, out, lse, ws)
    check_attend(c, out.cpu(), lse.cpu(), cu.oracle_attend(c))
    ds.cache_append(C, 0, k, v, *at, None, None, kp, vp)
    want = oc.append(*(x.double().numpy() for x in (c.k_pool, c.v_pool, c.k, c.v)), c.n_new, c.row_start, c.length,
                     c.table, layer=0, page=16)
    for got, ref in zip((kp, vp), want):
        np.testing.assert_array_equal(got.cpu().double().numpy(), ref)
