"""A tree that is a chain against the same tokens as a sequence, for more than 16 rows a kv head: the tree's kernel has the
sequence's tiles, operands and order of summation, so that results are equal bit for bit wherever its waves do not share
rows.  They share them with head size 64 where a tile of 128 rows has 64 or fewer; there both are held against the oracle."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import tree as ot  # noqa: E402
from tests import tree_util as tu  # noqa: E402
from tests.test_gpu_cache import ds  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def chain(seed, dtype, D, n, Hq=8, Hkv=2):
    c = tu.make(seed, dtype, 16, D, Hq, Hkv, n, [n[0] + 100, 77, n[2]])
    parent = np.concatenate([np.arange(x) - 1 for x in n])
    return (c, *ot.mask(parent, c.n_new, c.row_start, len(parent), int(max(n))))


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("dtype", ["bf16", "f8", "f8t"])
@pytest.mark.parametrize("D,n", [(128, [40, 38, 7]), (128, [10, 8, 5]), (128, [33, 1, 0]), (256, [40, 38, 7]),
                                 (256, [9, 5, 6]), (64, [32, 30, 20]), (64, [64, 49, 17])])
def test_equal_bit_for_bit(ds, dtype, D, n, window):  # noqa: F811
    # (head size 64: 65 rows or more in every tile of 128)
    c, words, depth = chain(11, dtype, D, n)
    if window:
        words, depth = ot.mask(np.concatenate([np.arange(x) - 1 for x in n]), c.n_new, c.row_start, len(c.q), max(n), window)
    out, lse = tu.gpu_tree(ds, c, words, depth, window=window)
    want, want_lse = tu.gpu_attend(ds, c, window=window)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype", ["bf16", "f8", "f8t"])
@pytest.mark.parametrize("n", [[10, 8, 5], [16, 15, 9], [40, 38, 7]])
def test_shared_rows(ds, dtype, n):  # noqa: F811
    c, words, depth = chain(12, dtype, 64, n)
    ref = tu.oracle_tree(c, words, depth)
    tu.check(c, *tu.gpu_tree(ds, c, words, depth), ref)
    tu.check(c, *tu.gpu_attend(ds, c), ref)
