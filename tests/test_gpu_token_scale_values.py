"""Scales of tokens that are not finite, in a pool that others wrote: rows that do not see the token have the results that
they have without it."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import tree as ot  # noqa: E402
from tests import tree_util as tu  # noqa: E402
from tests.test_gpu_cache import ds  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["k_tok", "v_tok"])
@pytest.mark.parametrize("D,rows,base,width", [(64, 4, 50, None), (64, 40, 50, None), (128, 40, 61, 200), (128, 3, 16, 200),
                                               (256, 40, 3, None), (64, 20, 0, None)])
def test_rows_that_do_not_see_the_token(ds, bad, which, D, rows, base, width):  # noqa: F811
    def case():
        return tu.make(90, "f8t", 16, D, 4, 2, [rows, 2], [rows + base, 30], width=width)

    node = 1
    c, d = case(), case()
    p, off = d.table[0, (base + node) // 16], (base + node) % 16
    getattr(d, which)[0, p, 0, off] = bad
    # a tree: the node's descendants, and itself, see it
    parent, words, _ = tu.trees(91, c)
    see = np.array([node in chain for chain in ot.ancestors(parent[:rows])] + [False] * 2)
    assert see.any() and not see.all()
    for f, blind in ((lambda x: tu.gpu_tree(ds, x, words, None), ~see),
                     (lambda x: tu.gpu_attend(ds, x), np.arange(rows + 2) != np.clip(np.arange(rows + 2), node, rows - 1))):
        (out, lse), (want, want_lse) = f(d), f(c)
        assert torch.equal(out[blind], want[blind]) and torch.equal(lse[blind], want_lse[blind])
        assert torch.equal(out[:, 2:], want[:, 2:]) and torch.equal(lse[:, 2:], want_lse[:, 2:])  # (the other kv head)
    # as a sequence with a window that the last rows have left behind
    (out, lse), (want, want_lse) = (tu.gpu_attend(ds, x, window=2) for x in (d, c))
    blind = np.ones(rows + 2, bool)
    blind[node:node + 2] = False
    assert torch.equal(out[blind], want[blind]) and torch.equal(lse[blind], want_lse[blind])
