"""The oracle of drafted trees and of tokens' own scales, by hand and against what it has to agree with."""
import numpy as np

from oracle import cache as oc
from oracle import tree as ot
from tests import tree_util as tu


def test_mask_by_hand():
    #      0       5
    #    1   2
    #   3     4
    parent = [-1, 0, 0, 1, 2, -1]
    words, depth = ot.mask(parent, [6], [0], 7, 6)
    assert words[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100000, 0xFFFFFFFF]
    assert depth.tolist() == [0, 1, 1, 2, 2, 0, -7]
    words, _ = ot.mask(parent, [6], [0], 6, 6, window=2)
    assert words[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1010, 0b10100, 0b100000]


def test_parents_that_are_none():
    words, depth = ot.mask([0, 5, -3, 2], [4], [0], 4, 40)
    assert words.tolist() == [[1, 0], [2, 0], [4, 0], [12, 0]] and depth.tolist() == [0, 0, 0, 1]


def test_a_chain_is_a_sequence():
    for window in (0, 1, 3, 9, 50):
        c = tu.make(1, "f32", 16, 64, 4, 2, [5, 3, 0], [9, 40, 4])
        parent = np.full(len(c.q), -1)
        for n, r in zip(c.n_new, c.row_start):
            parent[r:r + n] = np.arange(n) - 1
        words, depth = ot.mask(parent, c.n_new, c.row_start, len(parent), 5, window)
        k, v = c.values()
        want = oc.attend(c.q.double().numpy(), c.n_new, c.row_start, c.length, c.table, k, v, layer=0, page=16, scale=0.125,
                         window=window)
        got = tu.oracle_tree(c, words, depth, scale=0.125, window=window)
        for x, y in zip(got, want):
            assert np.allclose(x, y, rtol=1e-12, atol=1e-12, equal_nan=True)


def test_a_branch_is_a_sequence_of_its_own():
    # a node's result is that of a request whose new tokens are its ancestors alone
    c = tu.make(6, "f32", 16, 64, 2, 1, [9], [30])
    parent, words, depth = tu.trees(7, c)
    got = tu.oracle_tree(c, words, depth)
    k, v = c.values()
    for i in range(9):
        chain = ot.ancestors(parent)[i][::-1]
        at = list(range(21)) + [21 + a for a in chain]
        ks = oc.sequence(k, 0, c.table[0], 30, 0, 16, False)[at]
        vs = oc.sequence(v, 0, c.table[0], 30, 0, 16, True)[at]
        t = ks @ c.q[i, 0].double().numpy() / 8
        w = np.exp(t - t.max())
        assert np.allclose(got[0][i, 0], w @ vs / w.sum(), rtol=1e-12)


def test_keep_by_hand():
    pool = np.arange(20).reshape(1, 2, 1, 10).astype(float)  # [layers][pages][heads][page]
    table, length = np.array([[1, 0]]), np.array([16])
    out = ot.keep([pool], np.array([[0, 2, 5, 9]]), [3], [8], length, table, page=10,
                  places=lambda p, page, off: p[:, page, :, off])
    # new tokens at positions 8 .. 15: nodes 0, 2, 5 are positions 8, 10, 13
    assert out.tolist() == [11]
    assert pool[0, 1, 0].tolist() == [10, 11, 12, 13, 14, 15, 16, 17, 18, 0] and pool[0, 0, 0, :4].tolist() == [3, 1, 2, 3]


def test_token_scales():
    x = np.array([[448.0, 1.0, -2.0], [0.0, 0.0, 0.0], [np.nan, 4.48, -np.inf], [np.inf, np.nan, 0.0], [1e-44, 0, 0]])
    q, s = ot.quantise_token(x)
    assert np.allclose(s, [1.0, 1.0, 0.01, 1.0, 2.0**-126]) and q[0].tolist() == [448.0, 1.0, -2.0]
    assert np.isnan(q[2, 0]) and q[2, 1] == 448 and q[2, 2] == -448 and q[3, 0] == 448 and (q[1] == 0).all()
    r = np.random.default_rng(0).standard_normal((50, 64)) * 10.0 ** np.arange(-25, 25)[:, None]
    q, s = ot.quantise_token(r)
    assert (np.abs(q).max(-1) == 448).all()
    # an entry is off by at most half a step of e4m3: 2^-4 of the value, 2^-10 below the normal numbers
    assert (np.abs(q * s[:, None] - r) <= np.maximum(2.0**-4 * np.abs(r), 2.0**-10 * s[:, None]) * (1 + 1e-5)).all()
