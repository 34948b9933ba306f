"""The arrangements of work that many requests with more than 16 rows a kv head get, for trees and over tokens' own scales,
against the oracle: whole segments in the order of their lengths with two and three row tiles a head, and keys dealt out
over more (request, row tile) pairs than a workgroup has threads."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import cache_util as cu  # noqa: E402
from tests import tree_util as tu  # noqa: E402
from tests.test_gpu_cache import ds  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def both(ds, c, seed, window=0):  # noqa: F811
    _, words, depth = tu.trees(seed, c, window=window)
    tu.check(c, *tu.gpu_attend(ds, c, window=window), cu.oracle_attend(c, window=window))
    tu.check(c, *tu.gpu_tree(ds, c, words, depth, window=window), tu.oracle_tree(c, words, depth, window=window))


@pytest.mark.parametrize("dtype,D", [("f8t", 64), ("f8t", 128), ("bf16", 64), ("f8", 128), ("f8t", 256)])
@pytest.mark.parametrize("tiles,width", [(2, 50), (2, 90), (3, 64)])
def test_longest_first_with_several_row_tiles(ds, dtype, D, tiles, width):  # noqa: F811
    # 560 or 600 segments, rows of the page table of 800, 1440 or 1024 tokens; many requests of one length, some without
    # new tokens, and of few of them, whose last row tiles are empty
    B, most = (140, 30) if tiles == 2 else (100, 40)
    i = np.arange(B)
    n = np.where(i % 7 == 2, 0, 1 + (i * 11) % most)
    n[[3, B - 1]] = most
    length = np.maximum(n, np.where(i % 3 == 0, 45, 20 + (i * 29) % 70))
    length[[3, 8, B - 2]] = 790, 512, 790
    c = tu.make(40 + tiles, dtype, 16, D, 16, 2, n, length, poison=False, width=width)
    assert -(-int(n.max()) * 8 // 128) == tiles
    both(ds, c, 41)


@pytest.mark.parametrize("dtype,D", [("f8t", 64), ("bf16", 64), ("f8t", 128), ("f8", 256)])
@pytest.mark.parametrize("tiles,window", [(1, 0), (2, 0), (1, 2000)])
def test_dealt_over_more_pairs_than_threads(ds, dtype, D, tiles, window):  # noqa: F811
    # one kv head: 300 pairs of a request and a row tile, 300 segments, rows of the page table of 4800 tokens
    B, most = (300, 11) if tiles == 1 else (150, 40)
    i = np.arange(B)
    n = np.where(i % 5 == 4, 0, 1 + (i * 7) % most)
    n[B // 2] = most
    length = np.where(i % 9 == 5, 0, 6 + (i * 13) % 80)
    length[[3, B // 2, B - 3]] = 1500, 290, 1300
    n = np.minimum(n, length)
    n[B // 2] = most
    c = tu.make(50 + tiles, dtype, 16, D, 4, 1, n, length, poison=False, width=300)
    assert -(-int(n.max()) * 4 // 128) == tiles and B * tiles > 256
    both(ds, c, 51, window=window)
