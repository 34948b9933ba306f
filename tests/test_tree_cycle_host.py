"""A cycle of drafted trees through runner.PagedCache on the CPU, where not every tree gets its rows: the library's calls
are replaced by their oracles, so that what the cache passes on is seen without a GPU.  A sequence's context stays as it
was, and of a tree that was cut short only nodes that ran are kept."""
from __future__ import annotations

import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache as oc  # noqa: E402
from oracle import tree as ot  # noqa: E402

PAGE, T, Hkv, D = 16, 8, 2, 64


@pytest.fixture
def world(monkeypatch):
    from draft_sampling_verification_markov_amd import dspark, runner
    if not os.path.exists(dspark.LIB_PATH):
        from draft_sampling_verification_markov_amd import build
        build.build()

    def update(C, parent, new_len, table, length, ref, table_out, length_out, ref_out, n_short, k_pool, v_pool, *rest):
        *got, copies = oc.update(parent, new_len.numpy(), table.numpy(), length.numpy(), ref.numpy(), page=PAGE)
        for t, v in zip((table_out, length_out, ref_out, n_short), got):
            t.copy_(torch.from_numpy(np.asarray(v).reshape(t.shape)))
        for a, b in copies:
            for p in (k_pool, v_pool):
                p[:, b] = p[:, a]

    def append(C, layer, k, v, n_new, row_start, max_new, length, table, ks, vs, k_pool, v_pool, stream):
        start = np.arange(C.B) * max_new if row_start is None else row_start.numpy()
        got = oc.append(k_pool.numpy(), v_pool.numpy(), k.numpy(), v.numpy(), n_new.numpy(), start, length.numpy(),
                        table.numpy(), layer=layer, page=PAGE)
        for t, x in zip((k_pool, v_pool), got):
            t.copy_(torch.from_numpy(x))

    def keep(C, path, n_keep, n_new, max_new, length, table, length_out, k_pool, v_pool, stream):
        n = np.full(C.B, max_new) if n_new is None else n_new.numpy()
        got = ot.keep([k_pool.numpy(), v_pool.numpy()], path.numpy(), n_keep.numpy(), n, length.numpy(), table.numpy(),
                      page=PAGE, places=lambda p, page, off: p[:, page, :, off // 8, :, off % 8] if p.ndim == 6
                      else p[:, page, :, off])
        length_out.copy_(torch.from_numpy(got))

    for name, f in (("cache_update", update), ("cache_append", append), ("tree_keep", keep)):
        monkeypatch.setattr(dspark, name, f)
    return dspark, runner


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32)


def contents(cache):
    """Each slot's keys and values, token by token."""
    k, v, table = cache.k.numpy(), cache.v.numpy(), cache.table.numpy()
    return [[(k[:, table[b, j // PAGE], :, j % PAGE].copy(), v[:, table[b, j // PAGE], :, j % PAGE // 8, :, j % 8].copy())
             for j in range(int(s))] for b, s in enumerate(cache.length)]


def same(a, b):
    return len(a) == len(b) and all(np.array_equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


def start(world, n_pages, max_pages, lengths, max_new=T):
    dspark, runner = world
    B = len(lengths)
    cache = runner.PagedCache(dspark.Cache.make(B, n_pages, PAGE, max_pages, 2, 2, Hkv, D, q="f32", cache="f32"), max_new,
                              device="cpu")
    gen = torch.Generator().manual_seed(5)
    cache.k.copy_(torch.randn(cache.k.shape, generator=gen))
    cache.v.copy_(torch.randn(cache.v.shape, generator=gen))
    cache.update(i32(lengths))
    assert cache.length.tolist() == lengths
    return cache


def cycle(cache, nodes, path, n_keep):
    """Grow, append, keep.  Returns the rows that each slot got; the rest is checked here."""
    B, layers = cache.C.B, cache.C.n_layers
    before = contents(cache)
    n_new = cache.grow(i32(nodes))
    assert n_new.dtype == torch.int32
    gen = torch.Generator().manual_seed(6)
    kv = torch.randn((2, layers, B * cache.max_new, Hkv, D), generator=gen)
    for layer in range(layers):
        cache.append(layer, kv[0, layer], kv[1, layer], n_new=n_new)
    cache.keep(i32(path), i32(n_keep), n_new=n_new)
    for b, (old, new, n) in enumerate(zip(before, contents(cache), n_new.tolist())):
        assert same(old, new[:len(old)]), f"slot {b}'s context changed"
        kept = [x for x in path[b][:n_keep[b]] if x < n]  # a path ascends: what ran of it comes first
        want = [(kv[0, :, b * cache.max_new + x].numpy(), kv[1, :, b * cache.max_new + x].numpy()) for x in kept]
        assert same(want, new[len(old):]), f"slot {b} keeps other tokens than {kept}"
    return n_new.tolist()


PATH = [[0, 2, 5, 7], [0, 1, 4, -1], [0, 3, 6, -1], [1, 2, 3, 4]]


def test_with_room(world):
    cache = start(world, 20, 4, [10, 0, 16, 31])
    assert cycle(cache, [8, 5, 8, 0], PATH, [4, 3, 2, 0]) == [8, 5, 8, 0]
    assert cache.length.tolist() == [14, 3, 18, 31] and int(cache.n_short) == 0


def test_a_pool_without_room(world):
    # all four pages held: slot 0's tree fits its last page; slots 1 and 3 need pages that are not there
    cache = start(world, 4, 4, [8, 16, 12, 13])
    assert cycle(cache, [8, 8, 4, 8], PATH, [4, 3, 2, 4]) == [8, 0, 4, 0]
    assert cache.length.tolist() == [12, 16, 14, 13] and int(cache.n_short) == 2
    # (the next cycle goes on from there)
    assert cycle(cache, [4, 0, 2, 3], [[1, 3], [0, 0], [0, 1], [0, 2]], [2, 0, 2, 2]) == [4, 0, 2, 3]


def test_the_end_of_the_table_row(world):
    # rows of two pages: 3 of 8 nodes, none, one, all
    cache = start(world, 20, 2, [29, 32, 31, 24])
    assert cycle(cache, [8, 8, 8, 8], PATH, [4, 3, 3, 4]) == [3, 0, 1, 8]
    assert cache.length.tolist() == [31, 32, 32, 28] and int(cache.n_short) == 0


def test_forks_of_a_page(world):
    # slots 0 and 1 share a partly filled page; one page is free, which slot 0's private copy takes
    cache = start(world, 2, 2, [10, 0])
    cache.update(i32([10, 10]), parent=i32([0, 0]))
    assert cycle(cache, [4, 4], [[0, 2], [0, 3]], [2, 2]) == [4, 0]
    assert cache.length.tolist() == [12, 10] and int(cache.n_short) == 1


def test_counts_out_of_range(world):
    cache = start(world, 20, 4, [10, 20])
    assert cycle(cache, [T + 9, -3], [[0, 2], [0, 3]], [2, 2]) == [T, 0]


def test_what_keep_refuses(world, monkeypatch):
    # (shapes and types as the library's binding has them, whatever broadcasting would make of them)
    cache = start(world, 20, 4, [10, 20])
    n_new = cache.grow(i32([4, 4]))
    path, n_keep = i32([[0, 1], [0, 2]]), i32([2, 1])
    for bad, error in ((i32([2]), ValueError), (n_keep.long(), TypeError), ([2, 1], TypeError), (None, TypeError)):
        with pytest.raises(error, match="n_keep"):
            cache.keep(path, bad, n_new=n_new)
        if bad is not None:
            with pytest.raises(error, match="n_new"):
                cache.keep(path, n_keep, n_new=bad)
    for bad, error in ((i32([0, 1]), ValueError), (i32([[0, 1]]), ValueError), (path.long(), TypeError), (None, TypeError)):
        with pytest.raises(error, match="path"):
            cache.keep(bad, n_keep, n_new=n_new)
    assert cache.length.tolist() == [14, 24]
    cache.keep(path, n_keep, n_new=n_new)
    assert cache.length.tolist() == [12, 21]
