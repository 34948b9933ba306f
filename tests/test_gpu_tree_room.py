"""Cycles of drafted trees through runner.PagedCache where not every tree gets its rows (a pool without room, the end of a
row of the page table, forks of one page): contexts stay bit for bit as they were, nodes that ran see what they should, and
of a path the nodes that ran are kept; eagerly, on another stream, and replayed as a graph."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import tree as ot  # noqa: E402
from tests import cache_util as cu  # noqa: E402
from tests import tree_util as tu  # noqa: E402
from tests.test_gpu_cache import ds  # noqa: E402,F401
from tests.test_gpu_tree import parts  # noqa: E402

pytestmark = pytest.mark.gpu

PAGE, T, Hq, Hkv, D, LAYERS = 16, 8, 4, 2, 64, 2


def contents(cache, dtype):
    """Each slot's tokens, each as the bits of its key, its value (and its scales) in all layers."""
    torch.cuda.synchronize()
    pools, table = parts(cache.C, cache.k, cache.v, dtype), cache.table.cpu().numpy()
    at = lambda p, page, off: (p[:, page, :, off // 8, :, off % 8] if p.ndim == 6 else p[:, page, :, off]).copy()  # noqa: E731
    return [[[at(p, table[b, j // PAGE], j % PAGE) for p in pools] for j in range(int(s))]
            for b, s in enumerate(cache.length.cpu())]


def same(a, b):
    return len(a) == len(b) and all(np.array_equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


class Turn:
    """A cache with sequences of these lengths, and the buffers of one cycle of trees over it."""

    def __init__(self, ds, dtype, n_pages, max_pages, lengths, parents=None):  # noqa: F811
        from draft_sampling_verification_markov_amd.runner import PagedCache
        B, self.dtype, self.data = len(lengths), dtype, cu.DATA["f8" if dtype == "f8t" else dtype]
        C = ds.Cache.make(B, n_pages, PAGE, max_pages, LAYERS, Hq, Hkv, D, q="f32" if dtype == "f32" else "bf16", cache=dtype)
        self.B, self.k, self.v, self.q, self.cache = B, [], [], [], PagedCache(C, T)
        self.gen = torch.Generator(device="cuda").manual_seed(3)
        own = cu.i32([x if parents is None or parents[b] == b else 0 for b, x in enumerate(lengths)])
        for _ in range(-(-max(lengths) // T)):
            n = self.cache.grow(own - self.cache.length)
            for layer in range(LAYERS):
                self.cache.append(layer, self.randn(B * T, Hkv, D), self.randn(B * T, Hkv, D), n_new=n)
        if parents is not None:
            self.cache.update(cu.i32(lengths), parent=cu.i32(parents))
        assert self.cache.length.tolist() == lengths
        for _ in range(LAYERS):
            self.k.append(self.randn(B * T, Hkv, D))
            self.v.append(self.randn(B * T, Hkv, D))
            self.q.append(self.randn(B * T, Hq, D))
        rng = np.random.default_rng(4)
        self.parent_host = np.concatenate([tu.parents(rng, T) for _ in range(B)])
        self.parent = cu.i32(self.parent_host)
        self.mask, self.depth = (torch.zeros(B * T, 1, dtype=torch.int32, device="cuda"),
                                 torch.zeros(B * T, dtype=torch.int32, device="cuda"))
        self.out = [torch.full_like(q, 77.0) for q in self.q]

    def randn(self, *shape):
        return torch.randn(shape, device="cuda", generator=self.gen).to(self.data)

    def run(self, nodes, stream=None):
        """The cycle up to the choice of a path."""
        n_new = self.cache.grow(nodes, stream=stream)
        self.cache.mask(self.parent, self.mask, self.depth, n_new=n_new, stream=stream)
        for layer in range(LAYERS):
            self.cache.append(layer, self.k[layer], self.v[layer], n_new=n_new, stream=stream)
            self.cache.tree_attend(layer, self.q[layer], self.mask, self.out[layer], n_new=n_new, stream=stream)
        return n_new

    def case(self, layer, n_new):
        """The state before the path is kept as the oracle takes it."""
        kp, vp = self.cache.k.cpu(), self.cache.v.cpu()
        tok = (None, None)
        if self.dtype == "f8t":
            (kp, kt), (vp, vt) = self.cache.C.token_views(kp), self.cache.C.token_views(vp, True)
            tok = kt, vt
        one = torch.ones(Hkv)
        c = tu.Case(self.dtype, PAGE, n_new, np.arange(self.B) * T, self.cache.length.cpu().numpy(),
                    self.cache.table.cpu().numpy(), kp, vp, one, one, self.q[layer].cpu(), self.k[layer].cpu(),
                    self.v[layer].cpu())
        c.k_tok, c.v_tok = tok
        return c


PATH = [[0, 2, 5, 7], [0, 1, 4, 6], [0, 3, 6, 7], [1, 2, 3, 4]]
WORLDS = [  # pages, width, lengths, nodes, what they get, pages missing, kept lengths (n_keep 4, 3, 2, 4), parents
    pytest.param(4, 4, [8, 16, 12, 13], [8, 8, 4, 8], [8, 0, 4, 0], 2, [12, 16, 14, 13], None, id="no-room"),
    pytest.param(20, 2, [29, 32, 31, 24], [8, 8, 8, 8], [3, 0, 1, 8], 0, [31, 32, 32, 28], None, id="end-of-the-row"),
    # (slots 0 and 1 share a page, and one is free: slot 0's private copy takes it)
    pytest.param(4, 2, [10, 10, 3, 9], [6, 6, 8, 0], [6, 0, 8, 0], 1, [13, 10, 5, 9], [0, 0, 2, 3], id="forks"),
]


@pytest.mark.parametrize("dtype", tu.TYPES)
@pytest.mark.parametrize("n_pages,width,lengths,nodes,got,short,kept,parents", WORLDS)
@pytest.mark.parametrize("side", [False, True])
def test_trees_without_room(ds, dtype, n_pages, width, lengths, nodes, got, short, kept, parents, side):  # noqa: F811
    t = Turn(ds, dtype, n_pages, width, lengths, parents)
    before = contents(t.cache, dtype)
    print(f"[gpu] trees without room {dtype} pages={n_pages} lengths={lengths} nodes={nodes}", flush=True)
    stream = torch.cuda.Stream() if side else None
    want_nodes, path, n_keep = cu.i32(nodes), cu.i32(PATH), cu.i32([4, 3, 2, 4])
    if side:
        stream.wait_stream(torch.cuda.current_stream())
    n_new = t.run(want_nodes, stream)
    if side:
        torch.cuda.current_stream().wait_stream(stream)
    n = n_new.cpu().numpy()
    assert n.tolist() == got and int(t.cache.n_short) == short
    ran = contents(t.cache, dtype)
    for b in range(t.B):
        assert same(before[b], ran[b][:lengths[b]]), f"slot {b}'s context changed"
    words, depth = ot.mask(t.parent_host, n, np.arange(t.B) * T, t.B * T, T)
    there = (np.arange(T) < n[:, None]).reshape(-1)
    assert np.array_equal(t.mask.cpu().numpy().view(np.uint32)[there], words[there])
    for layer in range(LAYERS):
        c = t.case(layer, n)
        tu.check(c, t.out[layer].cpu(), None, tu.oracle_tree(c, words, depth, layer=layer))
    if side:
        stream.wait_stream(torch.cuda.current_stream())
    t.cache.keep(path, n_keep, n_new=n_new, stream=stream)
    if side:
        torch.cuda.current_stream().wait_stream(stream)
    assert t.cache.length.tolist() == kept
    for b, (old, new) in enumerate(zip(before, contents(t.cache, dtype))):
        nodes_kept = [x for x in PATH[b][:[4, 3, 2, 4][b]] if x < n[b]]
        assert same(old + [ran[b][lengths[b] + x] for x in nodes_kept], new), f"slot {b}"


@pytest.mark.parametrize("dtype", ["bf16", "f8t"])
def test_graph_of_a_cycle(ds, dtype):  # noqa: F811
    """Grow, mask, append, attend and keep in one graph, replayed until the rows of the page table are full, each replay
    against the eager cycle."""
    lengths = [20, 9, 31, 0]
    eager, graph = (Turn(ds, dtype, 20, 3, lengths) for _ in range(2))
    nodes, path, n_keep = cu.i32([8, 5, 8, 3]), cu.i32(PATH), cu.i32([4, 3, 2, 2])

    def cycle(t):
        n_new = t.run(nodes)
        t.cache.keep(path, n_keep, n_new=n_new)
        return n_new

    first = [x.clone() for x in (graph.cache.k.view(torch.uint8), graph.cache.v.view(torch.uint8))]
    sets = [x.clone() for s in graph.cache._sets for x in s]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cycle(graph)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n_graph = cycle(graph)
    graph.cache.k.view(torch.uint8).copy_(first[0])
    graph.cache.v.view(torch.uint8).copy_(first[1])
    for x, y in zip([x for s in graph.cache._sets for x in s], sets):
        x.copy_(y)
    full = False
    for turn in range(9):
        for x in eager.out + graph.out:
            x.fill_(77.0)
        n = cycle(eager)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, n_graph), turn
        full |= bool((n < nodes).any())
        for x, y in zip(eager.out, graph.out):
            assert torch.equal(x, y), turn
        assert eager.cache.length.tolist() == graph.cache.length.tolist()
        a, b = contents(eager.cache, dtype), contents(graph.cache, dtype)
        assert all(same(x, y) for x, y in zip(a, b)), turn
    assert full
