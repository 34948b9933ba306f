"""A captured chain of the cache's calls (fork, append, attend, compact), every replay against the
oracle: the graph's outputs are buffers of its own that hold a mark before each replay, so a call
that did nothing in it would show.  And a captured decoding cycle over a cache, replayed from token
to token up to the end of the cache's rows, against the same cycles outside a graph."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache as oc  # noqa: E402
from tests import cache_util as cu  # noqa: E402
from tests.test_gpu_cache import check_attend, ds  # noqa: E402,F401

pytestmark = pytest.mark.gpu

MARK = 99


def marked(*shape):
    return torch.full(shape, MARK, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n_pages", [60, 9000])  # bookkeeping in one workgroup, and in several launches
@pytest.mark.parametrize("dtype", ["bf16", "f8"])
def test_fork_append_attend_compact_replayed(ds, n_pages, dtype):  # noqa: F811
    B, Hq, Hkv, D, page, width, T = 4, 8, 2, 64, 16, 12, 5
    C = ds.Cache.make(B, n_pages, page, width, 1, Hq, Hkv, D, cache=dtype)
    rng = np.random.default_rng(80)
    gen = torch.Generator(device="cuda").manual_seed(80)
    base = [torch.randn(s, device="cuda", generator=gen).to(C.cache_type) for s in (C.k_shape, C.v_shape)]
    kp, vp = (x.clone() for x in base)
    scale = torch.tensor([0.5, 0.75], device="cuda")
    ws = torch.empty(ds.cache_workspace_bytes(C, T), dtype=torch.uint8, device="cuda")
    # sequences over shuffled ids, slot 0 with a partly filled last page
    length = np.array([37, 90, 16, 5])
    table, ref, order, at = np.full((B, width), -1), np.zeros(n_pages, np.int64), rng.permutation(n_pages), 0
    for b, s in enumerate(length):
        table[b, :oc.held(s, page)] = order[at:at + oc.held(s, page)]
        at += oc.held(s, page)
    ref[table[table >= 0]] = 1
    t0, l0, r0 = cu.i32(table), cu.i32(length), cu.i32(ref)
    t1, l1, r1, short = marked(B, width), marked(B), marked(n_pages), marked(1)
    t2, r2, live = marked(B, width), marked(n_pages), marked(1)
    parent, new, n = marked(B), marked(B), marked(B)
    k, v = (torch.zeros(B * T, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B * T, Hq, D, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(B * T, Hq, device="cuda")

    def chain():
        ds.cache_update(C, parent, new, t0, l0, r0, t1, l1, r1, short, kp, vp, ws)
        ds.cache_append(C, 0, k, v, n, None, T, l1, t1, scale, scale, kp, vp)
        ds.cache_attend(C, 0, q, n, None, T, l1, t1, kp, vp, scale, scale, out, lse, ws)
        ds.cache_compact(C, t1, l1, r1, t2, r2, live, kp, vp, ws)

    plans = [([0, 0, 2, 0], [40, 37, 20, 42], [3, 0, 4, 5]),   # two forks that write, one that only shares
             ([0, 1, 2, 3], [42, 91, 16, 0], [5, 1, 0, 0]),     # no forks; one slot ends
             ([1, 1, 1, 1], [95, 94, 91, 90], [5, 4, 1, 0]),    # all of one
             ([3, 2, 1, 0], [10, 16, 50, 38], [5, 0, 0, 1])]    # reordered, one cut short
    parent.copy_(cu.i32(plans[0][0]))
    new.copy_(cu.i32(plans[0][1]))
    n.copy_(cu.i32(plans[0][2]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for i in range(6):
        plan = plans[i % len(plans)]
        print(f"[gpu] replay {i} {dtype} {n_pages} pages", flush=True)
        for dst, x in zip((parent, new, n), plan):
            dst.copy_(cu.i32(x))
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
        for x, b in zip((kp, vp), base):
            x.copy_(b)
        for x in (t1, l1, r1, short, t2, r2, live):
            x.fill_(MARK)
        out.fill_(77.0)
        lse.fill_(77.0)
        ws.fill_(0xA5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = oc.update(np.array(plan[0]), np.array(plan[1]), table, length, ref, page=page)
        for got, x in zip((t1, l1, r1, short), want):
            np.testing.assert_array_equal(got.cpu().numpy(), x)
        if i % len(plans) in (0, 2):
            assert want[4]  # (shared last pages were copied)
        pools = [x.cpu().double().numpy() for x in base]
        for x in pools:
            for a, b in want[4]:
                x[:, b] = x[:, a]
        rows = [x.cpu().float().numpy() for x in (k, v)]
        if dtype == "f8":
            rows = [oc.round_f8((x / scale.cpu().numpy()[:, None]).astype(np.float64)) for x in rows]
        start, count = np.arange(B) * T, np.array(plan[2])
        pools = oc.append(*pools, *(x.astype(np.float64) for x in rows), count, start, want[1], want[0], layer=0, page=page)
        seen = cu.Case(dtype, page, count, start, want[1], want[0], torch.from_numpy(pools[0]), torch.from_numpy(pools[1]),
                       scale.cpu(), scale.cpu(), q.cpu(), None, None)
        check_attend(seen, out.cpu(), lse.cpu(), cu.oracle_attend(seen))
        packed = oc.compact(*want[:3], page=page)
        for got, x in zip((t2, r2, live), packed):
            np.testing.assert_array_equal(got.cpu().numpy(), x)
        assert packed[3]  # (pages were moved)
        for got, x in zip((kp, vp), pools):
            y = x.copy()
            for a, b in packed[3]:
                y[:, b] = x[:, a]
            np.testing.assert_array_equal(got.cpu().double().numpy(), y)
        _ = (kp.float().nan_to_num().abs().amax() + out.float().sum()).item()  # the program's own work between replays


def test_a_decoding_loop_of_replays(ds):  # noqa: F811
    import synth
    from draft_sampling_verification_markov_amd import runner
    cfg = synth.get_config("tbias").replace(B=5, K=4, V=1024, seed=12)
    P = ds.Problem.from_config(cfg)
    B, K, Hq, Hkv, D = 5, 4, 8, 2, 64
    C = ds.Cache.make(B, 12, 16, 2, 1, Hq, Hkv, D)
    gen = torch.Generator(device="cuda").manual_seed(81)
    book = torch.randn((cfg.V, Hkv + Hq, D), device="cuda", generator=gen).bfloat16()

    class Loop:
        def __init__(self):
            self.x = runner.CycleInputs.upload(synth.make_inputs(cfg), "cuda")
            self.o, self.cache = runner.CycleOutputs(P), runner.PagedCache(C, K + 1)
            self.out = torch.zeros(B * (K + 1), Hq, D, dtype=torch.bfloat16, device="cuda")

        def forward(self, tok, n_new):
            row = book[tok.long()].view(B * (K + 1), Hkv + Hq, D)
            self.cache.append(0, row[:, :Hkv], row[:, :Hkv], n_new)
            self.cache.attend(0, row[:, Hkv:], self.out, n_new=n_new)

        def cycle(self):
            n_new = runner.run_cached_cycle(P, self.x, self.o, self.cache, self.forward, path=ds.DRAFT_PER_POSITION)
            self.x.anchor.copy_(self.o.next_anchor)
            return n_new

        def state(self):
            o, c = self.o, self.cache
            return [o.tok, o.n_sched, o.out_tok, o.n_acc, o.next_anchor, c.table, c.length, c.ref, c.n_short, self.out, c.k,
                    c.v]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Loop().cycle()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    eager, graphed = Loop(), Loop()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rows = graphed.cycle()
    ended = 0
    for i in range(14):
        print(f"[gpu] decoding loop, replay {i}", flush=True)
        g.replay()
        n_new = eager.cycle()
        torch.cuda.synchronize()
        assert torch.equal(rows, n_new), i
        for j, (a, b) in enumerate(zip(graphed.state(), eager.state())):
            assert torch.equal(a, b), (i, j)
        ended += int((n_new == 0).sum())
        assert (n_new > 0).any() or i > 4
    assert ended and (eager.cache.length <= 32).all()
