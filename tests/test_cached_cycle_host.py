"""The host side of runner.run_cached_cycle on the CPU: the library's calls are replaced by
plain ones (the cache's bookkeeping by its oracle), so that what the cycle passes on and what
it reports are seen without a GPU.  Pools without room and sequences at the end of their
table row."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import cache as oc  # noqa: E402

B, K, V, PAGE = 4, 3, 40, 16
STALE = 39  # the token that logits of an earlier cycle name


@pytest.fixture
def world(monkeypatch):
    import os
    from draft_sampling_verification_markov_amd import dspark, runner
    if not os.path.exists(dspark.LIB_PATH):
        from draft_sampling_verification_markov_amd import build
        build.build()

    def draft(P, x, o, stream=None, path=0):
        o.tok.copy_(torch.arange(B * K, dtype=torch.int32).view(B, K))

    def schedule(P, surv, T, n_sched, n_total, ws, stream):
        n_sched.copy_(torch.tensor([3, 3, 2, 0], dtype=torch.int32))

    def verify(P, Zt, Z, E, Wt, anchor, tok, logq, lse, n_sched, out_tok, n_acc, next_anchor, logp, resid, ws, stream):
        """Accepts every scheduled draft; the next token is the row's largest logit."""
        for b, n in enumerate(n_sched.tolist()):
            y = int(Zt[b, n].argmax())
            out_tok[b] = torch.tensor(tok[b, :n].tolist() + [y] + [-1] * (K - n), dtype=torch.int32)
            n_acc[b], next_anchor[b] = n, y

    def update(C, parent, new_len, table, length, ref, table_out, length_out, ref_out, n_short, *rest):
        got = oc.update(parent, new_len.numpy(), table.numpy(), length.numpy(), ref.numpy(), page=PAGE)
        for t, v in zip((table_out, length_out, ref_out, n_short), got):
            t.copy_(torch.from_numpy(np.asarray(v).reshape(t.shape)))

    monkeypatch.setattr(runner, "draft", draft)
    for name, f in (("schedule", schedule), ("verify", verify), ("cache_update", update)):
        monkeypatch.setattr(runner.dspark, name, f)
    return dspark, runner


def start(dspark, runner, n_pages, max_pages, lengths, max_new=K + 1, slots=B):
    P = dspark.Problem(B, K, V, 16, 8, dspark.BF16, dspark.BF16, dspark.BF16, 1.0, 7)
    Zt = torch.zeros(B, K + 1, V)
    Zt[:, :, STALE] = 1.0
    x = runner.CycleInputs(None, Zt, None, None, None, None, 0.0, None, torch.tensor([30, 31, 32, 33], dtype=torch.int32),
                           None)
    o = runner.CycleOutputs(P, device="cpu")
    cache = runner.PagedCache(dspark.Cache.make(slots, n_pages, PAGE, max_pages, 1, 1, 1, 64), max_new, device="cpu")
    if lengths is not None:
        cache.update(torch.tensor(lengths, dtype=torch.int32))
        assert cache.length.tolist() == lengths and int(cache.n_short) == 0

    def forward(tok, n_new):
        """Row i of request b names token 20 + i; rows that are not there keep what they held."""
        assert torch.equal(tok, torch.cat([x.anchor[:, None], o.tok], 1))
        for b, n in enumerate(n_new.tolist()):
            for i in range(n):
                Zt[b, i] = 0.0
                Zt[b, i, 20 + i] = 1.0

    return P, x, o, cache, forward


def check(x, o, cache, lengths, n_new, got):
    assert got.tolist() == n_new
    for b, n in enumerate(n_new):
        a = int(o.n_acc[b])
        if n == 0:  # nothing ran: nothing is emitted, and the request can be tried again
            assert a == -1 and o.out_tok[b].tolist() == [-1] * (K + 1) and int(o.next_anchor[b]) == int(x.anchor[b])
        else:
            assert a == n - 1  # (this verify accepts all that ran)
            assert o.out_tok[b].tolist() == o.tok[b, :a].tolist() + [20 + a] + [-1] * (K - a)
            assert int(o.next_anchor[b]) == 20 + a
        assert int(cache.length[b]) == lengths[b] + a + 1


def test_a_cycle_with_room(world):
    lengths = [10, 0, 16, 31]
    P, x, o, cache, forward = start(*world, 20, 4, lengths)
    got = world[1].run_cached_cycle(P, x, o, cache, forward)
    check(x, o, cache, lengths, [4, 4, 3, 1], got)
    assert int(cache.n_short) == 0


def test_a_pool_without_room_is_reported(world):
    # 4 pages, all held: slots 0 and 2 stay on their last page, slot 1 needs a page that is not there, and so slot 3
    lengths = [10, 16, 12, 16]
    P, x, o, cache, forward = start(*world, 4, 4, lengths)
    got = world[1].run_cached_cycle(P, x, o, cache, forward)
    check(x, o, cache, lengths, [4, 0, 3, 0], got)
    assert int(cache.n_short) == 2
    assert o.n_sched.tolist() == [3, 3, 2, 0]
    # with two pages free again (slots 0 and 2 begin anew) slot 1 goes on from the anchor that it kept; 2 and 3 wait
    cache.update(torch.tensor([0, 16, 0, 16], dtype=torch.int32))
    got = world[1].run_cached_cycle(P, x, o, cache, forward)
    check(x, o, cache, [0, 16, 0, 16], [4, 4, 0, 0], got)
    assert int(cache.n_short) == 2


def test_the_end_of_the_table_row(world):
    # rows of two pages: slot 0 has room for 2 of its 4 tokens, slot 1 for none, slot 2 for 1 of 3, slot 3 for its one
    lengths = [30, 32, 31, 31]
    P, x, o, cache, forward = start(*world, 40, 2, lengths)
    got = world[1].run_cached_cycle(P, x, o, cache, forward)
    check(x, o, cache, lengths, [2, 0, 1, 1], got)
    assert (cache.length <= 32).all() and int(cache.n_short) == 0


@pytest.mark.parametrize("kw", [dict(max_new=K), dict(slots=B + 1), dict(slots=B - 1)], ids=str)
def test_a_cache_of_another_shape_is_refused(world, kw):
    # fewer rows a call than a cycle can schedule, or other slots than the problem's requests
    P, x, o, cache, forward = start(*world, 40, 2, None, **kw)
    with pytest.raises(ValueError):
        world[1].run_cached_cycle(P, x, o, cache, forward)
    assert cache.length.tolist() == [0] * cache.C.B
