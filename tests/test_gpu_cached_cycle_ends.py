"""Cached cycles where a request does not get all of its scheduled rows, through the library:
what such a cycle emits depends on no logits that its forward pass did not write, and is what
the verification makes of the rows that there are."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import synth  # noqa: E402
from tests import cache_util as cu  # noqa: E402

pytestmark = pytest.mark.gpu

B, K = 5, 4
OUTPUTS = ("tok", "n_sched", "out_tok", "n_acc", "next_anchor")


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from draft_sampling_verification_markov_amd import dspark, runner
    dspark.load()
    return dspark, runner


def cycle(lib, n_pages, max_pages, lengths, stale):
    """One cycle from sequences of these lengths; rows that do not run hold the logits `stale`.  Returns the outputs,
    n_new, the cache, and what dspark_verify makes of the whole batch with the drafts that ran."""
    dspark, runner = lib
    cfg = synth.get_config("tbias").replace(B=B, K=K, V=1024, seed=11)
    P = dspark.Problem.from_config(cfg)
    x = runner.CycleInputs.upload(synth.make_inputs(cfg), "cuda")
    x.T.copy_(torch.ones_like(x.T))  # a step costs the same whatever it holds: all drafts are scheduled
    logits = x.Zt.clone()
    x.Zt.fill_(stale)
    o, plain = runner.CycleOutputs(P), runner.CycleOutputs(P)
    cache = runner.PagedCache(dspark.Cache.make(B, n_pages, 16, max_pages, 1, 2, 1, 64), K + 1)
    cache.update(cu.i32(lengths))
    assert cache.length.tolist() == lengths

    def forward(tok, n_new):
        ran = torch.arange(K + 1, device="cuda") < n_new[:, None]
        x.Zt.copy_(torch.where(ran[..., None], logits, x.Zt))
        k = torch.randn(B * (K + 1), 1, 64, device="cuda").bfloat16()
        cache.append(0, k, k, n_new)
        q = torch.randn(B * (K + 1), 2, 64, device="cuda").bfloat16()
        cache.attend(0, q, torch.empty_like(q), n_new=n_new)

    print(f"[gpu] cycle over {n_pages} pages, rows of {max_pages}, lengths {lengths}", flush=True)
    n_new = runner.run_cached_cycle(P, x, o, cache, forward)
    assert (o.n_sched == K).all()
    x.Zt.copy_(logits)
    runner.draft(P, x, plain)
    plain.n_sched.copy_((n_new - 1).clamp(min=0))
    runner.verify(P, x, plain)
    torch.cuda.synchronize()
    return x, o, n_new.tolist(), cache, plain


def check(x, o, n_new, cache, plain, lengths):
    for b, n in enumerate(n_new):
        a = int(o.n_acc[b])
        if n == 0:
            assert a == -1 and (o.out_tok[b] == -1).all() and int(o.next_anchor[b]) == int(x.anchor[b])
            assert torch.isnan(o.logp[b]).all() and torch.isnan(o.resid_mass[b])
        else:
            assert a < n
            for name in ("out_tok", "n_acc", "next_anchor"):
                assert torch.equal(getattr(o, name)[b], getattr(plain, name)[b]), (b, name)
        assert int(cache.length[b]) == lengths[b] + a + 1


@pytest.mark.parametrize("stale", [0.0, 1e4])
def test_a_pool_without_room(lib, stale):
    # all pages held: slots 0, 2 and 4 stay on their last page, 1 and 3 need one that is not there
    lengths = [10, 16, 11, 16, 1]
    x, o, n_new, cache, plain = cycle(lib, 5, 4, lengths, stale)
    assert n_new == [5, 0, 5, 0, 5] and int(cache.n_short.item()) == 2
    check(x, o, n_new, cache, plain, lengths)


@pytest.mark.parametrize("stale", [0.0, 1e4])
def test_the_end_of_the_table_row(lib, stale):
    # rows of 32 tokens: room for 2 of 5 rows, for none, for one, for four, for all
    lengths = [30, 32, 31, 28, 3]
    x, o, n_new, cache, plain = cycle(lib, 20, 2, lengths, stale)
    assert n_new == [2, 0, 1, 4, 5] and int(cache.n_short.item()) == 0
    check(x, o, n_new, cache, plain, lengths)
    assert (cache.length <= 32).all()
