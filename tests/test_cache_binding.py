"""The cache binding's checks of its tensors, on the CPU: what is dense is taken, what is no
tensor is a TypeError."""
from __future__ import annotations

import os

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ds():
    from draft_sampling_verification_markov_amd import dspark
    if not os.path.exists(dspark.LIB_PATH):
        from draft_sampling_verification_markov_amd import build
        build.build()
    dspark.load()
    return dspark


@pytest.mark.parametrize("rows", [1, 5])
def test_rows_of_one_head(ds, rows):
    # one head: the stride of that axis says nothing
    x = torch.zeros(1, rows, 64, dtype=torch.bfloat16).transpose(0, 1)
    assert x.stride() == (64, rows * 64, 1)
    assert ds._rows(x, torch.bfloat16, (rows, 1, 64), -1, "k") == (x.data_ptr(), 64)
    y = torch.zeros(rows, 3, 64, dtype=torch.bfloat16)[:, 1:2]
    assert ds._rows(y, torch.bfloat16, (rows, 1, 64), -1, "k") == (y.data_ptr(), 192)


def test_rows_that_are_not_dense(ds):
    for x in (torch.zeros(2, 5, 64).transpose(0, 1), torch.zeros(5, 64, 2).transpose(1, 2), torch.zeros(5, 2, 128)[:, :, ::2],
              torch.zeros(5, 1, 64).expand(5, 2, 64)):
        with pytest.raises(ValueError, match="dense"):
            ds._rows(x, torch.float32, (5, 2, 64), -1, "q")


@pytest.mark.parametrize("bad", [None, 3, [[1.0]]])
def test_what_is_no_tensor(ds, bad):
    C = ds.Cache.make(4, 100, 16, 10, 2, 8, 2, 128)
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ds._rows(bad, torch.bfloat16, (4, 2, 128), -1, "k")
    with pytest.raises(TypeError):
        ds._workspace(bad, -1)
    for call in (lambda: ds.cache_append(C, 0, x, x, None, None, 1, x, x, None, None, bad, x),
                 lambda: ds.cache_attend(C, 0, x, None, None, 1, x, x, bad, x, None, None, x, None, x),
                 lambda: ds.cache_update(C, None, x, x, x, x, x, x, x, x, bad, x, x),
                 lambda: ds.cache_compact(C, x, x, x, x, x, x, bad, x, x)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("bad", [None, 3])
def test_rows_that_are_no_tensor(ds, bad, monkeypatch):
    # past the device check, as on a GPU: the rows of k and q are asked for their number
    monkeypatch.setattr(ds, "_device", lambda t: -1)
    C = ds.Cache.make(4, 100, 16, 10, 2, 8, 2, 128)
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ds.cache_append(C, 0, bad, x, None, None, 1, x, x, None, None, x, x)
    with pytest.raises(TypeError):
        ds.cache_attend(C, 0, bad, None, None, 1, x, x, x, x, None, None, x, None, x)
    with pytest.raises(ValueError):
        ds.cache_append(C, 0, torch.zeros((), dtype=torch.bfloat16), x, None, None, 1, x, x, None, None, x, x)
