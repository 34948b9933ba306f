"""The cache binding's checks of its tensors, on the CPU: what is dense is taken."""
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
