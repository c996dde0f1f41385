"""CPU checks of the paged cache's Python binding: what it refuses before the library is called."""
from __future__ import annotations

import pytest
import torch


@pytest.fixture
def b():
    from lora_bgmv_shrink_amd import binding
    return binding


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on a device, for checks that end before any launch."""
    is_cuda = property(lambda self: True)

    @staticmethod
    def of(t):
        return t.as_subclass(OnDevice)


def ints(*v):
    return OnDevice.of(torch.tensor(v, dtype=torch.int32))


def groups(b, **kw):
    """Four sequences of one row in two groups, pages of 16 tokens."""
    return b.KvBatch(ints(0, 1, 2, 3, 4), ints(5, 6, 7, 8), ints([0], [1], [2], [3]), 4, 1, 8, ints(0, 2, 4),
                     ints(16, 30), ints([4, 5], [6, 7]), **kw)


def test_groups_need_their_bounds(b):
    for kw in ({}, {"max_prefix_len": 30}, {"max_group_rows": 2}):
        with pytest.raises(AssertionError, match="max_prefix_len and max_group_rows"):
            groups(b, **kw)
    batch = groups(b, max_prefix_len=30, max_group_rows=2)
    assert (batch.struct.max_prefix_len, batch.struct.max_group_rows, batch.n_groups) == (30, 2, 2)
    with pytest.raises(AssertionError, match="prefix_len and prefix_pages"):
        b.KvBatch(ints(0, 1), ints(5), ints([0]), 1, 1, 5, ints(0, 1), max_prefix_len=0, max_group_rows=1)
    plain = b.KvBatch(ints(0, 1), ints(5), ints([0]), 1, 1, 5)
    assert (plain.n_groups, plain.struct.max_prefix_len, plain.struct.max_group_rows) == (0, 0, 0)
