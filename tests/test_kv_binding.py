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


class Recorder:
    """Stands in for the library's functions: a call that gets this far has passed the binding's checks."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lib(b, monkeypatch):
    monkeypatch.setattr(OnDevice, "get_device", lambda self: 0, raising=False)
    rec = Recorder()
    monkeypatch.setattr(b, "_lib", rec)
    monkeypatch.setattr(b, "_stream", lambda device: 0)
    return rec


def dev(*shape, dtype=torch.float32):
    return OnDevice.of(torch.zeros(shape, dtype=dtype))


def setup(b):
    cache = b.KvCache(dev(4, 16, 2, 64), dev(4, 16, 2, 64))
    batch = b.KvBatch(ints(0, 1, 2), ints(5, 6), ints([0], [1]), 2, 1, 8)
    return cache, batch


def test_attention_refuses_host_tensors(b, lib):
    """The address of a tensor that is not on the cache's device never reaches a kernel."""
    cache, batch = setup(b)
    q, ws = dev(2, 256), dev(64, dtype=torch.uint8)
    b.lora_attn_paged(cache, batch, q, 0.1, o=dev(2, 256), lse=dev(2, 4), status=ints(0), ws=ws)
    assert lib.calls == 1
    good = dict(o=dev(2, 256), lse=dev(2, 4), status=ints(0), ws=ws)
    for name, bad in (("lse", torch.zeros(2, 4)), ("status", torch.zeros(1, dtype=torch.int32)),
                      ("ws", torch.zeros(64, dtype=torch.uint8)), ("o", torch.zeros(2, 256))):
        with pytest.raises(AssertionError):
            b.lora_attn_paged(cache, batch, q, 0.1, **dict(good, **{name: bad}))
    with pytest.raises(AssertionError):
        b.lora_attn_paged(cache, batch, torch.zeros(2, 256), 0.1, **good)
    # one status word at least, and a workspace whose bytes lie side by side
    with pytest.raises(AssertionError):
        b.lora_attn_paged(cache, batch, q, 0.1, **dict(good, status=ints()))
    with pytest.raises(AssertionError):
        b.lora_attn_paged(cache, batch, q, 0.1, **dict(good, ws=dev(1, dtype=torch.uint8).expand(64)))
    assert lib.calls == 1


def test_append_refuses_host_tensors(b, lib):
    cache, batch = setup(b)
    q, k = dev(2, 256), dev(2, 128)
    good = dict(q_out=dev(2, 256), status=ints(0))
    b.lora_kv_append(cache, batch, q, k, k, **good)
    assert lib.calls == 1
    for name, bad in (("status", torch.zeros(1, dtype=torch.int32)), ("q_out", torch.zeros(2, 256))):
        with pytest.raises(AssertionError):
            b.lora_kv_append(cache, batch, q, k, k, **dict(good, **{name: bad}))
    for args in ((torch.zeros(2, 256), k, k), (q, torch.zeros(2, 128), k), (q, k, torch.zeros(2, 128))):
        with pytest.raises(AssertionError):
            b.lora_kv_append(cache, batch, *args, **good)
    table = dev(8, 32)
    b.Rope(table, dev(8, 32))
    for cos, sin in ((torch.zeros(8, 32), table), (table, torch.zeros(8, 32))):
        with pytest.raises(AssertionError):
            b.Rope(cos, sin)
    assert lib.calls == 1


def test_one_device(b, lib, monkeypatch):
    """Tensors of another device than the cache's are refused."""
    class Other(OnDevice):
        pass

    monkeypatch.setattr(Other, "get_device", lambda self: 1, raising=False)

    def other(t):
        return t.as_subclass(Other)

    cache, batch = setup(b)
    q, k, ws = dev(2, 256), dev(2, 128), dev(64, dtype=torch.uint8)
    far = b.KvBatch(*(other(t) for t in batch.tensors[:3]), 2, 1, 8)
    with pytest.raises(AssertionError):
        b.KvBatch(other(batch.tensors[0]), batch.tensors[1], batch.tensors[2], 2, 1, 8)
    for bt, x, kw in ((far, q, {}), (batch, other(q), {}), (batch, q, {"lse": other(dev(2, 4))})):
        with pytest.raises(AssertionError):
            b.lora_attn_paged(cache, bt, x, 0.1, o=dev(2, 256), ws=ws, **kw)
    rope = b.Rope(other(dev(8, 32)), other(dev(8, 32)))
    for bt, x, y, r in ((far, q, k, None), (batch, q, other(k), None), (batch, q, k, rope)):
        with pytest.raises(AssertionError):
            b.lora_kv_append(cache, bt, x, y, k, r, q_out=dev(2, 256))
    assert lib.calls == 0
