"""CPU checks of the 8-bit cache's and the step tables' entry points: what they refuse, before any device work."""
from __future__ import annotations

import ctypes

import pytest
import torch

from test_kv_binding import OnDevice, Recorder, ints

FAKE, MIS = 0x1000, 0x1008   # never dereferenced: every call here ends in the checks


def structs():
    from lora_bgmv_shrink_amd import binding as b
    cache = b.KvCacheQ8T(FAKE, FAKE, FAKE, FAKE, 2 * 16 * 64, 64, 16 * 64, 8, 2, 1, 8, 16, 4, 2, 64)
    batch = b.KvBatchT(FAKE, FAKE, FAKE, 4, 3, 5, 4, 60, None, None, None, 0, 0, 0, 0)
    rope = b.RopeT(FAKE, FAKE, 32, 100, 64, 0)
    return b, cache, batch, rope


def attn(b, cache, batch, fn="lora_attn_paged_q8", q=FAKE, ldq=256, hq=4, scale=0.1, window=0, n_sink=0, o=FAKE,
         o_dtype=1, ldo=256, lse=None, ws=FAKE, ws_bytes=0):
    return getattr(b.library(), fn)(None if cache is None else ctypes.addressof(cache),
                                    None if batch is None else ctypes.addressof(batch), q, ldq, hq, scale, window,
                                    n_sink, o, o_dtype, ldo, lse, None, ws, ws_bytes, None)


def append(b, cache, batch, rope, dtype=1, q=FAKE, ldq=256, hq=4, k=FAKE, ldk=128, v=FAKE, ldv=128, qo=FAKE, ldqo=256,
           status=None):
    return b.library().lora_kv_append_q8(None if cache is None else ctypes.addressof(cache),
                                         None if batch is None else ctypes.addressof(batch),
                                         None if rope is None else ctypes.addressof(rope), dtype, q, ldq, hq, k, ldk, v,
                                         ldv, qo, ldqo, status, None)


@pytest.mark.parametrize("field,value,unsupported", [
    ("k", 0, False), ("v", 0, False), ("k", MIS, True), ("k_scale", 0, False), ("v_scale", 0, False),
    ("k_scale", 0x1002, True), ("n_pages", 0, False), ("page_size", 12, True), ("page_size", 0, False),
    ("block_size", 0, False), ("block_size", 3, True), ("block_size", 32, False), ("n_kv_heads", 0, False),
    ("head_dim", 80, True), ("head_dim", 0, False), ("token_stride", 72, True), ("page_stride", -16, False),
    ("page_stride", 24, True), ("head_stride", 8, True), ("scale_head_stride", -1, False),
    ("scale_block_stride", 1 << 40, True), ("token_stride", 1 << 40, True)])
def test_cache_refusals(field, value, unsupported):
    b, cache, batch, rope = structs()
    setattr(cache, field, value)
    want = b.LORA_E_UNSUPPORTED if unsupported else b.LORA_E_INVALID
    assert attn(b, cache, batch) == want
    assert append(b, cache, batch, rope) == want
    n = ctypes.c_size_t()
    assert b.library().lora_attn_workspace_q8(ctypes.addressof(cache), ctypes.addressof(batch), 4, ctypes.byref(n)) == want


def test_blocks_of_more_than_128_tokens():
    b, cache, batch, rope = structs()
    cache.page_size = cache.block_size = 256
    assert attn(b, cache, batch) == b.LORA_E_UNSUPPORTED
    assert append(b, cache, batch, rope) == b.LORA_E_UNSUPPORTED


@pytest.mark.parametrize("field,value", [("row_off", 0), ("kv_len", 0), ("pages", 0), ("n_rows", -1), ("n_seqs", -1),
                                         ("max_rows", -1), ("ldp", -1), ("n_groups", -1), ("pages", 0x1002)])
def test_batch_refusals(field, value):
    b, cache, batch, rope = structs()
    setattr(batch, field, value)
    assert attn(b, cache, batch) == b.LORA_E_INVALID
    assert append(b, cache, batch, rope) == b.LORA_E_INVALID


def test_attention_refusals():
    b, cache, batch, _ = structs()
    I, U = b.LORA_E_INVALID, b.LORA_E_UNSUPPORTED
    assert attn(b, None, batch) == I and attn(b, cache, None) == I
    assert attn(b, cache, batch, hq=3) == I and attn(b, cache, batch, hq=0) == I
    assert attn(b, cache, batch, window=-1) == I and attn(b, cache, batch, n_sink=-1) == I
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert attn(b, cache, batch, scale=scale) == I
    assert attn(b, cache, batch, q=None) == I and attn(b, cache, batch, o=None) == I
    assert attn(b, cache, batch, o_dtype=5) == I
    assert attn(b, cache, batch, ldq=255) == I and attn(b, cache, batch, ldo=255) == I
    assert attn(b, cache, batch, q=MIS) == U and attn(b, cache, batch, ldq=260) == U and attn(b, cache, batch, ldo=260) == U
    assert attn(b, cache, batch, lse=0x1002) == U
    assert attn(b, cache, batch, fn="lora_attn_prefix_q8") == I
    batch.group_off = batch.prefix_len = batch.prefix_pages = FAKE
    batch.n_groups, batch.ldpp, batch.max_prefix_len, batch.max_group_rows = 1, 4, 60, 5
    assert attn(b, cache, batch) == I
    assert attn(b, cache, batch, fn="lora_attn_prefix_q8") == b.LORA_E_WORKSPACE
    n = ctypes.c_size_t()
    assert b.library().lora_attn_workspace_q8(ctypes.addressof(cache), ctypes.addressof(batch), 4, ctypes.byref(n)) == b.LORA_OK
    assert n.value > 0
    assert attn(b, cache, batch, fn="lora_attn_prefix_q8", ws_bytes=n.value - 1) == b.LORA_E_WORKSPACE
    assert attn(b, cache, batch, fn="lora_attn_prefix_q8", ws=MIS, ws_bytes=n.value) == b.LORA_E_WORKSPACE


def test_append_refusals():
    b, cache, batch, rope = structs()
    I, U = b.LORA_E_INVALID, b.LORA_E_UNSUPPORTED
    assert append(b, None, batch, rope) == I and append(b, cache, None, rope) == I
    assert append(b, cache, batch, rope, dtype=9) == I and append(b, cache, batch, rope, hq=-1) == I
    assert append(b, cache, batch, rope, k=None) == I and append(b, cache, batch, rope, v=None) == I
    assert append(b, cache, batch, rope, q=None) == I and append(b, cache, batch, rope, qo=None) == I
    assert append(b, cache, batch, rope, ldk=127) == I and append(b, cache, batch, rope, ldq=255) == I
    assert append(b, cache, batch, rope, k=MIS) == U and append(b, cache, batch, rope, ldv=132) == U
    assert append(b, cache, batch, rope, qo=MIS) == U and append(b, cache, batch, rope, ldqo=260) == U
    assert append(b, cache, batch, rope, status=0x1002) == U
    for field, value, want in (("cos", 0, I), ("rot_dim", 80, I), ("rot_dim", 24, U), ("ld", 31, I), ("ld", 34, U), ("n_pos", 0, I)):
        _, _, _, r = structs()
        setattr(r, field, value)
        assert append(b, cache, batch, r) == want, field
    batch.n_rows = 0
    assert append(b, cache, batch, rope, k=None, v=None, q=None, qo=None) == b.LORA_OK
    batch.n_rows, batch.n_seqs, cache.n_kv_heads = 5, 1 << 24, 1 << 10
    assert append(b, cache, batch, rope, ldk=1 << 20, ldv=1 << 20) == U
    _, cache, batch, rope = structs()
    for field in ("n_rows", "n_seqs"):   # more blocks than a launch has workgroups
        _, cache, batch, rope = structs()
        cache.block_size = 1
        setattr(batch, field, 1 << 26)
        assert append(b, cache, batch, rope) == U, field


def plan_struct(b):
    return b.KvPlanT(FAKE, FAKE, FAKE, FAKE, FAKE, 8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 3, 1, 16,
                     100, 64)


@pytest.mark.parametrize("field,value,unsupported", [
    ("new_rows", 0, False), ("kv_len", 0, False), ("kv_len_out", 0, False), ("pages", 0, False), ("free_pages", 0, False),
    ("n_free", 0, False), ("n_free_out", 0, False), ("row_off", 0, False), ("group_off", 0, False),
    ("prefix_len", 0, False), ("n_seqs", -1, False), ("n_groups", -1, False), ("page_size", 0, False),
    ("page_size", 48, True), ("page_size", 1 << 21, True), ("max_free", -1, False), ("max_rows", -1, False),
    ("ldp", -1, False), ("n_seqs", (1 << 20) + 1, True), ("ldp", 1 << 40, True), ("kv_len", 0x1002, True),
    ("row_slot", 0x1004, True), ("row_pos", 0x1001, True), ("max_rows", 2 ** 31 - 1, True)])
def test_plan_refusals(field, value, unsupported):
    from lora_bgmv_shrink_amd import binding as b
    p = plan_struct(b)
    setattr(p, field, value)
    want = b.LORA_E_UNSUPPORTED if unsupported else b.LORA_E_INVALID
    n = ctypes.c_size_t()
    assert b.library().lora_kv_plan_workspace(ctypes.addressof(p), ctypes.byref(n)) == want
    assert b.library().lora_kv_plan(ctypes.addressof(p), None, FAKE, 1 << 30, None) == want


def test_plan_workspace():
    from lora_bgmv_shrink_amd import binding as b
    lib, n = b.library(), ctypes.c_size_t()
    p = plan_struct(b)
    assert lib.lora_kv_plan_workspace(None, ctypes.byref(n)) == b.LORA_E_INVALID
    assert lib.lora_kv_plan_workspace(ctypes.addressof(p), None) == b.LORA_E_INVALID
    for k in ("adapter", "row_seq", "row_adapter", "row_pos", "row_slot"):   # not asked for
        setattr(p, k, 0)
    assert lib.lora_kv_plan_workspace(ctypes.addressof(p), ctypes.byref(n)) == b.LORA_OK and n.value > 0
    for ws, size in ((None, n.value), (FAKE, n.value - 1), (MIS, n.value)):
        assert lib.lora_kv_plan(ctypes.addressof(p), None, ws, size, None) == b.LORA_E_WORKSPACE
    assert lib.lora_kv_plan(ctypes.addressof(p), 0x1002, FAKE, n.value, None) == b.LORA_E_UNSUPPORTED


# ---- the binding's own checks ----------------------------------------------

@pytest.fixture
def b(monkeypatch):
    from lora_bgmv_shrink_amd import binding
    monkeypatch.setattr(OnDevice, "get_device", lambda self: getattr(self, "card", 0), raising=False)
    return binding


def eight(*shape):
    return OnDevice.of(torch.zeros(shape, dtype=torch.uint8)).view(torch.float8_e4m3fn)


def floats(*shape):
    return OnDevice.of(torch.zeros(shape))


def test_cache_q8(b):
    c = b.KvCacheQ8(eight(5, 16, 2, 64), eight(5, 16, 2, 64), floats(5, 4, 2), floats(5, 4, 2))
    assert (c.block_size, c.page_size, c.struct.scale_page_stride, c.dtype) == (4, 16, 8, torch.bfloat16)
    for k, ks in ((eight(5, 16, 2, 64), floats(5, 3, 2)), (eight(5, 16, 2, 64), floats(4, 4, 2)),
                  (eight(5, 16, 2, 64), floats(5, 4, 3)), (eight(5, 16, 2, 64), floats(5, 4, 2).double()),
                  (OnDevice.of(torch.zeros((5, 16, 2, 64), dtype=torch.uint8)), floats(5, 4, 2)),
                  (eight(5, 16, 2, 128)[..., ::2], floats(5, 4, 2))):
        with pytest.raises(AssertionError):
            b.KvCacheQ8(k, k, ks, ks)
    far = floats(5, 4, 2)
    far.card = 1
    with pytest.raises(AssertionError, match="one device"):
        b.KvCacheQ8(eight(5, 16, 2, 64), eight(5, 16, 2, 64), far, far)


def test_plan_binding(b, monkeypatch):
    lens, pages, free, height = ints(5, 6), ints([0, 1], [2, 3]), ints(9, 8, 7), ints(3)
    with pytest.raises(AssertionError, match="pages"):
        b.KvPlan(lens, ints([0, 1]), free, height, 16, 8)
    with pytest.raises(AssertionError, match="prefix_len"):
        b.KvPlan(lens, pages, free, height, 16, 8, group_off=ints(0, 2))
    with pytest.raises(AssertionError, match="int32"):
        b.KvPlan(lens.long(), pages, free, height, 16, 8)
    with pytest.raises(b.LoraError) as e:
        b.KvPlan(lens, pages, free, height, 12, 8)
    assert e.value.status == b.LORA_E_UNSUPPORTED
    plan = b.KvPlan(lens, pages, free, height, 16, 8)
    assert plan.kv_len_out is lens and plan.n_free_out is height and plan.row_slot.dtype == torch.int64
    rec = Recorder()
    monkeypatch.setattr(b, "_lib", rec)
    monkeypatch.setattr(b, "_stream", lambda dev: 0)
    for rows in (ints(1), ints(1, 2).long(), torch.tensor([1, 2], dtype=torch.int32)):
        with pytest.raises(AssertionError):
            b.lora_kv_plan(plan, rows)
    with pytest.raises(AssertionError, match="status"):
        b.lora_kv_plan(plan, ints(1, 1), status=ints(0).long())
    assert rec.calls == 0
    assert b.lora_kv_plan(plan, ints(1, 1), ints(0, 0)) is plan and rec.calls == 1


def test_caches_are_not_mixed_up(b, monkeypatch):
    """The two caches are different structures: an entry point of one refuses the other's."""
    rec = Recorder()
    eight_bits = b.KvCacheQ8(eight(5, 16, 2, 64), eight(5, 16, 2, 64), floats(5, 4, 2), floats(5, 4, 2))
    wide = b.KvCache(*(OnDevice.of(torch.zeros((5, 16, 2, 64), dtype=torch.bfloat16)) for _ in range(2)))
    batch = b.KvBatch(ints(0, 1), ints(5), ints([0]), 1, 1, 5)
    q, k = (OnDevice.of(torch.zeros((1, n), dtype=torch.bfloat16)) for n in (256, 128))
    monkeypatch.setattr(b, "_lib", rec)
    for cache, fns in ((wide, (b.lora_attn_paged_q8, b.lora_attn_prefix_q8)), (eight_bits, (b.lora_attn_paged, b.lora_attn_prefix))):
        for fn in fns:
            with pytest.raises(AssertionError, match="takes a KvCache"):
                fn(cache, batch, q, 0.1)
    for cache, fns in ((wide, (b.lora_kv_append_q8,)), (eight_bits, (b.lora_kv_append,))):
        for fn in fns:
            with pytest.raises(AssertionError, match="takes a KvCache"):
                fn(cache, batch, q, k, k)
    for fn, cache in ((b.lora_attn_workspace, eight_bits), (b.lora_attn_workspace_q8, wide)):
        with pytest.raises(AssertionError, match="takes a KvCache"):
            fn(cache, batch, 4)
    assert rec.calls == 0
