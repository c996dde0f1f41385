"""CPU checks of the paged cache's entry points: what they refuse, before any device work."""
from __future__ import annotations

import ctypes

import pytest

FAKE, MIS = 0x1000, 0x1008   # never dereferenced: every call here ends in the checks


def structs():
    from lora_bgmv_shrink_amd import binding as b
    cache = b.KvCacheT(FAKE, FAKE, 2 * 16 * 64, 64, 16 * 64, b.LORA_BF16, 8, 16, 2, 64)
    batch = b.KvBatchT(FAKE, FAKE, FAKE, 4, 3, 5, 4, 60, None, None, None, 0, 0, 0, 0)
    rope = b.RopeT(FAKE, FAKE, 32, 100, 64, 0)
    return b, cache, batch, rope


def attn(b, cache, batch, fn="lora_attn_paged", q=FAKE, ldq=256, hq=4, scale=0.1, window=0, n_sink=0, o=FAKE, o_dtype=1,
         ldo=256, lse=None, ws=FAKE, ws_bytes=0):
    return getattr(b.library(), fn)(None if cache is None else ctypes.addressof(cache),
                                    None if batch is None else ctypes.addressof(batch), q, ldq, hq, scale, window,
                                    n_sink, o, o_dtype, ldo, lse, None, ws, ws_bytes, None)


def append(b, cache, batch, rope, dtype=1, q=FAKE, ldq=256, hq=4, k=FAKE, ldk=128, v=FAKE, ldv=128, qo=FAKE, ldqo=256):
    return b.library().lora_kv_append(ctypes.addressof(cache), ctypes.addressof(batch),
                                      None if rope is None else ctypes.addressof(rope), dtype, q, ldq, hq, k, ldk, v,
                                      ldv, qo, ldqo, None, None)


@pytest.mark.parametrize("field,value,unsupported", [
    ("k", 0, False), ("k", MIS, True), ("dtype", 7, False), ("n_pages", 0, False), ("page_size", 12, True),
    ("page_size", 0, False), ("n_kv_heads", 0, False), ("head_dim", 80, True), ("head_dim", 0, False),
    ("token_stride", 65, True), ("page_stride", -16, False)])
def test_cache_refusals(field, value, unsupported):
    b, cache, batch, rope = structs()
    setattr(cache, field, value)
    want = b.LORA_E_UNSUPPORTED if unsupported else b.LORA_E_INVALID
    assert attn(b, cache, batch) == want
    assert append(b, cache, batch, rope) == want
    n = ctypes.c_size_t()
    assert b.library().lora_attn_workspace(ctypes.addressof(cache), ctypes.addressof(batch), 4, ctypes.byref(n)) == want


def test_head_dim_256_is_bf16_only():
    b, cache, batch, _ = structs()
    cache.head_dim, cache.dtype = 256, b.LORA_F32
    assert attn(b, cache, batch, ldq=1024, ldo=1024) == b.LORA_E_UNSUPPORTED


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
    assert attn(b, cache, batch, hq=3) == I and attn(b, cache, batch, hq=0) == I     # not a multiple of the key heads
    assert attn(b, cache, batch, window=-1) == I and attn(b, cache, batch, n_sink=-1) == I
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert attn(b, cache, batch, scale=scale) == I
    assert attn(b, cache, batch, q=None) == I and attn(b, cache, batch, o=None) == I
    assert attn(b, cache, batch, o_dtype=5) == I
    assert attn(b, cache, batch, ldq=255) == I and attn(b, cache, batch, ldo=255) == I
    assert attn(b, cache, batch, q=MIS) == U and attn(b, cache, batch, ldq=260) == U and attn(b, cache, batch, ldo=260) == U
    assert attn(b, cache, batch, lse=0x1002) == U
    # groups go with one entry point and not with the other
    assert attn(b, cache, batch, fn="lora_attn_prefix") == I
    batch.group_off = batch.prefix_len = batch.prefix_pages = FAKE
    batch.n_groups, batch.ldpp, batch.max_prefix_len, batch.max_group_rows = 1, 4, 60, 5
    assert attn(b, cache, batch) == I
    assert attn(b, cache, batch, fn="lora_attn_prefix") == b.LORA_E_WORKSPACE
    n = ctypes.c_size_t()
    assert b.library().lora_attn_workspace(ctypes.addressof(cache), ctypes.addressof(batch), 4, ctypes.byref(n)) == 0
    assert n.value > 0
    assert attn(b, cache, batch, fn="lora_attn_prefix", ws=MIS, ws_bytes=n.value) == b.LORA_E_WORKSPACE
    assert attn(b, cache, batch, fn="lora_attn_prefix", ws_bytes=n.value - 1) == b.LORA_E_WORKSPACE
    batch.prefix_len = None
    assert attn(b, cache, batch, fn="lora_attn_prefix") == I


def test_workspace_covers_every_window():
    """The size does not depend on the window, so it bounds what any window's plan takes."""
    b, cache, batch, _ = structs()
    lib = b.library()
    cache.n_kv_heads, batch.n_seqs, batch.n_rows, batch.max_rows, batch.max_kv_len = 2, 9, 300, 200, 5000
    n = ctypes.c_size_t()
    assert lib.lora_attn_workspace(ctypes.addressof(cache), ctypes.addressof(batch), 4, ctypes.byref(n)) == 0
    for window in (0, 1, 63, 64, 100, 1000, 4999, 2 ** 31 - 1):
        # one byte less is refused whatever the window: all calls check the same size
        assert attn(b, cache, batch, window=window, n_sink=4, ws_bytes=n.value - 1) == b.LORA_E_WORKSPACE


def test_append_refusals():
    b, cache, batch, rope = structs()
    I, U = b.LORA_E_INVALID, b.LORA_E_UNSUPPORTED
    assert append(b, cache, batch, rope, dtype=9) == I
    assert append(b, cache, batch, rope, k=None) == I and append(b, cache, batch, rope, v=None) == I
    assert append(b, cache, batch, rope, q=None) == I and append(b, cache, batch, rope, qo=None) == I
    assert append(b, cache, batch, rope, ldk=127) == I and append(b, cache, batch, rope, ldq=255) == I
    assert append(b, cache, batch, rope, k=MIS) == U and append(b, cache, batch, rope, ldv=129) == U
    assert append(b, cache, batch, rope, ldqo=258) == U
    for field, value, want in (("cos", 0, I), ("rot_dim", 0, I), ("rot_dim", 80, I), ("rot_dim", 24, U), ("n_pos", 0, I),
                               ("ld", 31, I), ("ld", 33, U), ("sin", MIS, U)):
        _, _, _, r = structs()
        setattr(r, field, value)
        assert append(b, cache, batch, r) == want, (field, value)


def test_no_rows_is_a_no_op():
    b, cache, batch, rope = structs()
    batch.n_rows = batch.max_rows = 0
    assert append(b, cache, batch, rope) == b.LORA_OK
    assert attn(b, cache, batch) in (b.LORA_OK, b.LORA_E_WORKSPACE)
    batch.n_seqs = 0
    assert attn(b, cache, batch, ws=None) == b.LORA_OK


def workspace(b, cache, batch, hq):
    n = ctypes.c_size_t()
    assert b.library().lora_attn_workspace(ctypes.addressof(cache), ctypes.addressof(batch), hq, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("seed", range(40))
def test_workspace_serves_smaller_bounds(seed):
    """A workspace for a batch's bounds holds every batch whose bounds are no larger, one without groups too."""
    import random
    rng = random.Random(seed)
    b, cache, _, _ = structs()
    hq, cache.n_kv_heads = rng.choice([(32, 8), (64, 8), (4, 4), (20, 1), (64, 2), (5, 1), (512, 256)])
    cache.dtype, cache.head_dim = rng.choice([(b.LORA_BF16, 64), (b.LORA_BF16, 128), (b.LORA_BF16, 256), (b.LORA_F32, 128)])
    cache.page_stride, cache.token_stride, cache.head_stride = 1 << 20, cache.head_dim, 16 * cache.head_dim

    def size(n_seqs, n_rows, max_rows, max_kv_len, n_groups, max_prefix, max_group_rows):
        batch = b.KvBatchT(FAKE, FAKE, FAKE, 4, n_seqs, n_rows, max_rows, max_kv_len, FAKE, FAKE, FAKE, 4, n_groups,
                           max_prefix, max_group_rows)
        return workspace(b, cache, batch, hq)

    def upto(n):
        return rng.choice([n, n, max(1, n - 1), max(1, n // 2), max(1, n // 3), rng.randint(1, n)])

    for _ in range(200):
        most = [rng.choice([1, 8, 32, 33, 200, 600, 5000]), rng.choice([1, 32, 100, 900, 4096, 20000]),
                rng.choice([1, 4, 5, 17, 100, 4096]), rng.choice([1, 128, 512, 513, 2047, 2048, 2049, 9000, 60000]),
                rng.choice([0, 1, 3, 8, 600]), rng.choice([1, 64, 2500, 9000]), rng.choice([1, 4, 32, 300, 4096])]
        large = size(*most)
        for _ in range(20):
            less = [upto(n) if n else 0 for n in most]
            if rng.random() < 0.2:
                less[4] = 0
            small = size(*less)
            assert small <= large, (most, large, less, small)


def test_workspace_serves_a_shrinking_server():
    """32 requests of up to 2048 tokens, and what is left of them; a long prompt, and a short one."""
    b, cache, batch, _ = structs()
    cache.n_kv_heads, cache.head_dim, cache.token_stride, cache.head_stride = 8, 128, 128, 16 * 128
    cache.page_stride = 8 * 16 * 128
    batch.max_rows, batch.max_kv_len = 1, 2048
    sizes = []
    for n in (32, 31, 8, 1):
        batch.n_seqs = batch.n_rows = n
        sizes.append(workspace(b, cache, batch, 32))
    assert sizes == sorted(sizes, reverse=True), sizes
    batch.n_seqs, batch.max_kv_len, sizes = 1, 8192, []
    for n in (4096, 256, 100, 5):
        batch.n_rows = batch.max_rows = n
        sizes.append(workspace(b, cache, batch, 32))
    assert sizes == sorted(sizes, reverse=True), sizes


def test_tables_without_columns():
    """A page table of no columns has no address: its sequences or prefixes have no tokens."""
    b, cache, batch, rope = structs()
    batch.pages, batch.ldp = None, 0
    n = workspace(b, cache, batch, 4)
    assert attn(b, cache, batch, ws=None, scale=0.0) == b.LORA_E_INVALID
    if n:
        assert attn(b, cache, batch, ws=None) == b.LORA_E_WORKSPACE
    batch.pages, batch.ldp = FAKE, 4
    batch.group_off = batch.prefix_len = FAKE
    batch.prefix_pages, batch.n_groups, batch.ldpp, batch.max_prefix_len, batch.max_group_rows = None, 1, 0, 0, 5
    assert workspace(b, cache, batch, 4) > 0
    assert attn(b, cache, batch, fn="lora_attn_prefix", ws=None) == b.LORA_E_WORKSPACE
    batch.ldpp = 1
    assert attn(b, cache, batch, fn="lora_attn_prefix", ws=None) == b.LORA_E_INVALID


@pytest.mark.parametrize("stride", [1 << 26, 1 << 60, (1 << 62) + 64])
def test_token_strides_past_a_page(stride):
    """Offsets in a page are 32-bit; a stride whose product with the page wraps around is no smaller."""
    b, cache, batch, _ = structs()
    cache.token_stride = stride
    n = ctypes.c_size_t()
    got = b.library().lora_attn_workspace(ctypes.addressof(cache), ctypes.addressof(batch), 4, ctypes.byref(n))
    assert got == b.LORA_E_UNSUPPORTED


def test_more_groups_than_launches_hold():
    """Groups times key heads is a count of workgroups, as sequences times key heads is."""
    b, cache, batch, _ = structs()
    cache.n_kv_heads = 8
    batch.group_off = batch.prefix_len = batch.prefix_pages = FAKE
    batch.ldpp, batch.max_prefix_len, batch.max_group_rows = 4, 60, 5
    n = ctypes.c_size_t()
    for n_groups in ((1 << 27) + 1, 1 << 28, 1 << 30, 2 ** 31 - 1):
        batch.n_groups = n_groups
        got = b.library().lora_attn_workspace(ctypes.addressof(cache), ctypes.addressof(batch), 8, ctypes.byref(n))
        assert got == b.LORA_E_UNSUPPORTED, n_groups
    batch.n_groups = 1 << 20
    assert workspace(b, cache, batch, 8) > 0
