"""Append to and attention over a cache in 8 bits against their definitions in 64 bits.

Tolerances.  A number of the cache (4 significant bits times a power of two) is a bf16 number, and a power of two
that goes into a weight instead changes none of its bits, so attention rounds where it does over a bf16 cache: the
weights by at most 2^-8 of themselves and o by 2^-8 |o|, each that much only when every rounding errs fully and one
way, and half of their sum is asked for; a score's fp32 sum moves o by less than 2e-4 of the largest |v|.  So (2^-8 +
2e-4) vmax, and 1e-4 for lse.  What append writes is compared bit by bit: it rounds a value once, from 64 bits, and
ties are decided by that value.
"""
from __future__ import annotations

import math

import pytest
import torch

import _kv_q8
from _gpu import binding, requires_gpu, say
from _kv import DEV, rotate
from _kv_q8 import CaseQ8

pytestmark = [pytest.mark.gpu, requires_gpu]

BF, F32 = torch.bfloat16, torch.float32
O_TOL = 2.0 ** -8 + 2e-4


def vmax(c):
    return max([float(x[1].abs().max()) for x in c.own + c.pre if x[1].numel()] + [1e-30])


def attend(c, window=0, n_sink=0, what="", scale=None, ref=None, **kw):
    b = binding()
    cache, batch = c.cache(b), c.batch(b)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lse = torch.full((c.n_rows, c.hq), 7.0, device=DEV)
    o = torch.full((c.n_rows, c.hq * c.d), 7.0, dtype=BF, device=DEV)
    scale = scale or 1.0 / math.sqrt(c.d)
    say(f"{what}: rows {c.nq} tokens {c.kv_len} prefix {c.prefix} heads {c.hq}/{c.hkv} d {c.d} page {c.page} "
        f"block {c.block} window {window} sinks {n_sink}")
    fn = b.lora_attn_prefix_q8 if c.prefix else b.lora_attn_paged_q8
    fn(cache, batch, c.q.to(DEV), scale, window=window, n_sink=n_sink, o=o, lse=lse, status=status, **kw)
    torch.cuda.synchronize()
    ro, rl = ref or c.reference(scale, window, n_sink)
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.isfinite(o).all(), f"{what}: o is not finite"
    e = float((o - ro).abs().max()) / vmax(c) if o.numel() else 0.0
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty), f"{what}: rows that see nothing"
    assert bool((lse[empty] < 0).all())
    el = float((lse - rl)[~empty].abs().max()) if bool((~empty).any()) else 0.0
    say(f"  {what}: o {e:.2e} of vmax (tol {O_TOL:.1e}), lse {el:.2e}")
    assert e <= O_TOL, what
    assert el <= 1e-4, what
    assert int(status.item()) == 0
    return o


LENS = [1, 2, 31, 32, 33, 63, 64, 65, 255, 256, 257, 511, 700]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [(8, 2), (4, 4), (12, 4), (16, 1), (5, 1)], ids=lambda h: f"{h[0]}on{h[1]}")
def test_decode(d, heads):
    """One row a sequence, lengths on both sides of every edge; whole heads per workgroup, and shares of long ones."""
    attend(CaseQ8([1] * len(LENS), LENS, *heads, d, page=16, heads_first=heads[0] % 2 == 0, seed=1), what="decode")
    attend(CaseQ8([1] * 3, [1, 2600, 1300], *heads, d, page=32, block=8, seed=2), what="long")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [(8, 2), (12, 4), (20, 1)], ids=lambda h: f"{h[0]}on{h[1]}")
def test_prompts(d, heads):
    nq = [1, 70, 0, 3, 17, 130, 1, 64, 4]
    ln = [90, 70, 55, 3, 200, 131, 1, 700, 65]
    attend(CaseQ8(nq, ln, *heads, d, page=16, heads_first=False, seed=3), what="prompts")


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (64, 5), (100, 0), (100, 200), (129, 70), (5000, 3)])
def test_window(d, window, sinks):
    nq = [1, 1, 1, 80, 5, 1, 33, 1]
    ln = [1, 150, 333, 300, 129, 1000, 33, 64]
    attend(CaseQ8(nq, ln, 8, 2, d, page=8, block=4, seed=4), window, sinks, what="window")


def test_long_split():
    """A few long sequences: every workgroup's run starts and ends inside a head; prompt pieces that are split."""
    attend(CaseQ8([1, 1, 1], [9000, 20, 4100], 8, 2, 128, page=64, seed=5), what="long")
    attend(CaseQ8([40, 1], [5000, 3000], 8, 2, 128, page=64, seed=6), what="long prompt pieces")
    attend(CaseQ8([40, 1], [5000, 3000], 8, 2, 128, page=64, seed=6), 1500, 9, what="long prompt pieces, window")


WIDE = [
    # rows, own tokens, prefixes, groups, window, sinks: enough rows for the tiles of 256 columns
    ([700, 1, 0, 430], [720, 300, 10, 450], None, None, 0, 0),
    ([650, 20, 500], [900, 20, 777], None, None, 200, 5),
    ([600, 1, 550, 2], [600, 40, 570, 9], [130, 333], [0, 2, 4], 0, 0),
    ([600, 1, 550, 2], [600, 40, 570, 9], [130, 333], [0, 2, 4], 250, 70),
    ([1100], [900], [77], [0, 1], 0, 0),     # 200 rows without a place
]


@pytest.mark.parametrize("case", range(len(WIDE)))
@pytest.mark.parametrize("d,page,block", [(128, 16, 16), (64, 64, 16), (64, 2, 1)])
def test_wide_tiles(case, d, page, block):
    nq, ln, pre, off, window, sinks = WIDE[case]
    c = CaseQ8(nq, ln, 64, 8, d, page=page, block=block, heads_first=case % 2 == 0, prefix=pre, group_off=off, seed=30 + case)
    attend(c, window, sinks, what="wide")


@pytest.mark.parametrize("page,block", [(1, 1), (2, 2), (4, 1), (16, 2), (128, 128), (1024, 64), (256, 1)])
def test_pages_and_blocks(page, block):
    attend(CaseQ8([1, 30, 1], [77, 190, 400], 8, 2, 64, page=page, block=block, grow=3.0, seed=7, k_div=20.0), what="blocks")


@pytest.mark.parametrize("n_seqs", [65, 300, 700])
def test_many_sequences(n_seqs):
    g = torch.Generator().manual_seed(n_seqs)
    ln = torch.randint(1, 400, (n_seqs,), generator=g).tolist()
    nq = [0 if i % 7 == 3 else 1 for i in range(n_seqs)]
    attend(CaseQ8(nq, ln, 4, 2, 64, seed=8), what="many")


PREFIX = [
    # rows, own tokens, prefixes, groups
    ([1] * 6, [5, 1, 40, 300, 64, 129], [200], [0, 6]),
    ([1] * 9, [5, 1, 40, 30, 64, 129, 17, 16, 33], [64, 700, 1], [0, 1, 7, 9]),
    ([40, 1, 0, 7, 90], [40, 20, 9, 100, 91], [130, 333], [0, 3, 5]),
    ([1, 1, 20, 1], [300, 30, 20, 400], [0, 77], [0, 1, 3]),        # an empty prefix, a sequence of no group
    ([1] * 40, list(range(1, 41)), [2500], [0, 40]),
    ([1] * 20, [30] * 20, [9000], [0, 20]),
    ([1, 1, 9, 1], [5, 300, 9, 40], [500, 70], [0, 2, 4]),
]


@pytest.mark.parametrize("case", range(len(PREFIX)))
@pytest.mark.parametrize("d,heads", [(128, (8, 2)), (64, (16, 1)), (256, (4, 2)), (64, (20, 1))])
def test_prefix(case, d, heads):
    nq, ln, pre, off = PREFIX[case]
    attend(CaseQ8(nq, ln, *heads, d, prefix=pre, group_off=off, page=64 if pre[0] > 1000 else 16, seed=9), what="prefix")


@pytest.mark.parametrize("case", range(len(PREFIX)))
@pytest.mark.parametrize("window,sinks", [(50, 4), (300, 0), (10, 100)])
def test_prefix_window(case, window, sinks):
    nq, ln, pre, off = PREFIX[case]
    attend(CaseQ8(nq, ln, 8, 2, 128, prefix=pre, group_off=off, seed=10), window, sinks, what="prefix, window")


def test_rows_that_see_nothing():
    attend(CaseQ8([3, 20, 1], [1, 8, 0], 4, 2, 64, seed=11), what="no place")
    attend(CaseQ8([3, 20, 1], [1, 8, 400], 4, 2, 64, prefix=[33], group_off=[0, 3], seed=12), what="no place, prefix")


@pytest.mark.parametrize("nq,ln,heads", [([1] * 5, [300, 40, 1, 700, 2000], (32, 8)), ([200, 1], [300, 90], (8, 2)),
                                         ([1100], [1100], (64, 8))], ids=["few", "tiles", "wide"])
def test_like_a_bf16_cache(nq, ln, heads):
    """The same numbers in a bf16 cache: rows differ by the order of sums alone, at most a rounding or two of o."""
    b = binding()
    c = CaseQ8(nq, ln, *heads, 128, grow=2.0, k_div=8.0, seed=13)
    got = attend(c, what="8 bits")
    cache = b.KvCache(*(torch.nan_to_num(x, 0.0).to(BF).to(DEV) for x in (c.cpu_k, c.cpu_v)))
    want = b.lora_attn_paged(cache, c.batch(b), c.q.to(DEV), 1.0 / math.sqrt(128))
    torch.cuda.synchronize()
    assert float((got - want.double().cpu()).abs().max()) <= O_TOL * vmax(c)


@pytest.mark.parametrize("power", [-90, 60])
@pytest.mark.parametrize("nq", [[1, 1], [60, 90], [1100]], ids=["few", "tiles", "wide"])
def test_large_and_small_scales(power, nq):
    """Values (keys the other way) of far powers of two, next to the ends of what a scale can be."""
    ln = [n + 40 for n in nq]
    c = CaseQ8(nq, ln, 64, 8, 64, block=8, seed=14)
    c.scales[1] *= 2.0 ** power
    c.scales[0] *= 2.0 ** (-power / 2)
    c.q = (c.q.float() * 2.0 ** (power / 2)).to(BF)
    c.reread()
    attend(c, what="far scales")


def test_only_the_exponent_of_a_scale_counts():
    b = binding()
    c = CaseQ8([1, 50], [300, 90], 8, 2, 64, block=4, seed=15)
    want = attend(c, what="powers of two")
    cache = c.cache(b)
    for s in (cache.k_scale, cache.v_scale):
        s.mul_(1.0 + 0.999 * torch.rand_like(s))
    say("other scales")
    got = b.lora_attn_paged_q8(cache, c.batch(b), c.q.to(DEV), 0.125)
    torch.cuda.synchronize()
    assert torch.equal(got.double().cpu(), want)


def test_outputs_and_strides():
    """q and o inside wider tensors; o in fp32; lse not asked for; padding comes back untouched."""
    b = binding()
    c = CaseQ8([1, 33, 2], [300, 40, 129], 8, 2, 64, seed=16)
    cache, batch = c.cache(b), c.batch(b)
    ref = c.reference(0.125)
    w = c.hq * c.d
    qb = torch.full((c.n_rows, w + 24), float("nan"), dtype=BF, device=DEV)
    qb[:, :w] = c.q.to(DEV)
    for dt in (BF, F32):
        ob = torch.full((c.n_rows, w + 8), 1234.5, dtype=dt, device=DEV)
        say(f"strided, o {dt}")
        b.lora_attn_paged_q8(cache, batch, qb[:, :w], 0.125, o=ob[:, :w])
        torch.cuda.synchronize()
        assert bool((ob[:, w:] == 1234.5).all())
        e = float((ob[:, :w].double().cpu() - ref[0]).abs().max()) / vmax(c)
        assert e <= (O_TOL if dt == BF else 2.0 ** -9 + 2e-4)


def test_strided_cache():
    """Pages inside wider rows, scales a slice of a larger table."""
    b = binding()
    c = CaseQ8([1, 40], [300, 90], 6, 3, 64, page=16, block=4, heads_first=False, seed=17)
    n, page, hkv, d = c.cpu_k.shape
    wide = torch.zeros((2, n, page, 2 * hkv * d + 32), dtype=torch.uint8, device=DEV)
    wide.fill_(0x7f)
    table = torch.full((2, hkv + 2, n, page // 4 + 3), float("nan"), device=DEV)
    parts = []
    for i in (0, 1):
        view = wide[i, :, :, 16:16 + hkv * d].unflatten(2, (hkv, d))
        view.copy_(c.codes[i].to(DEV))
        s = table[i, 1:1 + hkv, :, 2:2 + page // 4].permute(1, 2, 0)
        s.copy_(c.scales[i].float().to(DEV))
        parts.append((view.view(torch.float8_e4m3fn), s))
    cache = b.KvCacheQ8(parts[0][0], parts[1][0], parts[0][1], parts[1][1])
    say("strided cache")
    o = b.lora_attn_paged_q8(cache, c.batch(b), c.q.to(DEV), 0.125)
    torch.cuda.synchronize()
    assert float((o.double().cpu() - c.reference(0.125)[0]).abs().max()) <= O_TOL * vmax(c)
    x = {i: torch.randn((41, hkv * d)).to(BF) for i in "kv"}
    keep = wide.clone(), table.clone()
    b.lora_kv_append_q8(cache, c.batch(b), None, x["k"].to(DEV), x["v"].to(DEV))
    torch.cuda.synchronize()
    _kv_q8.append(c, x)
    for i in (0, 1):
        same_bits(parts[i][0].view(torch.uint8).cpu(), c.codes[i], "codes")
        assert torch.equal(torch.nan_to_num(parts[i][1].cpu(), 7.0), torch.nan_to_num(c.scales[i].float(), 7.0))
        wide[i, :, :, 16:16 + hkv * d] = keep[0][i, :, :, 16:16 + hkv * d]
        table[i, 1:1 + hkv, :, 2:2 + page // 4] = keep[1][i, 1:1 + hkv, :, 2:2 + page // 4]
    assert torch.equal(wide, keep[0]) and torch.equal(torch.nan_to_num(table, 7.0), torch.nan_to_num(keep[1], 7.0))


def test_rows_of_no_sequence():
    b = binding()
    c = CaseQ8([1, 33], [300, 40], 8, 2, 64, seed=18)
    cache, batch = c.cache(b), c.batch(b, extra_rows=5)
    n = c.n_rows + 5
    q = torch.randn((n, 512), device=DEV).to(BF)
    o = torch.full((n, 512), 3.0, dtype=BF, device=DEV)
    lse = torch.full((n, 8), 3.0, device=DEV)
    say("rows of no sequence")
    b.lora_attn_paged_q8(cache, batch, q, 0.125, o=o, lse=lse)
    k = torch.randn((n, 128), device=DEV).to(BF)
    out = b.lora_kv_append_q8(cache, batch, q, k, k)
    torch.cuda.synchronize()
    assert bool((o[c.n_rows:] == 3.0).all()) and bool((lse[c.n_rows:] == 3.0).all())
    assert bool((out[c.n_rows:] == 0).all()) and bool((out[:c.n_rows] == q[:c.n_rows]).all())


@pytest.mark.parametrize("d", [128, 64, 256])
@pytest.mark.parametrize("nq", [[1, 1], [3, 2], [60, 90], [600, 530]], ids=str)
@pytest.mark.parametrize("bad", [0x7f, 0xff])
def test_nan_where_masked(d, nq, bad):
    """A key or value that is NaN reaches the rows that see it, and only those."""
    b = binding()
    ln = [n + 40 for n in nq]
    hq = 64 if nq[0] > 500 else 4
    c = CaseQ8(nq, ln, hq, hq // 2 if hq == 4 else 8, d, seed=19)
    window, sinks = 30, 2
    clean = attend(c, window, sinks, what="clean")
    at = [ln[0] - 1, 5]      # the last token of sequence 0; token 5 of sequence 1
    for s, t in enumerate(at):
        pg, o = c.pages[s][t // c.page], t % c.page
        c.codes[1][pg, o, :, 3] = bad
        c.codes[0][pg, o, 1, 0] = bad
    say("NaN where masked")
    got = b.lora_attn_paged_q8(c.cache(b), c.batch(b), c.q.to(DEV), 1.0 / math.sqrt(d), window=window, n_sink=sinks)
    torch.cuda.synchronize()
    got, row = got.double().cpu(), 0
    for s, n in enumerate(nq):
        for j in range(n):
            p, t = ln[s] - n + j, at[s]
            x = got[row].view(c.hkv, -1, d)
            if not (t <= p and (t > p - window or t < sinks)):
                assert torch.equal(got[row], clean[row]), (s, j)
            else:
                assert torch.isnan(x[0, :, 3]).all() and torch.isnan(x[1]).all(), (s, j)
                assert torch.isfinite(x[0, :, :3]).all() and torch.isfinite(x[0, :, 4:]).all(), (s, j)
            row += 1


@pytest.mark.parametrize("nq,ln", [([1], [9]), ([1, 1], [40, 3]), ([1] * 30, [3, 9] * 15), ([1, 25], [9, 60])],
                         ids=["one", "two", "thirty", "prompt"])
@pytest.mark.parametrize("d,heads", [(128, (2, 2)), (64, (8, 2)), (64, (32, 2))])
def test_nan_in_a_prefix(nq, ln, d, heads):
    b = binding()
    n, t, window = 200, 155, 50
    c = CaseQ8(nq, ln, *heads, d, prefix=[n], group_off=[0, len(nq)], seed=20)
    clean = attend(c, window, 2, what="clean prefix")
    c.codes[1][c.prefix_pages[0][t // c.page], t % c.page, :, 3] = 0x7f
    say("NaN in a prefix")
    got = b.lora_attn_prefix_q8(c.cache(b), c.batch(b), c.q.to(DEV), 1.0 / math.sqrt(d), window=window, n_sink=2)
    torch.cuda.synchronize()
    got, row = got.double().cpu(), 0
    for s, rows in enumerate(nq):
        for j in range(rows):
            p = n + ln[s] - rows + j
            if t <= p - window:
                assert torch.equal(got[row], clean[row]), (s, j)
            else:
                x = got[row].view(-1, d)
                assert torch.isnan(x[:, 3]).all() and torch.isfinite(x[:, :3]).all() and torch.isfinite(x[:, 4:]).all()
            row += 1


def test_bad_page_numbers():
    b = binding()

    def case():
        return CaseQ8([1, 20, 1], [200, 60, 500], 8, 2, 64, page=16, seed=21)

    c = case()
    good = b.lora_attn_paged_q8(c.cache(b), c.batch(b), c.q.to(DEV), 0.125)
    for wrong in (-1, c.n_pages, 2 ** 31 - 1):
        d = case()
        d.pages[1][1] = wrong          # tokens 16 .. 31 of sequence 1
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        say(f"bad page {wrong}")
        o = b.lora_attn_paged_q8(c.cache(b), d.batch(b), c.q.to(DEV), 0.125, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 1
        assert torch.equal(o[:1], good[:1]) and torch.equal(o[21:], good[21:])
        assert torch.isfinite(o).all()
        status.zero_()
        d.pages[1][1], d.pages[1][3] = c.pages[1][1], wrong   # tokens 48 on, among the rows from 40 on
        k = torch.randn((22, 128), device=DEV).to(BF)
        out = b.lora_kv_append_q8(c.cache(b), d.batch(b), c.q.to(DEV), k, k, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 1
        gone = (out == 0).all(1).nonzero()[:, 0].tolist()
        assert gone == list(range(1 + 8, 1 + 20))


def test_offsets_past_32_bits():
    """Pages whose bytes lie past 2^32."""
    b = binding()
    c = CaseQ8([1, 40], [700, 90], 8, 2, 128, page=16, seed=22)
    n_pages, hkv, page, d = 1200000, 2, 16, 128
    say(f"cache of {n_pages * hkv * page * d} bytes")
    k = torch.empty((n_pages, hkv, page, d), dtype=torch.uint8, device=DEV)
    v = torch.empty_like(k)
    far = torch.arange(n_pages - c.n_pages, n_pages, device=DEV)
    k[far], v[far] = (x.transpose(1, 2).contiguous().to(DEV) for x in c.codes)
    ks, vs = (torch.zeros((n_pages, 1, hkv), device=DEV) for _ in range(2))
    ks[far], vs[far] = (x.float().to(DEV) for x in c.scales)
    assert int(far[0]) * hkv * page * d > 2 ** 32
    c.pages = [[p + n_pages - c.n_pages if p >= 0 else p for p in row] for row in c.pages]
    cache = b.KvCacheQ8(*(x.view(torch.float8_e4m3fn).transpose(1, 2) for x in (k, v)), ks, vs)
    batch = c.batch(b)
    o = b.lora_attn_paged_q8(cache, batch, c.q.to(DEV), 0.09)
    torch.cuda.synchronize()
    assert float((o.double().cpu() - c.reference(0.09)[0]).abs().max()) <= O_TOL * vmax(c)
    new = torch.randn((c.n_rows, hkv * d), device=DEV).to(BF)
    b.lora_kv_append_q8(cache, batch, None, new, new)
    torch.cuda.synchronize()
    pg, at = c.pages[0][699 // page], 699 % page
    got = _kv_q8.values_of(k[pg, :, at].cpu()) * ks[pg, 0].double().cpu()[:, None]
    assert float((got - new[0].double().cpu().view(hkv, d)).abs().max()) <= 2.0 ** -4 * 6


def test_repeats_and_streams():
    b = binding()
    c = CaseQ8([1] * 5 + [50], [3000, 10, 1500, 64, 999, 800], 8, 2, 128, prefix=[500], group_off=[0, 6], seed=23)
    cache, batch, q = c.cache(b), c.batch(b), c.q.to(DEV)
    ws = b.attn_workspace_q8(cache, batch, 8)
    first = b.lora_attn_prefix_q8(cache, batch, q, 0.09, ws=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        ws.fill_(255)   # any content: NaN in every partial result
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o = b.lora_attn_prefix_q8(cache, batch, q, 0.09, ws=ws)
        side.synchronize()
        assert torch.equal(o, first)


def test_one_workspace_for_a_shrinking_batch():
    b = binding()

    def case(n, seed):
        return CaseQ8([1] * n + [30], [2000 - 40 * i for i in range(n)] + [700], 32, 8, 64, page=64, seed=seed)

    c = case(33, 42)
    need = b.lora_attn_workspace_q8(c.cache(b), c.batch(b), 32)
    whole = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    for n in (33, 31, 5, 1):
        for window in (0, 900):
            attend(case(n, 42 + n), window, 3 if window else 0, what=f"{n} decode rows and a prompt", ws=whole[:need])
            assert bool((whole[need:] == 0xA5).all())


def test_tables_without_columns():
    b = binding()
    c = CaseQ8([1, 20, 1], [30, 40, 9], 8, 2, 64, prefix=[0, 0], group_off=[0, 2, 3], table_pad=0, seed=24)
    attend(c, what="empty prefixes")
    c = CaseQ8([1, 20, 0], [0, 0, 0], 8, 2, 64, table_pad=0, seed=25)
    attend(c, what="no tokens")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    k = torch.randn((21, 128), device=DEV).to(BF)
    out = b.lora_kv_append_q8(c.cache(b), c.batch(b), c.q.to(DEV), k, k, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 1 and bool((out == 0).all())


def test_empty_batch():
    b = binding()
    c = CaseQ8([0, 0], [10, 20], 4, 2, 64, seed=26)
    q = torch.empty((0, 256), dtype=BF, device=DEV)
    say("no rows")
    b.lora_kv_append_q8(c.cache(b), c.batch(b), q, q[:, :128], q[:, :128])
    assert b.lora_attn_paged_q8(c.cache(b), c.batch(b), q, 0.125).shape == (0, 256)
    torch.cuda.synchronize()


@pytest.mark.parametrize("nq,ln,prefix", [([1, 1], [1500, 40], None), ([300], [700], [90]), ([1100], [1100], None)],
                         ids=["few", "tiles", "wide"])
def test_scores_that_jump(nq, ln, prefix):
    """Scores that grow by hundreds from one block to the next, and a scale of next to nothing.

    Keys are up to 448, 110 in the mean, so scores spread by 8 * 110 and stay below 4096: each of 64 fp32 additions
    errs by at most half a unit there, 2^-12, 1.6e-2 in all; lse's own rounding adds one, and a weight moves by twice
    as much at the most."""
    hq, hkv = (64, 8) if len(nq) == 1 else (8, 2)
    c = CaseQ8(nq, ln, hq, hkv, 64, page=64, prefix=prefix, group_off=prefix and [0, len(nq)], seed=27)
    for pages in c.pages + c.prefix_pages:
        for j, pg in enumerate(pages):
            if 0 <= pg < c.n_pages:
                c.scales[0][pg] = 2.0 ** (j % 7 - 6)
    c.reread()
    b = binding()
    fn = b.lora_attn_prefix_q8 if prefix else b.lora_attn_paged_q8
    lse = torch.empty((c.n_rows, hq), device=DEV)
    say("jumping scores")
    o = fn(c.cache(b), c.batch(b), c.q.to(DEV), 1.0, lse=lse)
    torch.cuda.synchronize()
    ro, rl = c.reference(1.0)
    assert float((lse.double().cpu() - rl).abs().max()) <= 1.7e-2
    assert float((o.double().cpu() - ro).abs().max()) <= (O_TOL + 3.4e-2) * vmax(c)
    attend(c, what="scale of next to nothing", scale=1e-38)


# ---- append ----------------------------------------------------------------

def same_bits(got, want, what):
    """Codes that stand for the same number (NaN has two)."""
    nan = (got & 127) == 127
    assert torch.equal(nan, (want & 127) == 127), f"{what}: NaN"
    assert torch.equal(got[~nan], want[~nan]), f"{what}: {int((got[~nan] != want[~nan]).sum())} codes differ"


def check_append(c, cache, what):
    for i, name in enumerate(("k", "v")):
        same_bits(getattr(cache, name).view(torch.uint8).cpu(), c.codes[i], f"{what}: {name}")
        got, want = getattr(cache, name + "_scale").double().cpu(), c.scales[i]
        assert torch.equal(torch.nan_to_num(got, 7.0), torch.nan_to_num(want, 7.0)), f"{what}: scales of {name}"


def rope_of(b, n_pos, rot, interleaved, seed=0):
    g = torch.Generator().manual_seed(seed)
    ang = torch.rand((n_pos, rot // 2), generator=g) * 6.28
    cos, sin = ang.cos(), ang.sin()
    return (cos, sin, interleaved), b.Rope(cos.to(DEV), sin.to(DEV), interleaved=interleaved)


@pytest.mark.parametrize("given", [BF, F32])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (128, 128, False), (128, 64, True), (64, 32, False),
                                               (128, 128, True), (256, 256, False), (256, 16, True), (128, 48, False)])
@pytest.mark.parametrize("page,block", [(8, 8), (16, 4), (64, 32), (128, 64)])
def test_append(given, d, rot, interleaved, page, block):
    b = binding()
    nq, ln = [1, 0, 17, 1, 64, 3, 150], [40, 9, 17, 1, 300, 3, 190]
    c = CaseQ8(nq, ln, 6, 2, d, page=page, block=block, heads_first=rot != 64, prefix=[33, 5], group_off=[0, 3, 5], seed=30)
    cache, batch = c.cache(b), c.batch(b)
    g = torch.Generator().manual_seed(31)
    # rows of many sizes: some raise their block's scale and some do not
    size = torch.exp2(torch.round(2 * torch.randn((c.n_rows, 1), generator=g)))
    x = {n: (torch.randn((c.n_rows, h * d), generator=g) * size).to(given) for n, h in (("q", 6), ("k", 2), ("v", 2))}
    tables, rope = rope_of(b, 400, rot, interleaved)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    say(f"append {given} in 8 bits, d {d} rot {rot} interleaved {interleaved} page {page} block {block}")
    q = b.lora_kv_append_q8(cache, batch, *(x[n].to(DEV) for n in "qkv"), rope, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert _kv_q8.append(c, x, tables) == list(range(c.n_rows))
    check_append(c, cache, "append")
    row, starts = 0, c.starts()
    for s, n in enumerate(nq):
        before = 0 if c.group_of(s) is None else c.prefix[c.group_of(s)]
        for j in range(n):
            p = before + ln[s] - n + j
            want = rotate(x["q"][row].double().view(6, d), tables[0][p].double(), tables[1][p].double(), interleaved)
            err = (q[row].double().cpu().view(6, d) - want).abs()
            assert bool((err <= 2.0 ** -8 * want.abs() + 2.0 ** -21 * float(x["q"][row].abs().max())).all())
            row += 1


@pytest.mark.parametrize("d,page,block", [(64, 1, 1), (64, 16, 16), (128, 16, 16), (128, 64, 2), (256, 128, 128),
                                          (256, 32, 1), (64, 128, 128)])
def test_tokens_one_by_one(d, page, block):
    """Decode steps that fill and open blocks; every few steps a larger token scales the ones before it again."""
    b = binding()
    g = torch.Generator().manual_seed(d + block)
    start, steps = [0, 5, block - 1, 30], 9
    c = CaseQ8([1] * 4, start, 2, 2, d, page=page, block=block, seed=32, spare_pages=256, table_pad=1 + steps // page + 1)
    spare = [p for p in range(c.n_pages) if p not in {x for r in c.pages for x in r}]
    for r in c.pages:
        for j, p in enumerate(r):
            if p < 0:
                r[j] = spare.pop()
    cache = c.cache(b)
    c.kv_len = list(start)
    batch = b.KvBatch(torch.arange(5, dtype=torch.int32, device=DEV), torch.tensor(start, dtype=torch.int32, device=DEV),
                      torch.tensor(c.pages, dtype=torch.int32, device=DEV), 4, 1, 200)
    tables, rope = rope_of(b, 200, d, False)
    say(f"tokens one by one: d {d} page {page} block {block}")
    for i in range(steps):
        batch.tensors[1].add_(1)
        c.kv_len = [n + 1 for n in c.kv_len]
        size = torch.exp2(torch.round(3 * torch.randn((4, 1), generator=g)))
        x = {n: (torch.randn((4, 2 * d), generator=g) * size).to(BF) for n in "kv"}
        b.lora_kv_append_q8(cache, batch, None, x["k"].to(DEV), x["v"].to(DEV), rope)
        torch.cuda.synchronize()
        _kv_q8.append(c, x, tables)
        check_append(c, cache, f"step {i}")


@pytest.mark.parametrize("given", [BF, F32])
def test_ties_and_borders(given):
    """Values half way between two numbers, a largest one next to 448 times a power of two, the least and the largest."""
    b = binding()
    d, block = 64, 4
    x = torch.zeros((5, 4, d), dtype=torch.float64)
    for i in range(4):
        x[0, i] = torch.cat((_kv_q8.BETWEEN[i * 31:i * 31 + 31], -_kv_q8.BETWEEN[i * 31:i * 31 + 31], torch.tensor([448.0, -0.0])))
    near = {BF: 2.0 ** -8, F32: 2.0 ** -23}[given]
    x[1] = torch.rand((4, d), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    for i, top in enumerate((448.0, 448.0 * (1 + 2 * near), 448.0 * (1 - near), 1.75 * 2.0 ** -20)):
        x[1, i] *= top * 0.4
        x[1, i, 7] = top
    x[2] = torch.tensor([0.0, 1e-38, 2.0 ** -110, 2.0 ** -109, 1.5 * 2.0 ** -109, 3e-33, -2.0 ** -105, 1e-30] * 8)
    x[3] = torch.tensor([1.0, -3e38, 1e35, 448.0 * 2.0 ** 100, 2.0 ** 91, 2.0 ** 108, -1e33, 0.0] * 8)
    x[4] = torch.tensor([1.0, float("inf"), -float("inf"), float("nan"), 2.0, 3.0, -5.0, 0.1] * 8)
    x[4, 1] = float("nan")
    say(f"ties and borders {given}")
    for which in range(5):
        for alone in (False, True):   # all four tokens of a block at once, and one by one
            c = CaseQ8([4], [4], 1, 1, d, page=16, block=block, seed=33)
            if alone:
                c.nq, c.n_rows = [1], 1
            cache, batch = c.cache(b), c.batch(b)
            rows = x[which].to(given)
            for t in range(4 if alone else 1):
                part = rows[t:t + 1] if alone else rows
                batch.tensors[1].fill_(t + 1 if alone else 4)
                c.kv_len = [t + 1 if alone else 4]
                b.lora_kv_append_q8(cache, batch, None, part.to(DEV).contiguous(), part.to(DEV).contiguous())
                torch.cuda.synchronize()
                _kv_q8.append(c, {"k": part, "v": part})
                check_append(c, cache, f"row {which}, {'one by one' if alone else 'at once'} {t}")


def test_rotation_of_large_values():
    """Products past fp32's range, infinities and NaN: the first saturate, the others become NaN, nothing else changes."""
    b = binding()
    c = CaseQ8([3], [3], 1, 1, 64, page=16, block=4, seed=34)
    cache, batch = c.cache(b), c.batch(b)
    k = torch.ones((3, 64))
    k[0, 5], k[0, 37] = 3.3e38, -3.3e38
    k[1, 1], k[2, 40] = float("inf"), float("nan")
    tables, rope = rope_of(b, 8, 64, False, seed=3)
    say("large rotations")
    b.lora_kv_append_q8(cache, batch, None, k.to(DEV), k.to(DEV), rope)
    torch.cuda.synchronize()
    _kv_q8.append(c, {"k": k, "v": k}, tables)
    check_append(c, cache, "large")


def test_append_in_place_and_strided():
    """q rotated where it lies; q, k and v as column slices of one wider projection."""
    b = binding()
    c = CaseQ8([1, 30], [77, 30], 4, 2, 64, page=16, seed=35)
    batch = c.batch(b)
    wide = torch.randn((31, 4 * 64 + 2 * 128 + 8), device=DEV).to(BF)
    keep = wide.clone()
    q, k, v = wide[:, :256], wide[:, 256:384], wide[:, 384:512]
    tables, rope = rope_of(b, 100, 64, False)
    cache = c.cache(b)
    say("append in place")
    want = b.lora_kv_append_q8(cache, batch, q, k, v, rope)
    got = b.lora_kv_append_q8(c.cache(b), batch, q, k, v, rope, q_out=q)
    torch.cuda.synchronize()
    assert got.data_ptr() == wide.data_ptr() and torch.equal(got, want)
    assert torch.equal(wide[:, 256:], keep[:, 256:])
    _kv_q8.append(c, {"k": k.cpu(), "v": v.cpu()}, tables)
    check_append(c, cache, "strided")


def test_append_refuses_places():
    """Positions past the tables and more rows than tokens: reported, not written; the other rows are."""
    b = binding()
    for nq, ln, n_pos, placed in (([2], [20], 19, [0]), ([3], [1], 50, [2]), ([6], [20], 17, [0, 1, 2])):
        c = CaseQ8(nq, ln, 2, 1, 64, page=16, block=8, seed=36)
        cache, batch = c.cache(b), c.batch(b)
        x = torch.randn((c.n_rows, 128)).to(BF)
        tables, rope = rope_of(b, n_pos, 64, False)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        say(f"append without a place: rows {nq} tokens {ln} positions {n_pos}")
        k = x[:, :64].contiguous()
        for q in (x.to(DEV), None):
            status.zero_()
            cache = c.cache(b)
            out = b.lora_kv_append_q8(cache, batch, q, k.to(DEV), k.to(DEV), rope, status=status)
            torch.cuda.synchronize()
            assert int(status.item()) == 1
            if q is not None:
                assert [r for r in range(c.n_rows) if not bool((out[r] == 0).all())] == placed
        assert _kv_q8.append(c, {"k": k, "v": k}, tables, n_pos) == placed
        check_append(c, cache, "places")


@pytest.mark.parametrize("nq,ln", [([3], [0]), ([1, 2], [5, 0]), ([2, 1], [-4, 9])], ids=str)
def test_rows_of_a_sequence_without_tokens(nq, ln):
    """No row of it has a place: reported, with queries and without, and nothing of the cache changes for it."""
    b = binding()
    for with_q in (True, False):
        c = CaseQ8(nq, [max(n, 0) for n in ln], 2, 1, 64, page=16, block=8, seed=38)
        cache, batch = c.cache(b), c.batch(b)
        batch.tensors[1].copy_(torch.tensor(ln, dtype=torch.int32))
        x = torch.randn((c.n_rows, 128)).to(BF)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        say(f"rows {nq} of sequences of {ln} tokens, {'q' if with_q else 'no q'}")
        k = x[:, :64].contiguous()
        b.lora_kv_append_q8(cache, batch, x.to(DEV) if with_q else None, k.to(DEV), k.to(DEV), status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 1
        _kv_q8.append(c, {"k": k, "v": k})
        check_append(c, cache, "no tokens")


def test_many_idle_sequences():
    """The blocks' numbering skips sequences without rows, and a batch whose bound is one row."""
    b = binding()
    g = torch.Generator().manual_seed(40)
    for most in (1, 40):
        nq = [int(torch.randint(0, 2, (1,), generator=g)) * int(torch.randint(1, most + 1, (1,), generator=g)) for _ in range(300)]
        ln = [n + int(torch.randint(0, 40, (1,), generator=g)) for n in nq]
        c = CaseQ8(nq, ln, 2, 1, 64, page=16, block=8, seed=37)
        cache, batch = c.cache(b), c.batch(b)
        x = {n: torch.randn((c.n_rows, 64), generator=g).to(BF) for n in "kv"}
        say(f"idle sequences, at most {most} rows")
        b.lora_kv_append_q8(cache, batch, None, x["k"].to(DEV), x["v"].to(DEV))
        torch.cuda.synchronize()
        _kv_q8.append(c, x)
        check_append(c, cache, "idle")
