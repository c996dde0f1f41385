"""Paged-cache append and attention against their definitions in 64 bits.

Tolerances.  Attention, with vmax the largest |v|: rounding to bf16 (8
significant bits) moves a value by at most 2^-8 of itself, so the weights'
rounding moves o by at most 2^-8 vmax and o's own by 2^-8 |o|; each is that
large only when every rounding errs fully and one way, and half of their sum
is asked for.  A score's fp32 sum of 64 to 256 products is off by less than
1e-4, which moves o by less than 2e-4 vmax.  So bf16: (2^-8 + 2e-4) vmax.
fp32: only the last kind, typically sqrt(d) 2^-24 of a product's size and not
d times, 5e-5 vmax.  lse: 1e-4.
Append: fp32 products of two terms, 2^-22 of the largest input, plus 2^-8 of
the value (half a unit in the last place of 8 bits) where the result is bf16.
"""
from __future__ import annotations

import math

import pytest
import torch

from _gpu import binding, requires_gpu, say
from _kv import DEV, Case, rotate

pytestmark = [pytest.mark.gpu, requires_gpu]

BF, F32 = torch.bfloat16, torch.float32
O_TOL = {BF: 2.0 ** -8 + 2e-4, F32: 5e-5}


def vmax(c):
    return max([float(x[1].abs().max()) for x in c.own + c.pre if x[1].numel()] + [1e-30])


def check(c, o, lse, ref, what, dtype=None):
    torch.cuda.synchronize()
    ro, rl = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.isfinite(o).all(), f"{what}: o is not finite"
    e = float((o - ro).abs().max()) / vmax(c) if o.numel() else 0.0
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty), f"{what}: rows that see nothing"
    assert bool((lse[empty] < 0).all())
    el = float((lse - rl)[~empty].abs().max()) if bool((~empty).any()) else 0.0
    say(f"  {what}: o {e:.2e} of vmax (tol {O_TOL[dtype or c.dtype]:.1e}), lse {el:.2e}")
    assert e <= O_TOL[dtype or c.dtype], what
    assert el <= 1e-4, what
    return o


def attend(c, window=0, n_sink=0, what="", **kw):
    b = binding()
    cache, batch = c.cache(b), c.batch(b)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lse = torch.full((c.n_rows, c.hq), 7.0, device=DEV)
    o = torch.full((c.n_rows, c.hq * c.d), 7.0, dtype=c.dtype, device=DEV)
    scale = 1.0 / math.sqrt(c.d)
    fn = b.lora_attn_prefix if c.prefix else b.lora_attn_paged
    say(f"{what}: rows {c.nq} tokens {c.kv_len} prefix {c.prefix} heads {c.hq}/{c.hkv} d {c.d} {c.dtype} page {c.page} "
        f"window {window} sinks {n_sink}")
    fn(cache, batch, c.q.to(DEV), scale, window=window, n_sink=n_sink, o=o, lse=lse, status=status, **kw)
    out = check(c, o, lse, c.reference(scale, window, n_sink), what)
    assert int(status.item()) == 0
    return out


LENS = [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 700]


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (BF, 256), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("heads", [(8, 2), (4, 4), (12, 4), (16, 1), (5, 1)], ids=lambda h: f"{h[0]}on{h[1]}")
def test_decode(dtype, d, heads):
    """One row a sequence, lengths on both sides of every tile edge; short batches run a workgroup per head."""
    attend(Case([1] * len(LENS), LENS, *heads, d, dtype, page=16, heads_first=heads[0] % 2 == 0, seed=1), what="shared")
    attend(Case([1] * 7, LENS[:7], *heads, d, dtype, page=32, seed=2), what="short")


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (BF, 256), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("heads", [(8, 2), (12, 4), (20, 1)], ids=lambda h: f"{h[0]}on{h[1]}")
def test_prompts(dtype, d, heads):
    """Prompt rows with and without earlier tokens, beside decode rows and sequences without rows."""
    nq = [1, 70, 0, 3, 17, 130, 1, 64, 4]
    ln = [90, 70, 55, 3, 200, 131, 1, 700, 65]
    attend(Case(nq, ln, *heads, d, dtype, page=16, heads_first=False, seed=3), what="prompts")


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (64, 5), (100, 0), (100, 200), (129, 70), (5000, 3)])
def test_window(dtype, d, window, sinks):
    nq = [1, 1, 1, 80, 5, 1, 33, 1]
    ln = [1, 150, 333, 300, 129, 1000, 33, 64]
    attend(Case(nq, ln, 8, 2, d, dtype, page=8, seed=4), window, sinks, what="window")


def test_long_split():
    """A few long sequences: every workgroup's run starts and ends inside a head."""
    attend(Case([1, 1, 1], [9000, 20, 4100], 8, 2, 128, BF, page=64, seed=5), what="long")
    attend(Case([40, 1], [5000, 3000], 8, 2, 128, BF, page=64, seed=6), what="long prompt pieces")
    attend(Case([40, 1], [5000, 3000], 8, 2, 128, BF, page=64, seed=6), 1500, 9, what="long prompt pieces, window")


# Enough rows for the tiles of 256 columns (they have to fill the card).
WIDE = [
    # rows, own tokens, prefixes, groups, window, sinks
    ([700, 1, 0, 430], [720, 300, 10, 450], None, None, 0, 0),
    ([650, 20, 500], [900, 20, 777], None, None, 200, 5),
    ([600, 1, 550, 2], [600, 40, 570, 9], [130, 333], [0, 2, 4], 0, 0),
    ([600, 1, 550, 2], [600, 40, 570, 9], [130, 333], [0, 2, 4], 250, 70),
    ([1100], [900], [77], [0, 1], 0, 0),     # 200 rows without a place
]


@pytest.mark.parametrize("case", range(len(WIDE)))
@pytest.mark.parametrize("dtype,d,page", [(BF, 128, 16), (BF, 64, 64), (F32, 64, 2)])
def test_wide_tiles(case, dtype, d, page):
    nq, ln, pre, off, window, sinks = WIDE[case]
    c = Case(nq, ln, 64, 8, d, dtype, page=page, heads_first=case % 2 == 0, prefix=pre, group_off=off, seed=30 + case)
    attend(c, window, sinks, what="wide")


@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
def test_wide_tiles_odd_values(bad):
    """A value that is not finite in a tile of 256 columns reaches the rows from its token on, and only those."""
    b = binding()
    c = Case([1100], [1110], 64, 8, 64, BF, seed=36)
    clean = attend(c, what="wide, clean")
    t = 640
    c.cpu_v[c.pages[0][t // 16], t % 16, :, 5] = bad
    say(f"wide, odd value {bad}")
    got = b.lora_attn_paged(c.cache(b), c.batch(b), c.q.to(DEV), 0.125)
    torch.cuda.synchronize()
    got = got.double().cpu()
    sees = t - 10     # row r is at position r + 10
    assert torch.equal(got[:sees], clean[:sees])
    after = got[sees:].view(-1, 64, 64)
    assert not torch.isfinite(after[:, :, 5]).any()
    assert torch.isfinite(after[:, :, :5]).all() and torch.isfinite(after[:, :, 6:]).all()


def test_scores_that_jump():
    """Scores that grow by hundreds from one tile to the next: the softmax's reference has to follow them."""
    for nq, ln, hq, hkv in (([1, 1], [900, 33], 8, 2), ([300], [700], 8, 2), ([1100], [1100], 64, 8)):
        c = Case(nq, ln, hq, hkv, 64, F32, page=64, seed=37)
        for s, pages in enumerate(c.pages):
            k, v = c.own[s]
            up = (1.0 + 4.0 * (torch.arange(ln[s]) // 150)).view(-1, 1, 1)
            k *= up
            for t in range(0, ln[s], c.page):
                m = min(c.page, ln[s] - t)
                c.cpu_k[pages[t // c.page], :m] = k[t:t + m].float()
        b = binding()
        say(f"jumping scores: rows {nq} tokens {ln}")
        lse = torch.empty((c.n_rows, hq), device=DEV)
        o = b.lora_attn_paged(c.cache(b), c.batch(b), c.q.to(DEV), 1.0, lse=lse)
        torch.cuda.synchronize()
        ro, rl = c.reference(1.0)
        # scores of up to about 1000: fp32 sums err by 2^-24 * 64 * 1000 at the very most, 4e-3, and o by twice that
        assert float((lse.double().cpu() - rl).abs().max()) <= 4e-3
        assert float((o.double().cpu() - ro).abs().max()) <= 8e-3 * vmax(c)


@pytest.mark.parametrize("heads", [(20, 1), (34, 2), (64, 2)], ids=lambda h: f"{h[0]}on{h[1]}")
def test_prefix_many_heads_per_key_head(heads):
    """More than 16 query heads on one key head: even one row takes the tiled form, and walks its prefix itself."""
    attend(Case([1, 1, 9, 1], [5, 300, 9, 40], *heads, 64, BF, prefix=[500, 70], group_off=[0, 2, 4], seed=38), what="heads")


def test_prefix_split():
    """A long prefix whose tiles are split among workgroups, for decode rows and beside prompts."""
    attend(Case([1] * 20, [30] * 20, 8, 2, 128, BF, prefix=[9000], group_off=[0, 20], page=64, seed=39), what="split prefix")
    attend(Case([1] * 20 + [40], [30] * 20 + [50], 8, 2, 128, BF, prefix=[9000], group_off=[0, 21], page=64, seed=40),
           what="split prefix beside a prompt")


@pytest.mark.parametrize("page", [1, 2, 4, 128, 1024])
def test_page_sizes(page):
    attend(Case([1, 30, 1], [77, 190, 400], 8, 2, 64, BF, page=page, seed=7), what="page")


@pytest.mark.parametrize("n_seqs", [65, 300, 700])
def test_many_sequences(n_seqs):
    g = torch.Generator().manual_seed(n_seqs)
    ln = torch.randint(1, 400, (n_seqs,), generator=g).tolist()
    nq = [0 if i % 7 == 3 else 1 for i in range(n_seqs)]
    attend(Case(nq, ln, 4, 2, 64, BF, seed=8), what="many")


PREFIX = [
    # rows, own tokens, prefixes, groups
    ([1] * 6, [5, 1, 40, 300, 64, 129], [200], [0, 6]),
    ([1] * 9, [5, 1, 40, 30, 64, 129, 17, 16, 33], [64, 700, 1], [0, 1, 7, 9]),
    ([40, 1, 0, 7, 90], [40, 20, 9, 100, 91], [130, 333], [0, 3, 5]),
    ([1, 1, 20, 1], [300, 30, 20, 400], [0, 77], [0, 1, 3]),        # an empty prefix, a sequence of no group
    ([1] * 40, list(range(1, 41)), [2500], [0, 40]),
]


@pytest.mark.parametrize("case", range(len(PREFIX)))
@pytest.mark.parametrize("dtype,d,heads", [(BF, 128, (8, 2)), (BF, 64, (16, 1)), (F32, 64, (6, 2)), (BF, 256, (4, 2)),
                                           (F32, 128, (4, 1))])
def test_prefix(case, dtype, d, heads):
    nq, ln, pre, off = PREFIX[case]
    c = Case(nq, ln, *heads, d, dtype, prefix=pre, group_off=off, seed=9)
    attend(c, what="prefix")


@pytest.mark.parametrize("case", range(len(PREFIX)))
@pytest.mark.parametrize("window,sinks", [(50, 4), (300, 0), (10, 100)])
def test_prefix_window(case, window, sinks):
    nq, ln, pre, off = PREFIX[case]
    attend(Case(nq, ln, 8, 2, 128, BF, prefix=pre, group_off=off, seed=10), window, sinks, what="prefix, window")


def test_rows_that_see_nothing():
    """More rows than tokens: the first have no place and see nothing, with a prefix too."""
    attend(Case([3, 20, 1], [1, 8, 0], 4, 2, 64, BF, seed=11), what="no place")
    attend(Case([3, 20, 1], [1, 8, 400], 4, 2, 64, BF, prefix=[33], group_off=[0, 3], seed=12), what="no place, prefix")


def test_outputs_and_strides():
    """q and o inside wider tensors; o in the other type; lse not asked for; padding comes back untouched."""
    b = binding()
    c = Case([1, 33, 2], [300, 40, 129], 8, 2, 64, BF, seed=13)
    cache, batch = c.cache(b), c.batch(b)
    scale = 0.125
    ref = c.reference(scale)
    w = c.hq * c.d
    qb = torch.full((c.n_rows, w + 24), float("nan"), dtype=BF, device=DEV)
    qb[:, :w] = c.q.to(DEV)
    for dt in (BF, F32):
        ob = torch.full((c.n_rows, w + 8), 1234.5, dtype=dt, device=DEV)
        say(f"strided, o {dt}")
        b.lora_attn_paged(cache, batch, qb[:, :w], scale, o=ob[:, :w])
        torch.cuda.synchronize()
        assert bool((ob[:, w:] == 1234.5).all())
        e = float((ob[:, :w].double().cpu() - ref[0]).abs().max()) / vmax(c)
        assert e <= (O_TOL[BF] if dt == BF else 2.0 ** -9 + 2e-4)


def test_rows_of_no_sequence():
    """Rows past the last sequence (a padded batch): o and lse stay, q_out is zero."""
    b = binding()
    c = Case([1, 33], [300, 40], 8, 2, 64, BF, seed=14)
    cache, batch = c.cache(b), c.batch(b, extra_rows=5)
    n = c.n_rows + 5
    q = torch.randn((n, 512), device=DEV).to(BF)
    o = torch.full((n, 512), 3.0, dtype=BF, device=DEV)
    lse = torch.full((n, 8), 3.0, device=DEV)
    say("rows of no sequence")
    b.lora_attn_paged(cache, batch, q, 0.125, o=o, lse=lse)
    k = torch.randn((n, 128), device=DEV).to(BF)
    out = b.lora_kv_append(cache, batch, q, k, k)
    torch.cuda.synchronize()
    assert bool((o[c.n_rows:] == 3.0).all()) and bool((lse[c.n_rows:] == 3.0).all())
    assert bool((out[c.n_rows:] == 0).all()) and bool((out[:c.n_rows] == q[:c.n_rows]).all())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("nq", [[1, 1], [3, 2], [60, 90]], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_odd_values_where_masked(dtype, d, nq, bad):
    """A key or value that is not finite reaches the rows that see it, and only those."""
    b = binding()
    ln = [n + 40 for n in nq]
    c = Case(nq, ln, 4, 2, d, dtype, seed=15)
    window, sinks = 30, 2
    clean = attend(c, window, sinks, what="clean")
    at = [ln[0] - 1, 5]      # the last token of sequence 0; token 5 of sequence 1
    for s, t in enumerate(at):
        pg, o = c.pages[s][t // c.page], t % c.page
        c.cpu_v[pg, o, :, 3] = bad
        c.cpu_k[pg, o, 1, 0] = bad
    say(f"odd values: {bad}")
    got = b.lora_attn_paged(c.cache(b), c.batch(b), c.q.to(DEV), 1.0 / math.sqrt(d), window=window, n_sink=sinks)
    torch.cuda.synchronize()
    got = got.double().cpu()
    row = 0
    for s, n in enumerate(nq):
        for j in range(n):
            p = ln[s] - n + j
            t = at[s]
            sees = t <= p and (t > p - window or t < sinks)
            if not sees:
                assert torch.equal(got[row], clean[row]), (s, j)
            else:
                # head pair 0 has finite scores and the odd value in dimension 3
                assert not torch.isfinite(got[row].view(4, d)[:2, 3]).any(), (s, j)
                if bad != bad:
                    assert torch.isnan(got[row].view(4, d)[2:]).all()
                else:
                    assert bool((got[row].view(4, d)[:2, 3] == bad).all())
                assert torch.isfinite(got[row].view(4, d)[:2, :3]).all()
            row += 1


def test_bad_page_numbers():
    """A page number out of range is reported and its tokens are not seen; nothing else changes."""
    b = binding()
    c = Case([1, 20, 1], [200, 60, 500], 8, 2, 64, BF, page=16, seed=16)
    cache = c.cache(b)
    good = b.lora_attn_paged(cache, c.batch(b), c.q.to(DEV), 0.125)
    for wrong in (-1, c.n_pages, 2 ** 31 - 1):
        d = Case([1, 20, 1], [200, 60, 500], 8, 2, 64, BF, page=16, seed=16)
        d.pages[1][1] = wrong          # tokens 16 .. 31 of sequence 1
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        say(f"bad page {wrong}")
        o = b.lora_attn_paged(cache, d.batch(b), c.q.to(DEV), 0.125, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 1
        assert torch.equal(o[:1], good[:1]) and torch.equal(o[21:], good[21:])
        assert torch.isfinite(o).all()
        before = cache.k.clone(), cache.v.clone()
        status.zero_()
        d.pages[1][1], d.pages[1][2] = c.pages[1][1], wrong   # tokens 32 .. 47: not among the rows before 40
        k = torch.randn((22, 128), device=DEV).to(BF)
        b.lora_kv_append(cache, d.batch(b), None, k, k, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 1
        cache.k.copy_(before[0])
        cache.v.copy_(before[1])


def test_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 (and bytes past 2^32)."""
    b = binding()
    c = Case([1, 40], [700, 90], 8, 2, 128, BF, page=16, seed=17)
    n_pages, hkv, page, d = 600000, 2, 16, 128
    say(f"cache of {n_pages * hkv * page * d} elements")
    k = torch.empty((n_pages, hkv, page, d), dtype=BF, device=DEV)
    v = torch.empty_like(k)
    far = torch.arange(n_pages - c.n_pages, n_pages, device=DEV)
    k[far] = c.cpu_k.to(BF).transpose(1, 2).contiguous().to(DEV)
    v[far] = c.cpu_v.to(BF).transpose(1, 2).contiguous().to(DEV)
    assert int(far[0]) * hkv * page * d > 2 ** 31
    c.pages = [[p + n_pages - c.n_pages if p >= 0 else p for p in row] for row in c.pages]
    cache, batch = b.KvCache(k.transpose(1, 2), v.transpose(1, 2)), c.batch(b)
    lse = torch.empty((c.n_rows, 8), device=DEV)
    o = b.lora_attn_paged(cache, batch, c.q.to(DEV), 0.09, lse=lse)
    check(c, o, lse, c.reference(0.09), "far pages")
    new = torch.randn((c.n_rows, hkv * d), device=DEV).to(BF)
    b.lora_kv_append(cache, batch, None, new, new)
    torch.cuda.synchronize()
    t = 699
    assert torch.equal(k[c.pages[0][t // page], :, t % page].reshape(-1), new[0])


def test_repeats_and_streams():
    """The same bits every time, on a stream of its own too."""
    b = binding()
    c = Case([1] * 5 + [50], [3000, 10, 1500, 64, 999, 800], 8, 2, 128, BF, prefix=[500], group_off=[0, 6], seed=18)
    cache, batch, q = c.cache(b), c.batch(b), c.q.to(DEV)
    ws = b.attn_workspace(cache, batch, 8)
    first = b.lora_attn_prefix(cache, batch, q, 0.09, ws=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        ws.fill_(255)   # any content: NaN in every partial result
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o = b.lora_attn_prefix(cache, batch, q, 0.09, ws=ws)
        side.synchronize()
        assert torch.equal(o, first)


def test_graph_replays():
    """Captured append and attention follow in-place changes of the batch's lengths within its bounds."""
    b = binding()
    c = Case([1] * 4, [900, 300, 40, 128], 8, 2, 128, BF, seed=19, spare_pages=8)
    cache, batch, q = c.cache(b), c.batch(b), c.q.to(DEV)
    ws = b.attn_workspace(cache, batch, 8)
    k = torch.randn((4, 256), device=DEV).to(BF)
    q_out, o = torch.empty_like(q), torch.empty_like(q)
    lens = batch.tensors[1]
    ang = torch.randn((1000, 64), device=DEV)
    rope = b.Rope(ang.cos(), ang.sin())

    def step():
        b.lora_kv_append(cache, batch, q, k, k, rope, q_out=q_out)
        b.lora_attn_paged(cache, batch, q_out, 0.09, window=600, n_sink=2, o=o, ws=ws)

    say("graph: eager, capture, replays")
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in ([900, 300, 40, 128], [10, 299, 1, 100], [850, 2, 33, 64]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        step()
        want = o.clone()
        o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), n


# ---- append ----------------------------------------------------------------

@pytest.mark.parametrize("given,kept", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (128, 128, False), (128, 64, True), (64, 32, False),
                                               (128, 128, True), (256, 256, False), (256, 16, True), (128, 48, False)])
def test_append(given, kept, d, rot, interleaved):
    if d == 256 and kept == F32:
        pytest.skip("fp32 caches hold heads of 64 and 128")
    b = binding()
    nq, ln = [1, 0, 17, 1, 64, 3], [40, 9, 17, 1, 300, 3]
    pre, off = [33, 5], [0, 3, 5]
    c = Case(nq, ln, 6, 2, d, kept, page=8, heads_first=rot != 64, prefix=pre, group_off=off, seed=20)
    cache, batch = c.cache(b), c.batch(b)
    g = torch.Generator().manual_seed(21)
    rows = c.n_rows
    x = {n: torch.randn((rows, h * d), generator=g).to(given) for n, h in (("q", 6), ("k", 2), ("v", 2))}
    ang = torch.rand((400, rot // 2), generator=g) * 6.28
    cos, sin = ang.cos(), ang.sin()
    rope = b.Rope(cos.to(DEV), sin.to(DEV), interleaved=interleaved)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    say(f"append {given} into {kept}, d {d} rot {rot} interleaved {interleaved}")
    q = b.lora_kv_append(cache, batch, *(x[n].to(DEV) for n in "qkv"), rope, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want_k, want_v = c.cpu_k.double(), c.cpu_v.double()
    want_q = torch.empty((rows, 6, d), dtype=torch.float64)
    written = torch.zeros((c.n_pages, c.page), dtype=torch.bool)
    row = 0
    for s, n in enumerate(nq):
        grp = c.group_of(s)
        before = 0 if grp is None else pre[grp]
        for j in range(n):
            t = ln[s] - n + j
            cs, sn = cos[before + t].double(), sin[before + t].double()
            want_q[row] = rotate(x["q"][row].double().view(6, d), cs, sn, interleaved)
            pg, at = c.pages[s][t // 8], t % 8
            want_k[pg, at] = rotate(x["k"][row].double().view(2, d), cs, sn, interleaved)
            want_v[pg, at] = x["v"][row].double().view(2, d)
            written[pg, at] = True
            row += 1
    most = max(float(t.abs().max()) for t in x.values())
    tol = 2.0 ** -22 * most * 2

    def near(got, want, what):
        got = got.double().cpu()
        bound = tol + (2.0 ** -8 * want.abs() if kept == BF else 0.0)
        assert bool(((got - want).abs() <= bound).all()), what

    near(q.view(rows, 6, d), want_q, "q")
    gk, gv = cache.k.cpu(), cache.v.cpu()
    near(gk[written], want_k[written], "k")
    near(gv[written], want_v[written], "v")
    # every other token keeps its bits (NaN where nothing was)
    for got, was in ((gk, c.cpu_k), (gv, c.cpu_v)):
        was = was.to(kept)
        assert torch.equal(torch.nan_to_num(got[~written].float(), 77.0), torch.nan_to_num(was[~written].float(), 77.0))


def test_append_in_place_and_strided():
    """q rotated where it lies; q, k and v as column slices of one wider projection."""
    b = binding()
    c = Case([1, 30], [77, 30], 4, 2, 64, BF, page=16, seed=22)
    cache, batch = c.cache(b), c.batch(b)
    wide = torch.randn((31, 4 * 64 + 2 * 128 + 8), device=DEV).to(BF)
    keep = wide.clone()
    q, k, v = wide[:, :256], wide[:, 256:384], wide[:, 384:512]
    ang = torch.rand((100, 32), device=DEV)
    rope = b.Rope(ang.cos(), ang.sin())
    say("append in place")
    want = b.lora_kv_append(cache, batch, q, k, v, rope)
    got = b.lora_kv_append(cache, batch, q, k, v, rope, q_out=q)
    torch.cuda.synchronize()
    assert got.data_ptr() == wide.data_ptr() and torch.equal(got, want)
    assert torch.equal(wide[:, 256:], keep[:, 256:])


def test_append_refuses_places():
    """Positions past the tables or the page table, and more rows than tokens: reported, not written."""
    b = binding()
    for nq, ln, n_pos, bad_rows in (([2], [20], 19, [1]), ([3], [1], 50, [0, 1])):
        c = Case(nq, ln, 2, 1, 64, BF, page=16, seed=23)
        cache, batch = c.cache(b), c.batch(b)
        before = cache.k.clone()
        ang = torch.rand((n_pos, 32), device=DEV)
        x = torch.randn((c.n_rows, 128), device=DEV).to(BF)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        say(f"append without a place: rows {nq} tokens {ln} positions {n_pos}")
        q = b.lora_kv_append(cache, batch, x, x[:, :64], x[:, :64], b.Rope(ang.cos(), ang.sin()), status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 1
        for r in range(c.n_rows):
            assert bool((q[r] == 0).all()) == (r in bad_rows)
        changed = (torch.nan_to_num(cache.k.float(), 7.0) != torch.nan_to_num(before.float(), 7.0)).any(-1).sum()
        assert int(changed) == c.n_rows - len(bad_rows)


def test_empty_batch():
    b = binding()
    c = Case([0, 0], [10, 20], 4, 2, 64, BF, seed=24)
    cache, batch = c.cache(b), c.batch(b)
    q = torch.empty((0, 256), dtype=BF, device=DEV)
    say("no rows")
    b.lora_kv_append(cache, batch, q, q[:, :128], q[:, :128])
    o = b.lora_attn_paged(cache, batch, q, 0.125)
    torch.cuda.synchronize()
    assert o.shape == (0, 256)


# rows and own tokens of the sequences of one group: one row alone (a sequence whose row sits some tokens behind the
# prefix), a few rows, enough for the tiled form, and a prompt beside a decode row
ODD_PREFIX = [([1], [9]), ([1], [3]), ([1, 1], [40, 3]), ([1] * 30, [3, 9] * 15), ([1, 25], [9, 60])]


@pytest.mark.parametrize("case", range(len(ODD_PREFIX)))
@pytest.mark.parametrize("dtype,d,heads", [(BF, 128, (2, 2)), (BF, 64, (8, 2)), (BF, 64, (32, 2)), (F32, 64, (4, 2))])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_odd_values_in_a_prefix(case, dtype, d, heads, window, sinks, bad):
    """A key or value of a shared prefix that is not finite reaches the rows whose window holds it, and only those."""
    b = binding()
    nq, ln = ODD_PREFIX[case]
    hq, hkv = heads
    n, t = 200, 155
    c = Case(nq, ln, hq, hkv, d, dtype, prefix=[n], group_off=[0, len(nq)], seed=41)
    clean = attend(c, window, sinks, what="clean prefix")
    pg, at = c.prefix_pages[0][t // c.page], t % c.page
    c.cpu_v[pg, at, :, 3] = bad
    c.cpu_k[pg, at, 1, 0] = bad
    say(f"odd values in a prefix: {bad}")
    got = b.lora_attn_prefix(c.cache(b), c.batch(b), c.q.to(DEV), 1.0 / math.sqrt(d), window=window, n_sink=sinks)
    torch.cuda.synchronize()
    got = got.double().cpu()
    row = 0
    for s, rows in enumerate(nq):
        for j in range(rows):
            p = n + ln[s] - rows + j
            x = got[row].view(hkv, -1, d)
            if window and t <= p - window:
                assert torch.equal(got[row], clean[row]), (s, j)
            else:
                # the heads of key head 0 have finite scores and the odd value in dimension 3
                assert not torch.isfinite(x[0, :, 3]).any(), (s, j)
                assert torch.isfinite(x[0, :, :3]).all() and torch.isfinite(x[0, :, 4:]).all(), (s, j)
            row += 1


def test_one_workspace_for_a_shrinking_batch():
    """The workspace of a server's largest batch serves its smaller ones; nothing is written past its size."""
    b = binding()
    hq, hkv, d = 32, 8, 64

    def case(n, seed):
        return Case([1] * n + [30], [2000 - 40 * i for i in range(n)] + [700], hq, hkv, d, BF, page=64, seed=seed)

    c = case(33, 42)
    need = b.lora_attn_workspace(c.cache(b), c.batch(b), hq)
    whole = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    for n in (33, 31, 5, 1):
        for window in (0, 900):
            attend(case(n, 42 + n), window, 3 if window else 0, what=f"{n} decode rows and a prompt", ws=whole[:need])
            assert bool((whole[need:] == 0xA5).all())


def test_tables_without_columns():
    """All prefixes empty, or all sequences: a page table of no columns."""
    b = binding()
    c = Case([1, 20, 1], [30, 40, 9], 8, 2, 64, BF, prefix=[0, 0], group_off=[0, 2, 3], table_pad=0, seed=43)
    assert c.batch(b).tensors[5].shape == (2, 0)
    attend(c, what="empty prefixes")
    attend(c, 7, 2, what="empty prefixes, window")
    c = Case([1, 20, 0], [0, 0, 0], 8, 2, 64, BF, table_pad=0, seed=44)
    assert c.batch(b).tensors[2].shape == (3, 0)
    attend(c, what="no tokens")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    k = torch.randn((21, 128), device=DEV).to(BF)
    out = b.lora_kv_append(c.cache(b), c.batch(b), c.q.to(DEV), k, k, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 1 and bool((out == 0).all())


# a few columns in whole heads and in shares, the tiled form, its wide tiles
ROWS_AND_TOKENS = [([1], [300]), ([1, 1], [1500, 40]), ([300], [700]), ([1100], [1100])]


@pytest.mark.parametrize("case", range(len(ROWS_AND_TOKENS)))
@pytest.mark.parametrize("prefix", [None, [90]], ids=str)
@pytest.mark.parametrize("scale", [1e-36, 3e-38, 1e-40])
def test_scale_near_zero(case, prefix, scale):
    """Scores of next to nothing: every visible token weighs the same."""
    b = binding()
    nq, ln = ROWS_AND_TOKENS[case]
    c = Case(nq, ln, 64, 8, 64, F32, page=64, prefix=prefix, group_off=prefix and [0, len(nq)], seed=45)
    say(f"scale {scale}: rows {nq} tokens {ln} prefix {prefix}")
    lse = torch.empty((c.n_rows, c.hq), device=DEV)
    fn = b.lora_attn_prefix if prefix else b.lora_attn_paged
    o = fn(c.cache(b), c.batch(b), c.q.to(DEV), scale, lse=lse)
    check(c, o, lse, c.reference(scale), "scale near zero")


@pytest.mark.parametrize("case", range(len(ROWS_AND_TOKENS)))
@pytest.mark.parametrize("prefix", [None, [90]], ids=str)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("factor", [1e3, 1e4, 3e4, 1e6, 1e8])
def test_scores_without_bound(case, prefix, dtype, factor):
    """Scores up to 1e18: a row is the value of its highest score.

    Rows count whose two highest scores are further apart than fp32 sums of 64 products can move them, 64 * 2^-24 of
    |q| |k| each, and than the softmax has weight for (40).  Their o is one value times a weight over itself: in bf16
    the weight and o are rounded, 2^-8 each, in fp32 2^-22 covers it.  lse is the score.
    """
    b = binding()
    nq, ln = ROWS_AND_TOKENS[case]
    d, hq, hkv, scale = 64, 64, 8, 0.125
    c = Case(nq, ln, hq, hkv, d, dtype, page=64, prefix=prefix, group_off=prefix and [0, len(nq)], seed=46)
    c.q = (c.q.float() * factor).to(dtype)
    for k, pages in [(x[0], p) for x, p in zip(c.own + c.pre, c.pages + c.prefix_pages)]:
        k *= factor
        for t in range(0, len(k), c.page):
            m = min(c.page, len(k) - t)
            c.cpu_k[pages[t // c.page], :m] = k[t:t + m].float()
    say(f"scores without bound: factor {factor} rows {nq} tokens {ln} prefix {prefix} {dtype}")
    lse = torch.empty((c.n_rows, hq), device=DEV)
    fn = b.lora_attn_prefix if prefix else b.lora_attn_paged
    o = fn(c.cache(b), c.batch(b), c.q.to(DEV), scale, lse=lse)
    torch.cuda.synchronize()
    o, lse = o.double().cpu().view(-1, hq, d), lse.double().cpu()
    q, row, counted, rows = c.q.double().view(-1, hq, d), 0, 0, 0
    for s, n in enumerate(nq):
        k, v = (torch.cat((c.pre[0][i], c.own[s][i])) if prefix else c.own[s][i] for i in (0, 1))
        k, v = k.double(), v.double()
        hidden = torch.arange(len(k)) > torch.arange(len(k) - n, len(k))[:, None]
        for h in range(hq):
            qh, kh, vh = q[row:row + n, h], k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
            x = (torch.matmul(qh, kh.t()) * scale).masked_fill(hidden, -math.inf)
            top, at = x.topk(min(2, len(k)), -1)
            moved = 2 * 64 * 2.0 ** -24 * scale * qh.norm(dim=-1) * kh.norm(dim=-1).max()
            far = top[:, 0] - top[:, -1] > moved + 40
            counted, rows = counted + int(far.sum()), rows + n
            want, got = vh[at[:, 0]][far], o[row:row + n, h][far]
            bound = (2.0 ** -7 if dtype == BF else 2.0 ** -22) * want.abs() + 1e-30
            assert bool(((got - want).abs() <= bound).all()), (s, h)
            assert bool(((lse[row:row + n, h] - top[:, 0]).abs() <= moved + 1e-6 * top[:, 0].abs())[far].all()), (s, h)
        row += n
    say(f"  {counted} of {rows} rows and heads")
    assert counted > 0.9 * rows


@pytest.mark.parametrize("rows", [1, 2, 30])
def test_pages_behind_every_window(rows):
    """Prefix pages that every row's window has left may have any number: status stays 0."""
    b = binding()
    n, own, window = 200, 40, 50      # positions 239 on: tokens 190 on are seen
    c = Case([1] * rows, [own + i for i in range(rows)], 8, 2, 64, BF, page=16, prefix=[n], group_off=[0, rows], seed=47)
    q, status = c.q.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    for sinks in (0, 3):
        want = attend(c, window, sinks, what="windows past a prefix's pages")
        for page, needed in ((10, False), (9, False), (1, False), (12, True), (0, sinks > 0)):
            d = Case([1] * rows, c.kv_len, 8, 2, 64, BF, page=16, prefix=[n], group_off=[0, rows], seed=47)
            d.prefix_pages[0][page] = -1
            status.zero_()
            say(f"rows {rows} sinks {sinks} page {page}")
            o = b.lora_attn_prefix(c.cache(b), d.batch(b), q, 0.125, window=window, n_sink=sinks, status=status)
            torch.cuda.synchronize()
            assert int(status.item()) == int(needed), (page, sinks)
            if not needed:
                assert torch.equal(o.double().cpu(), want)
