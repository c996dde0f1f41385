"""What append writes to a cache in 8 bits, against rationals: rotated keys whose exact value lies next to a tie of two
numbers, or next to the border of two scales, by far less than 53 bits tell; and rows past the batch's bound.  Every
number has to be the same."""
from __future__ import annotations

from fractions import Fraction

import pytest
import torch

import _kv_q8
from _gpu import binding, requires_gpu, say
from _kv import DEV
from _kv_q8 import CaseQ8

pytestmark = [pytest.mark.gpu, requires_gpu]

CODES = [Fraction(float(v)) for v in _kv_q8.VALUES]


def code_of(x):
    """The nearest number's code: of two equally near ones the even one."""
    a = min(abs(x), CODES[-1])
    lo, hi = 0, len(CODES) - 1
    while lo < hi:   # the last one that is no more than a
        m = (lo + hi + 1) // 2
        lo, hi = (m, hi) if CODES[m] <= a else (lo, m - 1)
    if lo + 1 < len(CODES):
        below, above = a - CODES[lo], CODES[lo + 1] - a
        lo += above < below or (above == below and lo % 2 == 1)
    return lo + (128 if x < 0 else 0)


def exponent_for(top):
    return next(e for e in range(_kv_q8.LEAST, _kv_q8.MOST + 1) if top <= 448 * Fraction(2) ** e)


def crafted(d, interleaved, top_by):
    """Four keys of one head and their angles: pairs whose rotation is a tie plus or minus 2^-44 to 2^-86, in the first
    or in the second of the pair, and one that is 448 + top_by."""
    half = d // 2
    k, cos, sin = torch.zeros((4, d)), torch.ones((4, half)), torch.zeros((4, half))
    ties = [float(t) for t in _kv_q8.BETWEEN if 2.0 ** -5 < t < 400]
    n = 0
    for t in range(4):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            if i == 1:
                # 448 * 1 - b * sin
                k[t, a], k[t, b] = 448.0, 2.0 ** -40 if top_by else 0.0
                sin[t, i] = -top_by * 2.0 ** 40
                continue
            tie, gap = ties[(7 * n) % len(ties)], 44 + n % 43
            small = 2.0 ** (20 - gap)
            if n % 3 == 2:
                tie = -tie
            k[t, a], k[t, b] = (tie, small) if n % 2 == 0 else (small, tie)
            sin[t, i] = 2.0 ** -20 if (n // 2) % 2 == 0 else -2.0 ** -20
            n += 1
    return k, cos, sin


def rotated(k, cos, sin, interleaved):
    d, half = k.shape[1], cos.shape[1]
    out = []
    for t in range(k.shape[0]):
        y = [Fraction(0)] * d
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            p, q, c, s = (Fraction(float(x)) for x in (k[t, a], k[t, b], cos[t, i], sin[t, i]))
            y[a], y[b] = p * c - q * s, p * s + q * c
        out.append(y)
    return out


@pytest.mark.parametrize("given", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,page,block", [(64, 16, 4), (128, 32, 32), (256, 128, 128), (128, 64, 64)])
@pytest.mark.parametrize("top_by", [0.0, 2.0 ** -60, -2.0 ** -60])
def test_next_to_ties_and_borders(given, interleaved, d, page, block, top_by):
    b = binding()
    k, cos, sin = crafted(d, interleaved, top_by)
    assert torch.equal(k.to(given).float(), k)
    c = CaseQ8([4], [4], 1, 1, d, page=page, block=block, seed=50)
    cache = c.cache(b)
    say(f"next to ties: {given} interleaved {interleaved} d {d} block {block} largest 448 + {top_by}")
    x = k.to(given).to(DEV)
    b.lora_kv_append_q8(cache, c.batch(b), None, x, x, b.Rope(cos.to(DEV), sin.to(DEV), interleaved=interleaved))
    torch.cuda.synchronize()
    y = rotated(k, cos, sin, interleaved)
    e = exponent_for(max(abs(v) for r in y for v in r))
    assert e == (1 if top_by > 0 else 0)
    pg = c.pages[0][0]
    assert float(cache.k_scale[pg, 0, 0]) == 2.0 ** e
    want = torch.tensor([[code_of(v / Fraction(2) ** e) for v in r] for r in y], dtype=torch.uint8)
    got = cache.k.view(torch.uint8)[pg, :4, 0].cpu()
    far = (got != want).nonzero().tolist()
    assert not far, [(t, i, float(y[t][i]), int(got[t, i]), int(want[t, i])) for t, i in far[:5]]


@pytest.mark.parametrize("page,block", [(16, 4), (8, 1), (16, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("most", [0, 1, 3])
@pytest.mark.parametrize("with_q", [False, True])
def test_rows_past_the_bound(page, block, most, with_q):
    """max_rows below what sequences bring: rows that have no room for it are reported and the others written, all of
    them with a bound of more than a row."""
    b = binding()
    c = CaseQ8([3, 1, 0, 90, 2], [17, 4, 7, 95, 129], 4, 2, 64, page=page, block=block, seed=51)
    cache, full = c.cache(b), c.batch(b)
    batch = b.KvBatch(*full.tensors[:3], c.n_rows, most, max(c.kv_len))
    g = torch.Generator().manual_seed(52)
    x = {i: torch.randn((c.n_rows, 128), generator=g).to(torch.bfloat16) for i in "kv"}
    q = torch.randn((c.n_rows, 256), generator=g).to(torch.bfloat16).to(DEV) if with_q else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    say(f"rows past a bound of {most}: page {page} block {block}")
    out = b.lora_kv_append_q8(cache, batch, q, x["k"].to(DEV), x["v"].to(DEV), status=status)
    torch.cuda.synchronize()
    before = [[t.clone() for t in y] for y in (c.codes, c.scales)]
    assert _kv_q8.append(c, x) == list(range(c.n_rows))
    lost, starts = 0, c.starts()
    for s, (n, length) in enumerate(zip(c.nq, c.kv_len)):
        room = starts[s + 1] // block - starts[s] // block + (1 if most <= 1 else 2)
        for t0 in list(range((length - n) // block * block, length, block))[room:] if n else []:
            pg, at = c.pages[s][t0 // page], t0 % page
            lost += 1
            for i in (0, 1):
                c.codes[i][pg, at:at + block] = before[0][i][pg, at:at + block]
                c.scales[i][pg, at // block] = before[1][i][pg, at // block]
    assert int(status.item()) == (1 if lost else 0)
    assert bool(lost) == (most <= 1 and block > 1)
    for i, name in enumerate("kv"):
        got, want = getattr(cache, name).view(torch.uint8).cpu(), c.codes[i]
        nan = (want & 127) == 127
        assert torch.equal((got & 127) == 127, nan) and torch.equal(got[~nan], want[~nan]), name
        scales = getattr(cache, name + "_scale").double().cpu()
        assert torch.equal(torch.nan_to_num(scales, 7.0), torch.nan_to_num(c.scales[i], 7.0)), name
    assert q is None or torch.equal(out, q)
