"""Attention over long and split rows, with a bound per element that a lost or exchanged tile cannot hide under.

With p the softmax's weights of a row in 64 bits, rounding the weights to bf16 moves element d of o by sum_k p_k e_k v_kd,
|e_k| <= 2^-8 and of either sign: at most 2^-8 sqrt(12) |p v_d| for up to 12 keys, and six standard deviations for more
(a rounding error even over its range has 1 / sqrt(3) of it).  A bf16 o rounds by 2^-8 |o|.  fp32 sums of up to 128
products of unit normals are off by some 4e-6, times the scale 1/8 to 1/11, and exp2 by 2^-23: 2^-17 sum p |v| covers both.
"""
from __future__ import annotations

import math

import pytest
import torch

from _gpu import binding, requires_gpu, say
from _kv import DEV, Case

BF, F32 = torch.bfloat16, torch.float32

CASES = {
    # rows, own tokens, heads, d, page, prefixes, groups, window, sinks
    "decode in shares": ([1, 1, 1], [9000, 20, 4100], (8, 2), 128, 64, None, None, 0, 0),
    "decode in shares, window": ([1, 1, 1], [9000, 20, 4100], (8, 2), 128, 64, None, None, 3000, 5),
    "decode in whole heads": ([1] * 33, [1000 + 30 * i for i in range(33)], (32, 8), 64, 16, None, None, 0, 0),
    "split prompt pieces": ([40, 1], [5000, 3000], (8, 2), 128, 64, None, None, 0, 0),
    "split prompt pieces, window": ([40, 1], [5000, 3000], (8, 2), 128, 64, None, None, 1500, 9),
    "split prefix": ([1] * 20, [30] * 20, (8, 2), 128, 64, [9000], [0, 20], 0, 0),
    "split prefix, window": ([1] * 20, [30] * 20, (8, 2), 128, 64, [9000], [0, 20], 4000, 70),
    "prefix in shares": ([1, 1], [300, 4000], (8, 2), 64, 32, [7000, 90], [0, 1, 2], 0, 0),
    "split prefix beside a prompt": ([1] * 20 + [40], [30] * 20 + [50], (8, 2), 128, 64, [9000], [0, 21], 0, 0),
    "wide tiles": ([700, 1, 430], [1720, 300, 1450], (64, 8), 64, 16, None, None, 0, 0),
}


def case_of(name, dtype):
    nq, ln, heads, d, page, pre, off, window, sinks = CASES[name]
    return Case(nq, ln, *heads, d, dtype, page=page, prefix=pre, group_off=off, seed=50), window, sinks


def long_reference(c, window, sinks, dtype, values=lambda v: v):
    """(o, bound of its error, lse) in float64; ``values`` may plant a mistake in a sequence's values."""
    hq, share, d, scale = c.hq, c.hq // c.hkv, c.d, 1.0 / math.sqrt(c.d)
    o, bound = (torch.zeros((c.n_rows, hq, d), dtype=torch.float64) for _ in range(2))
    lse = torch.zeros((c.n_rows, hq), dtype=torch.float64)
    q, row = c.q.double().view(-1, hq, d), 0
    for s, n in enumerate(c.nq):
        g = c.group_of(s)
        k, v = (x if g is None else torch.cat((y, x)) for x, y in zip(c.own[s], c.pre[g] if g is not None else (0, 0)))
        k, v = k.double(), values(v.double())
        at, key = torch.arange(len(k) - n, len(k))[:, None], torch.arange(len(k))
        hidden = key > at
        if window:
            hidden |= (key <= at - window) & (key >= sinks)
        for h in range(hq):
            x = (torch.matmul(q[row:row + n, h], k[:, h // share].t()) * scale).masked_fill(hidden, -math.inf)
            lse[row:row + n, h] = torch.logsumexp(x, -1)
            p, vh = torch.softmax(x, -1), v[:, h // share]
            out = torch.matmul(p, vh)
            o[row:row + n, h] = out
            fp32 = 2.0 ** -17 * torch.matmul(p, vh.abs())
            bf16 = 2.0 ** -8 * (math.sqrt(12) * torch.matmul(p * p, vh * vh).sqrt() + out.abs())
            bound[row:row + n, h] = fp32 + (bf16 if dtype == BF else 0)
        row += n
    return o, bound, lse


@pytest.mark.gpu
@requires_gpu
@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_rows(name, dtype):
    b = binding()
    c, window, sinks = case_of(name, dtype)
    say(f"{name} {dtype}")
    lse = torch.empty((c.n_rows, c.hq), device=DEV)
    fn = b.lora_attn_prefix if c.prefix else b.lora_attn_paged
    o = fn(c.cache(b), c.batch(b), c.q.to(DEV), 1.0 / math.sqrt(c.d), window=window, n_sink=sinks, lse=lse)
    torch.cuda.synchronize()
    want, bound, want_lse = long_reference(c, window, sinks, dtype)
    over = ((o.double().cpu().view(want.shape) - want).abs() / bound).max()
    say(f"  largest error {float(over):.3f} of its bound, lse {float((lse.double().cpu() - want_lse).abs().max()):.1e}")
    assert over <= 1
    assert float((lse.double().cpu() - want_lse).abs().max()) <= 1e-4


@pytest.mark.parametrize("name", ["decode in shares", "split prompt pieces", "prefix in shares"])
def test_the_bound_tells(name):
    """Mistakes planted in the reference: a unit of 128 keys lost, two exchanged, one key's value of another token."""
    c, window, sinks = case_of(name, BF)
    want, bound, _ = long_reference(c, window, sinks, BF)

    def over(values):
        got, _, _ = long_reference(c, window, sinks, BF, values)
        return float(((got - want).abs() / bound).max())

    def lost(v):
        return torch.cat((v[:128] * 0, v[128:])) if len(v) > 2000 else v

    def exchanged(v):
        return torch.cat((v[128:256], v[:128], v[256:])) if len(v) > 2000 else v

    def shifted(v):
        return torch.cat((v[:256], v[255:-1])) if len(v) > 2000 else v

    for mistake in (lost, exchanged, shifted):
        assert over(mistake) > 3, mistake.__name__
