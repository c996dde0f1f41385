"""Caches in 8 bits and step tables for the tests: definitions in 64 bits on the CPU (no code of the library)."""
from __future__ import annotations

import torch

from _kv import DEV, Case, rotate

LEAST, MOST = -100, 100
# e4m3: the magnitudes of codes 0 .. 126, from the format's definition
VALUES = torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127],
                      dtype=torch.float64)
BETWEEN = (VALUES[1:] + VALUES[:-1]) / 2


def codes_of(x):
    """float64 -> e4m3 codes (uint8), to nearest, ties to the even code, past 448 the largest; NaN for what is not finite."""
    a = x.abs()
    at = torch.bucketize(a, BETWEEN)                       # borders below a
    tie = BETWEEN[at.clamp(max=BETWEEN.numel() - 1)] == a
    at = at + (tie & (at % 2 == 1)).long()
    at = torch.where(torch.isfinite(x), at, 127)
    return (at + 128 * torch.signbit(x)).to(torch.uint8)


def values_of(codes):
    mag = torch.cat((VALUES, torch.tensor([float("nan")], dtype=torch.float64)))[(codes & 127).long()]
    return torch.where(codes >= 128, -mag, mag)


def exponent_for(top):
    """The least e in [LEAST, MOST] with top <= 448 * 2^e (a number)."""
    for e in range(LEAST, MOST):
        if top <= 448.0 * 2.0 ** e:
            return e
    return MOST


def largest(x):
    """Of the finite elements of x [tokens, d]."""
    x = x.abs()[torch.isfinite(x)]
    return float(x.max()) if x.numel() else 0.0


class CaseQ8(Case):
    """A Case whose tokens are numbers that a cache in 8 bits holds.  What is not a token holds NaN, and so do the
    scales of blocks without tokens."""

    def __init__(self, nq, kv_len, hq, hkv, d, page=16, block=None, grow=0.0, **kw):
        super().__init__(nq, kv_len, hq, hkv, d, torch.bfloat16, page=page, **kw)
        self.block = block or page
        shape = (self.n_pages, page // self.block, hkv)
        self.codes, self.scales = [], []
        g = torch.Generator().manual_seed(kw.get("seed", 0) + 1000)
        for x in (self.cpu_k, self.cpu_v):
            b = x.double().view(self.n_pages, -1, self.block, hkv, d)
            b = b * torch.exp2(torch.round(grow * torch.randn((self.n_pages, 1, 1, hkv, 1), generator=g, dtype=torch.float64)))
            top = torch.nan_to_num(b, 0.0).abs().amax((2, 4))
            e = torch.tensor([exponent_for(float(t)) for t in top.reshape(-1)]).view(shape)
            s = torch.tensor([2.0 ** int(i) for i in e.reshape(-1)], dtype=torch.float64).view(shape)
            q = codes_of(b / s[:, :, None, :, None])
            used = ~torch.isnan(b).all(-1).all(-1).all(-1)
            self.codes.append(q.view(x.shape))
            self.scales.append(torch.where(used[:, :, None], s, float("nan")))
        self.reread()

    def reread(self):
        """The tokens as the pages hold them now."""
        k, v = (values_of(q) * s.repeat_interleave(self.block, 1)[..., None] for q, s in zip(self.codes, self.scales))
        self.cpu_k, self.cpu_v = k, v

        def tokens(lens, pages):
            out = []
            for n, pg in zip(lens, pages):
                idx = torch.tensor(pg[:-(-n // self.page)], dtype=torch.long)
                out.append(tuple(x[idx].reshape(-1, self.hkv, self.d)[:n] for x in (k, v)))
            return out

        self.own, self.pre = tokens(self.kv_len, self.pages), tokens(self.prefix, self.prefix_pages)

    def cache(self, b):
        def dev(x):
            if self.heads_first:
                return x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
            return x.contiguous().to(DEV)
        k, v = (dev(x.view(torch.float8_e4m3fn)) for x in self.codes)
        return b.KvCacheQ8(k, v, *(dev(s.float()) for s in self.scales))


def append(c, x, rope=None, n_pos=1 << 30):
    """Appends the rows x = {"k", "v"} [rows, hkv * d] of the step to the CPU copy of case c's cache, block by block, and
    returns the rows that have a place.  rope: (cos, sin, interleaved)."""
    starts, placed = c.starts(), []
    for s, (n, length) in enumerate(zip(c.nq, c.kv_len)):
        grp = c.group_of(s)
        before = 0 if grp is None else c.prefix[grp]
        first = length - n
        fresh = {}
        for t in range(max(first, 0), length):
            row = starts[s] + t - first
            if before + t >= n_pos:
                continue
            k, v = (x[i][row].double().view(c.hkv, c.d) for i in "kv")
            if rope:
                k = rotate(k, rope[0][before + t].double(), rope[1][before + t].double(), rope[2])
            fresh[t] = (k, v)
            placed.append(row)
        for t0 in sorted({t // c.block * c.block for t in fresh}):
            pg, at = c.pages[s][t0 // c.page], t0 % c.page
            for i in (0, 1):
                for h in range(c.hkv):
                    new = {t: y[i][h] for t, y in fresh.items() if t0 <= t < t0 + c.block}
                    e = exponent_for(max(largest(y) for y in new.values()))
                    code, scale = c.codes[i], c.scales[i]
                    if first > t0:
                        was = scale[pg, at // c.block, h].clone()
                        e = max(e, int(torch.frexp(was)[1]) - 1)
                        old = slice(at, at + first - t0)
                        code[pg, old, h] = codes_of(values_of(code[pg, old, h]) * (was / 2.0 ** e))
                    for t, y in new.items():
                        code[pg, at + t - t0, h] = codes_of(y / 2.0 ** e)
                    scale[pg, at // c.block, h] = 2.0 ** e
    return placed


def plan(new_rows, adapter, kv_len, pages, free, n_free, page, max_rows, prefix=None, group_off=None, max_free=None):
    """A step's tables from their definition: a dict of lists."""
    length, pages, wide = list(kv_len), [list(p) for p in pages], len(pages[0]) if pages else 0
    stack = list(free[:n_free])
    for s, n in enumerate(new_rows):
        if n < 0:
            stack += pages[s][:-(-length[s] // page)]
            length[s] = 0
    status = 0
    room = len(free) if max_free is None else max_free
    if len(stack) > room:
        stack, status = stack[:room], 2
    there, rows, off, asked_rows, asked_pages = len(stack), [], [0], 0, 0
    for s, n in enumerate(new_rows):
        if n > 0 and length[s] + n > wide * page:
            status |= 1
        elif n > 0:
            held, need = -(-length[s] // page), -(-(length[s] + n) // page)
            asked_rows, asked_pages = asked_rows + n, asked_pages + need - held
            if asked_rows > max_rows or (need > held and asked_pages > there):
                status |= 1
            else:
                for j in range(held, need):
                    pages[s][j] = stack.pop()
                before = 0
                for g in range(len(prefix or [])):
                    if group_off[g] <= s < group_off[g + 1]:
                        before = prefix[g]
                for t in range(length[s], length[s] + n):
                    rows.append((s, adapter[s] if adapter else -1, before + t, pages[s][t // page] * page + t % page))
                length[s] += n
        off.append(len(rows))
    rows += [(-1, -1, -1, -1)] * (max_rows - len(rows))
    return dict(row_off=off, row_seq=[r[0] for r in rows], row_adapter=[r[1] for r in rows], row_pos=[r[2] for r in rows],
                row_slot=[r[3] for r in rows], kv_len=length, pages=pages, free=stack + list(free[len(stack):]),
                n_free=len(stack), status=status)
