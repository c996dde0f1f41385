"""Paged-cache batches for the tests, and the operators' definitions in 64 bits on the CPU (no code of the library)."""
from __future__ import annotations

import math

import torch

DEV = "cuda"


class Case:
    """A cache, a batch and its tensors.  Tokens of every sequence are kept
    dense on the CPU too (``own_k[s]`` [len, hkv, d] and so on), so that the
    reference never looks at a page.  Unused tokens of the cache hold NaN."""

    def __init__(self, nq, kv_len, hq, hkv, d, dtype, page=16, heads_first=True, prefix=None, group_off=None, seed=0,
                 spare_pages=2, table_pad=1, k_div=1.0):
        g = torch.Generator().manual_seed(seed)
        self.nq, self.kv_len, self.hq, self.hkv, self.d, self.dtype, self.page = nq, kv_len, hq, hkv, d, dtype, page
        self.prefix, self.group_off = prefix or [], group_off
        self.n_rows = sum(nq)
        need = [-(-n // page) for n in kv_len]
        need_p = [-(-n // page) for n in self.prefix]
        self.n_pages = sum(need) + sum(need_p) + spare_pages
        order = torch.randperm(self.n_pages, generator=g).tolist()

        def tables(counts):
            width = max(counts + [0]) + table_pad
            rows = []
            for n in counts:
                rows.append([order.pop() for _ in range(n)] + [-7] * (width - n))
            return rows

        self.pages, self.prefix_pages = tables(need), tables(need_p)
        shape = (self.n_pages, page, hkv, d)
        k, v = torch.full(shape, float("nan")), torch.full(shape, float("nan"))

        def fill(lens, pages):
            out = []
            for n, pg in zip(lens, pages):
                a = (torch.randn((n, hkv, d), generator=g) / k_div).to(dtype)
                b = torch.randn((n, hkv, d), generator=g).to(dtype)
                for t in range(0, n, page):
                    m = min(page, n - t)
                    k[pg[t // page], :m] = a[t:t + m].float()
                    v[pg[t // page], :m] = b[t:t + m].float()
                out.append((a, b))
            return out

        self.own = fill(kv_len, self.pages)
        self.pre = fill(self.prefix, self.prefix_pages)
        self.q = torch.randn((self.n_rows, hq * d), generator=g).to(dtype)
        self.cpu_k, self.cpu_v, self.heads_first = k, v, heads_first

    def group_of(self, s):
        if not self.prefix:
            return None
        for g in range(len(self.prefix)):
            if self.group_off[g] <= s < self.group_off[g + 1]:
                return g
        return None

    def starts(self):
        out = [0]
        for n in self.nq:
            out.append(out[-1] + n)
        return out

    def cache(self, b):
        def dev(x):
            x = x.to(self.dtype)
            if self.heads_first:
                return x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
            return x.contiguous().to(DEV)
        return b.KvCache(dev(self.cpu_k), dev(self.cpu_v))

    def batch(self, b, extra_rows=0):
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
        kw = {}
        if self.prefix:
            off = self.group_off
            kw = dict(group_off=ints(off), prefix_len=ints(self.prefix), prefix_pages=ints(self.prefix_pages),
                      max_prefix_len=max(self.prefix),
                      max_group_rows=max([sum(self.nq[off[g]:off[g + 1]]) for g in range(len(off) - 1)]))
        return b.KvBatch(ints(self.starts()), ints(self.kv_len), ints(self.pages), self.n_rows + extra_rows,
                         max(self.nq), max(self.kv_len), **kw)

    def reference(self, scale, window=0, n_sink=0):
        """(o [rows, hq, d], lse [rows, hq]) in float64."""
        o = torch.zeros((self.n_rows, self.hq, self.d), dtype=torch.float64)
        lse = torch.full((self.n_rows, self.hq), -math.inf, dtype=torch.float64)
        share, starts = self.hq // self.hkv, self.starts()
        q = self.q.double().view(-1, self.hq, self.d)
        for s, (n, length) in enumerate(zip(self.nq, self.kv_len)):
            k, v = self.own[s]
            g = self.group_of(s)
            before = 0
            if g is not None:
                before = self.prefix[g]
                k, v = torch.cat((self.pre[g][0], k)), torch.cat((self.pre[g][1], v))
            k, v = k.double(), v.double()
            key = torch.arange(before + length)
            for j in range(n):
                p = before + length - n + j
                if length - n + j < 0:
                    continue   # more rows than tokens: no place, nothing seen
                see = key <= p
                if window:
                    see &= (key > p - window) | (key < n_sink)
                idx = see.nonzero()[:, 0]
                kk, vv = k[idx], v[idx]                      # only what the row sees
                x = torch.einsum("kgd,tkd->kgt", q[starts[s] + j].view(self.hkv, share, self.d), kk) * scale
                lse[starts[s] + j] = torch.logsumexp(x, -1).reshape(-1)
                o[starts[s] + j] = torch.einsum("kgt,tkd->kgd", torch.softmax(x, -1), vv).reshape(self.hq, self.d)
        return o.view(self.n_rows, -1), lse


def rotate(x, cos, sin, interleaved):
    """x [..., d] float64 rotated by cos, sin [rot / 2] (broadcast)."""
    half = cos.shape[-1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, a * sin + b * cos
    return y
