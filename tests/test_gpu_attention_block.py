"""The example's attention block (projections, append, attention over prefix and pages) against a dense one in 64 bits."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from _gpu import requires_gpu, say

pytestmark = [pytest.mark.gpu, requires_gpu]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def dense(block, x, adapter):
    """The block over the tokens x [n, d_model] of one request, all at once, in 64 bits on the CPU."""
    def layer(x, W, pool):
        A, B = pool.A[adapter].double().cpu(), pool.B[adapter].double().cpu()
        return x @ W.double().cpu().t() + 0.5 * (x @ A) @ B

    n, d = x.shape[0], block.d
    hkv = block.wk // d
    q, k, v = layer(x, block.w_qkv, block.qkv_pool).split([block.wq, block.wk, block.wk], dim=1)
    cos, sin = (t[:n].double().cpu()[:, None, :] for t in (block.rope.cos, block.rope.sin))

    def turn(t):
        a, b = t.reshape(n, -1, d).chunk(2, dim=-1)
        return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)

    q, k, v = turn(q), turn(k), v.reshape(n, hkv, d)
    k, v = (t.repeat_interleave(block.hq // hkv, dim=1) for t in (k, v))
    s = block.scale * torch.einsum("rhd,khd->hrk", q, k)
    at = torch.arange(n)
    sees = at[None, :] <= at[:, None]
    if block.window:
        sees &= (at[None, :] > at[:, None] - block.window) | (at[None, :] < block.n_sink)
    p = torch.softmax(s.masked_fill(~sees, -float("inf")), dim=-1)
    return layer(torch.einsum("hrk,khd->rhd", p, v).reshape(n, -1), block.w_o, block.o_pool)


# fp32: an element of q and k errs by about sqrt(256) 2^-24 = 1e-6, a score (64 products, 1 / 8) by about as much, o
# by 1e-5 at the most and y, 256 of them times 1 / 16, by 1.6e-4; 1e-3 allows for six times that.
# bf16: q is rounded twice and k once before a score, each by up to 2^-8 of itself (rms 2^-8 / sqrt(3)): rms 3e-3 to
# 4e-3 of a score, so up to 2e-2 of a weight, of which an average over several tokens leaves about 5e-3 in o; with o's
# own rounding y errs by 5e-3 rms, five times that at the most among some thousands, and 2^-8 |y| at the end.
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-3), (torch.bfloat16, 6e-2)], ids=["fp32", "bf16"])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (50, 3)])
def test_block(dtype, tol, window, n_sink):
    ex = example()
    d_model, steps = 256, 3
    block = ex.AttentionBlock(d_model, 4, 2, 64, n_adapters=3, rank=8, dtype=dtype, n_pages=80, window=window,
                              n_sink=n_sink, seed=5)
    prefix, prompts = [70, 33, 1], [[5, 40], [1], [90, 2, 17]]
    server = ex.Server(block, prefix, prompts, max_new=steps)
    g = torch.Generator().manual_seed(6)

    def rows(n):
        return torch.randn((n, d_model), generator=g).to(dtype)

    xp, xq = rows(sum(prefix)), rows(sum(server.prompt_len))
    xd = [rows(len(server.prompt_len)) for _ in range(steps)]
    say(f"attention block {dtype} window {window}")
    server.run_prefixes(xp.cuda())
    got = [server.run_prompts(xq.cuda())] + [server.run_decode(x.cuda()) for x in xd]
    torch.cuda.synchronize()
    assert int(block.status) == 0
    got = [y.double().cpu() for y in got]
    start_p = [sum(prefix[:a]) for a in range(len(prefix))]
    r0 = 0
    for s, (a, n) in enumerate(zip(server.adapter, server.prompt_len)):
        x = torch.cat([xp[start_p[a]:start_p[a] + prefix[a]], xq[r0:r0 + n]] + [x[s:s + 1] for x in xd])
        ref = dense(block, x.double(), a)[prefix[a]:]
        y = torch.cat([got[0][r0:r0 + n]] + [y[s:s + 1] for y in got[1:]])
        err = ((y - ref).abs() / ref.abs().clamp(min=1.0)).max()
        assert float(err) <= tol, (s, float(err))
        r0 += n


def test_example_runs(capsys):
    example().main()
    assert "decode: rows (8, 1024)" in capsys.readouterr().out
