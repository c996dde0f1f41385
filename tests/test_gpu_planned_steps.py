"""The step tables, the projections, the append and the attention together, as the example runs them."""
from __future__ import annotations

import importlib.util
import os
import random

import pytest
import torch

import _kv_q8
from _gpu import binding, requires_gpu, say


pytestmark = [pytest.mark.gpu, requires_gpu]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def schedule(seed, places, n_steps, max_rows, most):
    """Rows of each place, step by step; some requests end, some steps ask for more than there is."""
    rng = random.Random(seed)
    alive, out = [False] * places, []
    for _ in range(n_steps):
        new = []
        for i in range(places):
            if not alive[i]:
                n = rng.choice([0, rng.randint(1, most)])
                alive[i] = n > 0
            else:
                n = rng.choice([1, 1, 1, 0, -1])
                alive[i] = n >= 0
            new.append(n)
        out.append((new, [rng.randint(-1, 2) for _ in range(places)]))
    return out


def new_steps(block_size, n_pages, graph):
    ex = example("planned_steps")
    block = ex.AttentionBlock(256, 8, 2, 64, n_adapters=3, rank=8, dtype=torch.bfloat16, n_pages=n_pages, page_size=16,
                              block_size=block_size, seed=7)
    steps = ex.Steps(block, 9, max_rows=100, most=30, max_len=200)
    if graph:
        steps.capture()
    return steps


@pytest.mark.parametrize("block_size", [16, 4])
@pytest.mark.parametrize("n_pages", [60, 14], ids=["enough", "scarce"])
def test_replays_are_the_eager_steps(block_size, n_pages):
    """A captured step, replayed over requests that come, go and are refused, gives the bits of eager calls."""
    eager, replayed = new_steps(block_size, n_pages, False), new_steps(block_size, n_pages, True)
    g = torch.Generator().manual_seed(3)
    say(f"planned steps, blocks of {block_size}, {n_pages} pages")
    for new, adapter in schedule(5, 9, 12, 100, 30):
        x = torch.randn((100, 256), generator=g).to(torch.bfloat16).cuda()
        a = eager.step(new, adapter, x).clone()
        torch.cuda.synchronize()
        b = replayed.step(new, adapter, x).clone()
        torch.cuda.synchronize()
        for name in ("row_off", "row_adapter", "row_pos", "row_slot", "kv_len", "n_free", "pages"):
            assert torch.equal(getattr(eager.plan, name), getattr(replayed.plan, name)), name
        n = int(eager.plan.row_off[-1])
        assert torch.equal(a[:n], b[:n]) and torch.isfinite(a[:n]).all()
        for name in ("k_scale", "v_scale"):
            assert torch.equal(getattr(eager.block.cache, name), getattr(replayed.block.cache, name))
    assert int(eager.block.status) == int(replayed.block.status) == (1 if n_pages == 14 else 0)


def test_steps_against_the_definitions():
    """Every step's tables, cache and attention from the definitions, given the projections' outputs."""
    lb = binding()
    steps = new_steps(8, 60, False)
    block, plan = steps.block, steps.plan
    cache = block.cache
    c = _kv_q8.CaseQ8([0] * 9, [0] * 9, 8, 2, 64, page=16, block=8, table_pad=13, spare_pages=60)
    c.codes = [torch.zeros((60, 16, 2, 64), dtype=torch.uint8) for _ in range(2)]
    c.scales = [torch.ones((60, 2, 2), dtype=torch.float64) for _ in range(2)]
    pages = plan.pages.tolist()
    lens, free, height = [0] * 9, plan.free_pages.tolist(), 60
    cos, sin = block.rope.cos.cpu(), block.rope.sin.cpu()
    g = torch.Generator().manual_seed(4)
    seen = {}

    def attend(cache_, batch, q, scale, **kw):
        o = lb.lora_attn_paged_q8(cache_, batch, q, scale, **kw)
        seen.update(q=q.clone(), o=o.clone())
        return o

    def append(cache_, batch, q, k, v, rope, **kw):
        seen.update(k=k.clone(), v=v.clone())
        return lb.lora_kv_append_q8(cache_, batch, q, k, v, rope, **kw)

    block.attend, block.append = attend, append
    say("planned steps against the definitions")
    for new, adapter in schedule(6, 9, 8, 100, 30):
        steps.step(new, adapter, torch.randn((100, 256), generator=g).to(torch.bfloat16).cuda())
        torch.cuda.synchronize()
        w = _kv_q8.plan(new, adapter, lens, pages, free, height, 16, 100)
        lens, pages, free, height = w["kv_len"], w["pages"], w["free"], w["n_free"]
        for name in ("row_off", "row_adapter", "row_pos", "kv_len", "pages"):
            assert torch.equal(getattr(plan, name).cpu(), torch.tensor(w[name], dtype=torch.int32)), name
        c.nq = [b - a for a, b in zip(w["row_off"], w["row_off"][1:])]
        c.kv_len, c.pages, c.n_rows = lens, pages, w["row_off"][-1]
        _kv_q8.append(c, {i: seen[i].cpu() for i in "kv"}, (cos, sin, False))
        live = [(pg, t % 16) for s, n in enumerate(lens) for t in range(n) for pg in [pages[s][t // 16]]]
        for i, name in enumerate("kv"):
            got, want = getattr(cache, name).view(torch.uint8).cpu(), c.codes[i]
            for pg, t in live:
                assert torch.equal(got[pg, t], want[pg, t]), (name, pg, t)
        c.reread()
        c.q = seen["q"][:c.n_rows].cpu()
        ref = c.reference(block.scale)[0]
        # the weights' rounding and o's, 2^-8 each at the most, half of their sum; sums 2e-4 (test_gpu_kv_q8.py)
        vmax = max([float(x[1].abs().max()) for x in c.own if x[1].numel()] + [1e-30])
        assert float((seen["o"][:c.n_rows].double().cpu() - ref).abs().max()) <= (2.0 ** -8 + 2e-4) * vmax



def test_example_runs(capsys):
    example("planned_steps").main()
    out = capsys.readouterr().out
    assert "requests 9 free pages 256 of 256" in out


def test_attention_block_in_8_bits():
    """The other example's block with shared prefixes over a cache in 8 bits, beside one in bf16.

    A key or value is off by at most 2^-4 of itself, so o by 2^-4 of the values and by what the keys' errors move the
    weights: a score of this block (|q . k| / 8 below 8, errors of 64 products adding as squares) by some 2^-4, a
    weight by as much of itself.  o is off by at most an eighth of the values' size, y (o times a matrix of rows of
    norm 1) by an eighth of |o| sqrt(2): half of the outputs' own largest is asked for.
    """
    ex = example("attention_block")
    ys = []
    for block_size in (0, 8):
        block = ex.AttentionBlock(256, 4, 2, 64, n_adapters=3, rank=8, dtype=torch.bfloat16, n_pages=80, seed=5,
                                  block_size=block_size)
        server = ex.Server(block, [70, 33, 1], [[5, 40], [1], [90, 2, 17]], max_new=3)
        g = torch.Generator().manual_seed(6)

        def rows(n):
            return torch.randn((n, 256), generator=g).to(torch.bfloat16).cuda()

        server.run_prefixes(rows(104))
        y = [server.run_prompts(rows(155))] + [server.run_decode(rows(6)) for _ in range(3)]
        torch.cuda.synchronize()
        assert int(block.status) == 0
        ys.append(torch.cat(y).double().cpu())
    far = float((ys[0] - ys[1]).abs().max())
    say(f"8 bits beside bf16: {far:.3f} of {float(ys[0].abs().max()):.3f}")
    assert 0 < far <= 0.5 * float(ys[0].abs().max())
