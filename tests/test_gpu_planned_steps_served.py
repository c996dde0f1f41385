"""The example's steps when the plan serves some requests and not others, and at the bounds of its batch."""
from __future__ import annotations

import pytest
import torch

from _gpu import requires_gpu, say
from test_gpu_planned_steps import example

pytestmark = [pytest.mark.gpu, requires_gpu]


def new_steps(n_pages, max_len, places=3, max_rows=64, most=30, graph=False):
    ex = example("planned_steps")
    block = ex.AttentionBlock(256, 8, 2, 64, n_adapters=3, rank=8, dtype=torch.bfloat16, n_pages=n_pages, page_size=16,
                              block_size=8, seed=7)
    steps = ex.Steps(block, places, max_rows=max_rows, most=most, max_len=max_len)
    if graph:
        steps.capture()
    return steps


def rows_of(step, place, n):
    g = torch.Generator().manual_seed(100 * step + place)
    return torch.randn((max(n, 0), 256), generator=g).to(torch.bfloat16)


def run(steps, i, new):
    """One step; the output's rows of each place."""
    x = torch.cat([rows_of(i, p, n) for p, n in enumerate(new)]).cuda()
    y = steps.step(new, [0, 1, 2][:len(new)], x)
    torch.cuda.synchronize()
    return [t.clone() for t in y.split([max(n, 0) for n in new])]


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("n_pages,max_len,plan,refused", [
    (3, 200, [[5, 0, 4], [1, 30, 1], [1, 0, 1]], (1, 1)),        # two pages wanted, one left
    (20, 32, [[5, 20, 4], [1, 30, 20], [1, 1, 1]], (1, 1)),      # more than its table holds
    (2, 200, [[30, 3, 2], [1, 0, 0], [1, 0, 0]], (0, 1)),        # no page left for a prompt in the middle
], ids=["pages", "table", "prompt"])
def test_a_refused_request_leaves_the_others_alone(graph, n_pages, max_len, plan, refused):
    """Rows, adapters, keys and values of the others are those of a run in which it brings no rows."""
    at, place = refused
    got, want = new_steps(n_pages, max_len, graph=graph), new_steps(n_pages, max_len, graph=graph)
    say(f"refused in step {at}, place {place}: {plan}")
    for i, new in enumerate(plan):
        without = list(new)
        if i == at:
            without[place] = 0
        if n_pages == 2 and i == 0:   # places 1 and 2 find no page
            without = [30, 0, 0]
        a, b = run(got, i, new), run(want, i, without)
        for p in range(3):
            if without[p] == new[p]:
                assert torch.equal(a[p], b[p]), (i, p)
            else:
                assert bool((a[p] == 0).all()), (i, p)
        for name in ("kv_len", "pages", "n_free", "row_off", "row_adapter", "row_pos"):
            assert torch.equal(getattr(got.plan, name), getattr(want.plan, name)), (i, name)
        for name in ("k", "v"):
            x, y = (getattr(s.block.cache, name).view(torch.uint8) for s in (got, want))
            assert torch.equal(x, y), (i, name)
    assert int(got.block.status) == 1 and int(want.block.status) == 0


def test_who_was_served():
    steps = new_steps(3, 200)
    for i, (new, want) in enumerate((([5, 0, 4], [True] * 3), ([1, 30, 1], [True, False, True]), ([1, -1, -1], [True] * 3))):
        run(steps, i, new)
        assert steps.served() == want, i


def test_requests_as_long_as_their_tables():
    """max_len is rounded up to whole pages: what the plan grants, the attention sees."""
    tight, roomy = new_steps(8, 20, places=1), new_steps(8, 64, places=1)
    assert tight.plan.pages.shape[1] == 2
    say("up to the table's end")
    for i, n in enumerate([20] + [1] * 12):
        a, b = run(tight, i, [n])[0], run(roomy, i, [n])[0]
        assert torch.equal(a, b), f"step {i}"
    assert int(tight.plan.kv_len) == 32 and int(tight.block.status) == 0
    run(tight, 20, [1])
    assert int(tight.plan.kv_len) == 32 and int(tight.block.status) == 1


def test_more_rows_than_a_step_takes():
    """Rows that the attention's bound or the step does not cover are turned away, and nothing has changed."""
    steps = new_steps(20, 200, most=30, max_rows=64)
    run(steps, 0, [30, 4, 30])
    lens = steps.plan.kv_len.tolist()
    say("too many rows")
    for new, x in (([31, 0, 0], 31), ([30, 5, 30], 65), ([3, 0, 2], 4)):
        with pytest.raises(ValueError):
            steps.step(new, [0, 1, 2], torch.zeros((x, 256), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert steps.plan.kv_len.tolist() == lens == [30, 4, 30]
