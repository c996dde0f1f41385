"""A step's tables made on the GPU (lora_kv_plan) against their definition; every number has to be the same."""
from __future__ import annotations

import random

import pytest
import torch

import _kv_q8
from _gpu import binding, requires_gpu, say
from _kv import DEV

pytestmark = [pytest.mark.gpu, requires_gpu]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Server:
    """Lists on the CPU beside the tensors of a plan."""

    def __init__(self, b, kv_len, page, wide, spare, max_rows, seed=0, prefix=None, group_off=None, in_place=True,
                 max_free=None):
        rng = random.Random(seed)
        self.b, self.page, self.max_rows, self.prefix, self.group_off = b, page, max_rows, prefix, group_off
        held = [-(-n // page) for n in kv_len]
        ids = list(range(7, 7 + sum(held) + spare))
        rng.shuffle(ids)
        self.kv_len = list(kv_len)
        self.pages = [[ids.pop() for _ in range(n)] + [-9] * (wide - n) for n in held]
        room = max_free if max_free is not None else sum(held) + spare
        self.free, self.n_free = ids + [-5] * (room - len(ids)), len(ids)
        self.status = ints([0])
        kw = {} if in_place else dict(kv_len_out=ints([-3] * len(kv_len)), n_free_out=ints([-3]))
        if prefix:
            kw.update(group_off=ints(group_off), prefix_len=ints(prefix))
        table = ints(self.pages) if kv_len else torch.empty((0, wide), dtype=torch.int32, device=DEV)
        self.plan = b.KvPlan(ints(self.kv_len), table, ints(self.free), ints([self.n_free]), page, max_rows, **kw)

    def step(self, new_rows, adapter=None, what=""):
        say(f"plan {what}: {len(new_rows)} sequences, {sum(max(n, 0) for n in new_rows)} rows of {self.max_rows}, "
            f"{self.n_free} free pages")
        p = self.plan
        for t in (p.row_off, p.row_seq, p.row_adapter, p.row_pos, p.row_slot):
            t.fill_(-77)
        self.status.zero_()
        self.b.lora_kv_plan(p, ints(new_rows), None if adapter is None else ints(adapter), status=self.status)
        torch.cuda.synchronize()
        want = _kv_q8.plan(new_rows, adapter, self.kv_len, self.pages, self.free, self.n_free, self.page, self.max_rows,
                           self.prefix, self.group_off)
        got = dict(row_off=p.row_off, row_seq=p.row_seq, row_adapter=p.row_adapter, row_pos=p.row_pos,
                   row_slot=p.row_slot, kv_len=p.kv_len_out, pages=p.pages, free=p.free_pages, n_free=p.n_free_out)
        for name, t in got.items():
            w = torch.tensor(want[name], dtype=t.dtype).view(t.shape)
            assert torch.equal(t.cpu(), w), (what, name)
        assert int(self.status.item()) == want["status"], what
        self.kv_len, self.pages, self.free, self.n_free = want["kv_len"], want["pages"], want["free"], want["n_free"]
        return want


def random_step(rng, n, prompts, over):
    kinds = [rng.random() for _ in range(n)]
    return [-rng.randint(1, 5) if k < over else rng.randint(2, 70) if k < over + prompts else 0 if k > 0.9 else 1
            for k in kinds]


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 700, 1023, 1024, 1025, 2500])
@pytest.mark.parametrize("page", [1, 16])
def test_random_steps(n, page):
    """Steps in a row, with requests that end, on both sides of the single launch; pages never get lost."""
    rng = random.Random(n * 100 + page)
    lens = [rng.choice([0, 1, 15, 16, 17, rng.randint(0, 200)]) for _ in range(n)]
    s = Server(binding(), lens, page, 400 // page + 3, 12 * n + 5, 12 * n + 3, seed=n)
    every = sorted(s.free[:s.n_free] + [p for r in s.pages for p in r if p >= 0])
    for i in range(4):
        s.step(random_step(rng, n, 0.2, 0.1), [rng.randint(-1, 9) for _ in range(n)], f"step {i}")
        held = [p for r, m in zip(s.pages, s.kv_len) for p in r[:-(-m // page)]]
        assert sorted(s.free[:s.n_free] + held) == every


@pytest.mark.parametrize("in_place", [True, False])
def test_too_few(in_place):
    """Pages, rows or a table that do not suffice: whole requests are refused, later ones that need no page are not."""
    b = binding()
    s = Server(b, [16, 16, 3, 0, 5, 31], 16, 4, 3, 100, in_place=in_place)
    w = s.step([1, 40, 1, 20, 2, 1], [0, 1, 2, 3, 4, 5], "pages")
    assert w["status"] == 1 and w["row_off"] == [0, 1, 1, 2, 2, 4, 5]
    s = Server(b, [16, 0, 9], 16, 4, 50, 10)
    assert s.step([3, 8, 1], None, "rows")["row_off"] == [0, 3, 3, 3]      # 3 + 8 rows asked for; then 12
    s = Server(b, [60, 0, 64, 63], 16, 4, 50, 100)
    w = s.step([5, 64, 1, 1], None, "tables")
    assert w["row_off"] == [0, 0, 64, 64, 65] and w["status"] == 1
    s = Server(b, [4, 4, 4], 16, 2, 0, 8)
    w = s.step([2 ** 31 - 1, 3, 2 ** 30], None, "more than any table")
    assert w["row_off"] == [0, 0, 3, 3]


def test_released_pages_are_taken_at_once():
    """The stack is empty: what ends in this step serves it; more comes back than is taken, and less."""
    b = binding()
    s = Server(b, [100, 0, 40], 16, 12, 0, 200, seed=3)
    s.step([-1, 50, 1], [4, 5, 6], "7 back, 4 taken")
    s.step([0, -1, -1], None, "all back")
    s.step([130, 30, 1], None, "taken")
    s.step([-1, -1, -1], None, "nothing but ends")


def test_ended_requests_beside_refused_ones():
    rng = random.Random(5)
    for seed in range(6):
        s = Server(binding(), [rng.randint(0, 90) for _ in range(90)], 8, 14, 20, 150, seed=seed, in_place=seed % 2 == 0,
                   prefix=[33, 0, 7], group_off=[3, 20, 20, 80])
        s.step(random_step(rng, 90, 0.5, 0.05), [rng.randint(-1, 9) for _ in range(90)], f"scarce {seed}")


def test_more_back_than_the_stack_holds():
    """A table that names pages twice: the stack keeps what it has room for, and says so."""
    s = Server(binding(), [64, 64, 10], 16, 5, 3, 30, max_free=6)
    w = s.step([-1, -1, 30], None, "too many back")
    assert w["status"] == 2


def test_sums_past_32_bits():
    """Requests that ask for 2^30 rows each, by the hundred: refused, and the next that fits is not served for it."""
    b = binding()
    n = 300
    table = torch.full((n, 1 << 12), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(50, dtype=torch.int32, device=DEV)
    plan = b.KvPlan(ints([0] * n), table, free, ints([50]), 1 << 18, 64)
    status = ints([0])
    say("sums past 32 bits")
    b.lora_kv_plan(plan, ints([1] + [2 ** 30 - 8] * (n - 2) + [1]), status=status)
    torch.cuda.synchronize()
    assert plan.row_off.tolist() == [0] + [1] * n and int(status.item()) == 1
    assert int(plan.n_free.item()) == 49 and plan.kv_len.tolist() == [1] + [0] * (n - 1)


def test_nothing_and_one():
    s = Server(binding(), [], 16, 3, 5, 4)
    s.step([], None, "no sequences")
    s = Server(binding(), [0], 16, 3, 5, 0)
    s.step([0], None, "no rows")
    s.step([1], None, "no room for rows")
    s = Server(binding(), [0], 16, 0, 0, 4)
    s.step([1], None, "no table, no pages")


def test_row_arrays_that_are_not_wanted():
    b = binding()
    s = Server(b, [5, 9], 8, 4, 9, 12, seed=8)
    for name in ("row_seq", "row_adapter", "row_pos", "row_slot"):
        setattr(s.plan.struct, name, None)
    say("no row arrays")
    b.lora_kv_plan(s.plan, ints([4, 3]))
    torch.cuda.synchronize()
    assert s.plan.row_off.tolist() == [0, 4, 7] and s.plan.kv_len.tolist() == [9, 12]


@pytest.mark.parametrize("n", [40, 1500])
def test_wrong_contents_stay_in_bounds(n):
    """Lengths, heights and groups of any content: the arrays' neighbours are not touched."""
    b = binding()
    rng = random.Random(n)
    odd = [0, 1, -1, -2 ** 31, 2 ** 31 - 1, 2 ** 30, 77, 100000]

    def guarded(length, dtype=torch.int32):
        whole = torch.full((length + 128,), 123, dtype=dtype, device=DEV)
        return whole, whole[64:64 + length]

    for seed in range(5):
        say(f"wrong contents {seed}")
        sizes = dict(kv_len=n, pages=n * 6, free=50, n_free=1)
        arrays = {k: guarded(v) for k, v in sizes.items()}
        for k, (_, t) in arrays.items():
            t.copy_(ints([rng.choice(odd) for _ in range(t.numel())]))
        plan = b.KvPlan(arrays["kv_len"][1], arrays["pages"][1].view(n, 6), arrays["free"][1], arrays["n_free"][1], 16, 200,
                        group_off=ints([rng.choice(odd) for _ in range(4)]), prefix_len=ints([rng.choice(odd)] * 3))
        out = {}
        for k in ("row_off", "row_seq", "row_adapter", "row_pos", "row_slot"):
            t = getattr(plan, k)
            out[k] = guarded(t.numel(), t.dtype)
            setattr(plan.struct, k, out[k][1].data_ptr())
        b.lora_kv_plan(plan, ints([rng.choice(odd) for _ in range(n)]), ints([3] * n))
        torch.cuda.synchronize()
        for k, (whole, t) in list(arrays.items()) + list(out.items()):
            assert bool((whole[:64] == 123).all()) and bool((whole[64 + t.numel():] == 123).all()), k


def test_graph_replays_steps():
    """A captured plan goes on from the state that the last replay left; several replays, eager work between them."""
    b = binding()
    n = 48
    s = Server(b, [20 + i for i in range(n)], 16, 40, 200, 120, seed=9)
    want_rows, adapter = ints([1] * n), ints(list(range(n)))
    say("plan: eager, capture, replays")
    b.lora_kv_plan(s.plan, ints([0] * n), adapter)   # changes nothing
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.lora_kv_plan(s.plan, want_rows, adapter)
    rng = random.Random(10)
    for i in range(6):
        new = [rng.choice([1, 1, 1, 3, 0, -1]) for _ in range(n)]
        want_rows.copy_(ints(new))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        w = _kv_q8.plan(new, list(range(n)), s.kv_len, s.pages, s.free, s.n_free, 16, 120)
        p = s.plan
        for name, t in (("row_off", p.row_off), ("row_slot", p.row_slot), ("row_adapter", p.row_adapter),
                        ("kv_len", p.kv_len), ("pages", p.pages), ("n_free", p.n_free), ("free", p.free_pages)):
            assert torch.equal(t.cpu(), torch.tensor(w[name], dtype=t.dtype).view(t.shape)), (i, name)
        s.kv_len, s.pages, s.free, s.n_free = w["kv_len"], w["pages"], w["free"], w["n_free"]
