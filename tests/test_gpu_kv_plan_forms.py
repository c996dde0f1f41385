"""Every form of lora_kv_plan: one launch of one, four and sixteen waves and two launches, with prefixes whose tables are
searched in LDS and in memory.  Every number has to be the same as the definition's."""
from __future__ import annotations

import random

import pytest

from _gpu import binding, requires_gpu
from test_gpu_kv_plan import Server, random_step

pytestmark = [pytest.mark.gpu, requires_gpu]


def groups_of(rng, n, n_groups):
    off = sorted(rng.randint(0, n) for _ in range(n_groups + 1))   # some are empty, some sequences are in none
    return [rng.choice([0, rng.randint(1, 3000)]) for _ in range(n_groups)], off


@pytest.mark.parametrize("n_groups", [0, 8, 600])
@pytest.mark.parametrize("n,max_rows", [(1, 4), (64, 256), (64, 257), (65, 256), (256, 1024), (257, 1024), (256, 1025),
                                        (257, 4096), (1023, 4095), (1024, 4096), (1024, 4097), (1025, 4096), (3, 4096),
                                        (3, 4097), (2047, 5000), (2048, 5000), (2049, 5000)])
def test_random_steps(n, max_rows, n_groups):
    """Requests come, end and are refused for rows and for pages; pages never get lost."""
    rng = random.Random(n * 10000 + max_rows + n_groups)
    prefix, off = groups_of(rng, n, n_groups) if n_groups else (None, None)
    lens = [rng.choice([0, 1, 7, 8, 9, rng.randint(0, 100)]) for _ in range(n)]
    s = Server(binding(), lens, 8, 40, 3 * max_rows // 16 + 5, max_rows, seed=n, prefix=prefix, group_off=off)
    every = sorted(s.free[:s.n_free] + [p for r in s.pages for p in r if p >= 0])
    refused = 0
    for i in range(3):
        # from a few prompts among rows that fit to more of them than rows or pages
        w = s.step(random_step(rng, n, (0.02, 0.1, 0.5)[i], 0.1), [rng.randint(-1, 9) for _ in range(n)], f"step {i}")
        refused += w["status"] & 1
        held = [p for r, m in zip(s.pages, s.kv_len) for p in r[:-(-m // 8)]]
        assert sorted(s.free[:s.n_free] + held) == every
    assert refused or n < 64
