"""Attention over a cache in 8 bits whose values are as large as the header allows for sums in fp32, with weights as far
above the first score as the softmax's reference lets them be."""
from __future__ import annotations

import pytest
import torch

from _gpu import requires_gpu
from _kv_q8 import CaseQ8, codes_of
from test_gpu_kv_q8 import attend

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.mark.parametrize("nq,ln,heads,prefix", [([1, 1], [1500, 70], (8, 2), None), ([60, 90], [700, 130], (8, 2), None),
                                                ([1100], [1300], (64, 8), None), ([1] * 4, [700, 1, 30, 90], (8, 2), [900])],
                         ids=["few", "tiles", "wide", "prefix"])
@pytest.mark.parametrize("power", [68, -91])
def test_values_of_the_largest_and_least_size(nq, ln, heads, prefix, power):
    """Scores of 0 for the first 64 tokens of a sequence and its prefix, 13 (2^18.75 times the weight) after them; values
    up to 448 * 2^68 < 2^77, and of 2^-100 and less."""
    c = CaseQ8(nq, ln, *heads, 64, page=16, block=8, prefix=prefix, group_off=prefix and [0, len(nq)], seed=60)
    c.q = torch.ones_like(c.q)                      # scores are 64 / 8 times a key's element
    for pages, n in zip(c.pages + c.prefix_pages, c.kv_len + c.prefix):
        for j in range(-(-n // 16)):
            c.scales[0][pages[j]] = 1.0
            c.codes[0][pages[j]] = codes_of(torch.tensor([0.0 if j < 4 else 1.625], dtype=torch.float64))
    c.scales[1] = torch.where(torch.isnan(c.scales[1]), c.scales[1], 2.0 ** power)
    top = (c.codes[1] & 127) < 126
    c.codes[1] = torch.where(top & (torch.arange(64) % 3 == 0), 126, c.codes[1])   # 448 in some columns
    c.reread()
    assert max(float(v.abs().max()) for _, v in c.own + c.pre if v.numel()) == 448 * 2.0 ** power
    attend(c, what=f"values of 2^{power}")
    attend(c, window=100, n_sink=3, what=f"values of 2^{power}, window")
