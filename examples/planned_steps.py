"""A server's steps planned on the GPU, over keys and values in 8 bits.

    rows of each request -> tables of the step    lora_kv_plan
    q k v = x Wqkv (+ the row's adapter)          lora_layer_apply, ids from the tables
    rotate, keys and values into their pages      lora_kv_append_q8
    o = attention over the pages                  lora_attn_paged_q8
    y = o Wo (+ the row's adapter)                lora_layer_apply

The server has a fixed number of places.  A request takes a place with its
prompt, brings a row a step, and gives its pages back when it ends.  Lengths,
page tables and the stack of free pages stay on the GPU; the host says how many
rows each place brings.  A request for whose rows there is no room (pages, a
step's rows, its table) is left out of the step as a whole, so the rows that are
served are picked from those that were brought, on the GPU too.  Steps of at most
``max_rows`` rows are one captured graph, replayed with other requests, lengths
and adapters in the same tensors.

    python examples/planned_steps.py
"""
from __future__ import annotations

import os
import sys
from typing import List, Optional

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import torch  # noqa: E402

from attention_block import AttentionBlock  # noqa: E402  (puts the package on the path)
from lora_bgmv_shrink_amd import binding as lb  # noqa: E402


class Steps:
    """Steps of up to ``max_rows`` rows, ``most`` of them one request's, over ``n_places`` places.  A request has up
    to ``max_len`` tokens, rounded up to whole pages."""

    def __init__(self, block: AttentionBlock, n_places: int, max_rows: int, most: int, max_len: int):
        self.block, dev, page = block, block.device, block.cache.page_size
        self.most, self.max_rows = most, max_rows

        def ints(n, value=0):
            return torch.full((n,), value, dtype=torch.int32, device=dev)

        self.new_rows, self.adapter = ints(n_places), ints(n_places, -1)
        pages = torch.full((n_places, -(-max_len // page)), -1, dtype=torch.int32, device=dev)
        free = torch.arange(block.cache.n_pages, dtype=torch.int32, device=dev)
        self.plan = lb.KvPlan(ints(n_places), pages, free, ints(1, block.cache.n_pages), page, max_rows)
        # the tensors that every step's plan writes; bounds that hold for all that it may grant (a whole table's
        # tokens), as what is past them would be neither computed nor seen.  `most` is checked by step()
        self.batch = lb.KvBatch(self.plan.row_off, self.plan.kv_len, self.plan.pages, max_rows, most, pages.shape[1] * page)
        self.ws = block.workspace(block.cache, self.batch, block.hq)
        # rows as they are brought, place by place, the first of each place, and one past the last for the rows of a
        # step that are nobody's
        self.x = torch.zeros((max_rows + 1, block.w_qkv.shape[1]), dtype=block.dtype, device=dev)
        self.y = torch.zeros((max_rows + 1, block.w_o.shape[0]), dtype=block.dtype, device=dev)
        self.first = torch.zeros(n_places, dtype=torch.int64, device=dev)
        self.numbers = torch.arange(max_rows, device=dev)
        self.graph: Optional[torch.cuda.CUDAGraph] = None

    def _step(self) -> None:
        lb.lora_kv_plan(self.plan, self.new_rows, self.adapter, status=self.block.status)
        # the step's row r is row r - row_off[s] of place s = row_seq[r]
        seq = self.plan.row_seq
        s = seq.clamp(min=0).long()
        brought = torch.where(seq >= 0, self.first[s] + self.numbers - self.plan.row_off[s], self.numbers.numel())
        y = self.block.step(self.x[brought], self.plan.row_adapter, self.batch, self.ws)
        self.y.zero_().index_copy_(0, brought, y)

    def capture(self) -> None:
        """The step as a graph (places without rows: capturing runs nothing)."""
        self.new_rows.zero_()
        self._step()   # loads what loads lazily
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=side):
            self._step()

    def step(self, new_rows: List[int], adapter: List[int], x: torch.Tensor) -> torch.Tensor:
        """One step: place i brings new_rows[i] rows (below zero: its request is over); ``x`` are the rows, in the
        order of their places.  Returns theirs of the output, zeros where the place was not served."""
        if max(new_rows) > self.most or sum(max(n, 0) for n in new_rows) > min(self.max_rows, x.shape[0]):
            raise ValueError(f"more rows than {self.most} of a request, {self.max_rows} of a step, or {x.shape[0]} brought")
        first = torch.tensor([0] + new_rows).clamp(min=0).cumsum(0)
        self.first.copy_(first[:-1])
        self.new_rows.copy_(torch.tensor(new_rows, dtype=torch.int32))
        self.adapter.copy_(torch.tensor(adapter, dtype=torch.int32))
        self.x[:x.shape[0]].copy_(x)
        if self.graph is None:
            self._step()
        else:
            self.graph.replay()
        return self.y[:x.shape[0]]

    def served(self) -> List[bool]:
        """Of the last step, for each place: whether its rows were served.  Those that were not may be brought again."""
        return (self.plan.row_off.diff() == self.new_rows.clamp(min=0)).tolist()


def main() -> None:
    torch.manual_seed(0)
    d_model, places = 1024, 6
    block = AttentionBlock(d_model, 16, 4, 64, n_adapters=3, rank=16, dtype=torch.bfloat16, n_pages=256, block_size=16)
    steps = Steps(block, places, max_rows=64, most=40, max_len=300)
    steps.capture()
    rows, left = [0] * places, [0] * places   # rows that each place brings next, and steps after that
    waiting = [(0, 12, 5), (1, 40, 3), (2, 7, 9), (0, 3, 4), (1, 21, 6), (2, 33, 2), (0, 9, 3), (1, 5, 5), (2, 2, 2)]
    adapter, done, n, refused = [-1] * places, 0, 0, 0
    while done < 9:
        new, budget = [0] * places, 64
        for i in range(places):
            if adapter[i] >= 0 and left[i] < 0:   # its last row was the step before
                new[i], adapter[i], done = -1, -1, done + 1
                continue
            if adapter[i] < 0 and waiting:
                adapter[i], rows[i], left[i] = waiting.pop(0)
            if adapter[i] >= 0 and rows[i] <= budget:
                new[i] = rows[i]
                budget -= rows[i]
        brought = sum(max(r, 0) for r in new)
        y = steps.step(new, adapter, torch.randn((brought, d_model), device="cuda").to(torch.bfloat16))
        n += 1
        for i, ok in enumerate(steps.served()):
            if not ok:
                refused += 1               # brings the same rows again
            elif new[i] > 0:
                rows[i], left[i] = 1, left[i] - 1
        if refused > 100:
            raise SystemExit("too few pages")
    torch.cuda.synchronize()
    if int(block.status) and not refused:
        raise SystemExit("a row had no place")
    print("steps", n, "requests", done, "free pages", int(steps.plan.n_free), "of", block.cache.n_pages, "rows of the last",
          tuple(y.shape))


if __name__ == "__main__":
    main()
