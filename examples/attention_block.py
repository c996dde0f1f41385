"""One multi-LoRA attention block serving requests of several adapters.

    q k v = x Wqkv (+ the row's adapter)      lora_layer_apply
    rotate q and k, k and v into their pages  lora_kv_append
    o = attention over the pages              lora_attn_paged / lora_attn_prefix
    y = o Wo (+ the row's adapter)            lora_layer_apply

The requests of an adapter share a prefix (a system prompt).  Keys and values
depend on the adapter, so each adapter has a prefix of its own: it runs once,
as a sequence, and its pages then stand before the pages of every request of
that adapter.  Requests are admitted with prompts of different lengths and
decode one token a step.  Workspaces, page tables and outputs of the decode
step are allocated once: a step only changes lengths and inputs in place.

    python examples/attention_block.py
"""
from __future__ import annotations

import os
import sys
from typing import List

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from lora_bgmv_shrink_amd import binding as lb  # noqa: E402


def rotary_tables(n_pos: int, rot_dim: int, device, base: float = 10000.0):
    f = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * f
    return angle.cos().float().to(device), angle.sin().float().to(device)


class AttentionBlock:
    def __init__(self, d_model: int, n_q_heads: int, n_kv_heads: int, head_dim: int, n_adapters: int, rank: int,
                 dtype: torch.dtype, n_pages: int, page_size: int = 16, n_pos: int = 2048, window: int = 0,
                 n_sink: int = 0, device="cuda", seed: int = 0, block_size: int = 0):
        """``block_size`` > 0: keys and values in 8 bits, with a scale for that many tokens of a head."""
        g = torch.Generator().manual_seed(seed)
        self.hq, self.d, self.device, self.dtype = n_q_heads, head_dim, device, dtype
        self.wq, self.wk = n_q_heads * head_dim, n_kv_heads * head_dim
        self.scale, self.window, self.n_sink = head_dim ** -0.5, window, n_sink

        def layer(d_in, d_out):   # W [d_out, d_in] and the adapters' A, B
            W = torch.randn((d_out, d_in), generator=g) / d_in ** 0.5
            A = torch.randn((n_adapters, d_in, rank), generator=g) / d_in ** 0.5
            B = torch.randn((n_adapters, rank, d_out), generator=g) / rank ** 0.5
            W, A, B = (t.to(device=device, dtype=dtype) for t in (W, A, B))
            return W, lb.lora_pool_create(lb.LORA_LAYOUT_UNIFORM, A, B, n_adapters, d_in, d_out, rank,
                                          [0.5] * n_adapters)

        self.w_qkv, self.qkv_pool = layer(d_model, self.wq + 2 * self.wk)
        self.w_o, self.o_pool = layer(self.wq, d_model)
        # one head's tokens of a page side by side; the binding sees [page, token, head, dim]
        held = torch.uint8 if block_size else dtype
        pages = [torch.zeros((n_pages, n_kv_heads, page_size, head_dim), dtype=held, device=device) for _ in range(2)]
        k, v = (t.transpose(1, 2) for t in pages)
        if block_size:
            scales = [torch.ones((n_pages, page_size // block_size, n_kv_heads), device=device) for _ in range(2)]
            self.cache = lb.KvCacheQ8(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), *scales)
            self.append, self.attend, self.workspace = lb.lora_kv_append_q8, lb.lora_attn_paged_q8, lb.attn_workspace_q8
            self.attend_behind = lb.lora_attn_prefix_q8
        else:
            self.cache = lb.KvCache(k, v)
            self.append, self.attend, self.workspace = lb.lora_kv_append, lb.lora_attn_paged, lb.attn_workspace
            self.attend_behind = lb.lora_attn_prefix
        self.rope = lb.Rope(*rotary_tables(n_pos, head_dim, device))
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def step(self, x: torch.Tensor, ids: torch.Tensor, batch: lb.KvBatch, ws: torch.Tensor) -> torch.Tensor:
        """The block over one step's rows ``x`` [n_rows, d_model]."""
        qkv = lb.lora_layer_apply(self.qkv_pool, x, self.w_qkv, ids, lb.LORA_W_OUT_IN, y_dtype=self.dtype)
        q, k, v = qkv.split([self.wq, self.wk, self.wk], dim=1)
        q = self.append(self.cache, batch, q, k, v, self.rope, q_out=q, status=self.status)
        attend = self.attend_behind if batch.n_groups else self.attend
        o = attend(self.cache, batch, q, self.scale, window=self.window, n_sink=self.n_sink, status=self.status, ws=ws)
        return lb.lora_layer_apply(self.o_pool, o, self.w_o, ids, lb.LORA_W_OUT_IN, y_dtype=self.dtype)


class Server:
    """Requests [adapter][request] -> prompt length, in adapter order; adapter
    a's requests share a prefix of ``prefix_len[a]`` tokens."""

    def __init__(self, block: AttentionBlock, prefix_len: List[int], prompts: List[List[int]], max_new: int):
        self.block, page, dev = block, block.cache.page_size, block.device
        self.prefix_len, self.prompt_len = prefix_len, [n for group in prompts for n in group]
        self.adapter = [a for a, group in enumerate(prompts) for _ in group]
        free = list(range(block.cache.n_pages))

        def table(tokens):   # pages for these many tokens of each
            width = max(-(-n // page) for n in tokens)
            rows = [[free.pop() for _ in range(-(-n // page))] for n in tokens]
            return torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32, device=dev)

        self.prefix_pages = table(prefix_len)
        self.pages = table([n + max_new for n in self.prompt_len])
        self.max_len = max(self.prompt_len) + max_new
        counts = [len(group) for group in prompts]
        self.group_off = self._offsets(counts)
        self.prefix_dev = torch.tensor(prefix_len, dtype=torch.int32, device=dev)
        self.kv_len = torch.tensor(self.prompt_len, dtype=torch.int32, device=dev)
        self.decode_ids = torch.tensor(self.adapter, dtype=torch.int32, device=dev)
        n = len(self.prompt_len)
        self.decode_batch = self._requests([1] * n, max(counts))
        self.decode_ws = block.workspace(block.cache, self.decode_batch, block.hq)

    def _offsets(self, counts) -> torch.Tensor:
        return torch.cumsum(torch.tensor([0] + list(counts)), 0).to(torch.int32).to(self.block.device)

    def _requests(self, rows: List[int], group_rows: int) -> lb.KvBatch:
        return lb.KvBatch(self._offsets(rows), self.kv_len, self.pages, sum(rows), max(rows), self.max_len,
                          self.group_off, self.prefix_dev, self.prefix_pages, max(self.prefix_len), group_rows)

    def run_prefixes(self, x: torch.Tensor) -> torch.Tensor:
        """The prefixes as sequences, one per adapter: fills their pages."""
        n = self.prefix_len
        batch = lb.KvBatch(self._offsets(n), self.prefix_dev, self.prefix_pages, sum(n), max(n), max(n))
        ids = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n)).to(torch.int32).to(self.block.device)
        return self.block.step(x, ids, batch, self.block.workspace(self.block.cache, batch, self.block.hq))

    def run_prompts(self, x: torch.Tensor) -> torch.Tensor:
        n = self.prompt_len
        per_group = [sum(r for r, a in zip(n, self.adapter) if a == g) for g in range(len(self.prefix_len))]
        batch = self._requests(n, max(per_group))
        ids = torch.repeat_interleave(self.decode_ids, self.kv_len.long())
        return self.block.step(x, ids, batch, self.block.workspace(self.block.cache, batch, self.block.hq))

    def run_decode(self, x: torch.Tensor) -> torch.Tensor:
        """One more token of every request (at most ``max_new`` times)."""
        self.kv_len += 1   # the batch keeps this tensor: lengths change in place
        return self.block.step(x, self.decode_ids, self.decode_batch, self.decode_ws)


def main() -> None:
    torch.manual_seed(0)
    d_model, steps = 1024, 8
    block = AttentionBlock(d_model, 16, 4, 64, n_adapters=3, rank=16, dtype=torch.bfloat16, n_pages=512)
    server = Server(block, prefix_len=[300, 120, 64], prompts=[[5, 40, 130], [1, 77], [200, 9, 31]], max_new=steps)

    def rows(n):
        return torch.randn((n, d_model), device="cuda").to(torch.bfloat16)

    y = server.run_prefixes(rows(sum(server.prefix_len)))
    print("prefixes: rows", tuple(y.shape))
    y = server.run_prompts(rows(sum(server.prompt_len)))
    print("prompts: rows", tuple(y.shape))
    for _ in range(steps):
        y = server.run_decode(rows(len(server.prompt_len)))
    torch.cuda.synchronize()
    if int(server.block.status):
        raise SystemExit("a row had no place in the cache")
    print("decode: rows", tuple(y.shape), "tokens", server.kv_len.tolist(), "mean |y|", float(y.float().abs().mean()))


if __name__ == "__main__":
    main()
