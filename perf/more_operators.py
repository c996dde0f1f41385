"""Work on a paged key/value cache held in 8 bits and on the tables of a step, as cases to measure.

Four operators of one step of a multi-LoRA server, in the order in which the step calls them:

* ``plan``: from the rows that each request brings, the tables that the projections, the append and the attention of
  the step read: pages are taken from a free stack and given back to it, rows get their request, adapter, position and
  place (``lora_kv_plan``);
* ``append``: rotate the step's queries and keys by their positions and write keys and values into the pages as e4m3
  with a power of two for each block of tokens and key head; a block whose scale grows is written again
  (``lora_kv_append_q8``);
* ``window``: attention of the step's rows over such pages, with a sliding window and a few first tokens that stay
  visible (``lora_attn_paged_q8``; window 0 is plain causal attention);
* ``prefix``: the same for groups of sequences that share a long prefix held once (``lora_attn_prefix_q8``).

With ``own`` false, ``run`` computes them with elementary torch operations: the attention in 32 bits over the batch
padded to its longest sequence, the append in 64 (a rounding to 4 bits and a border between two scales are decided by
the last bits of a rotation).  Head layouts are those of the 8B (32 query heads on 8) and 70B (64 on 8) layers, 128
wide, and a few odd ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")
LARGEST = 448.0          # e4m3
LEAST, MOST = -100, 100  # exponents of a scale
MOST_SCORES = 2.7e9      # padded scores of one attention case
MOST_ROWS = 20000        # rows of an append in the widest layout
MOST_KV = 5.0e8          # padded elements of one attention case's keys
MOST_TABLE = 4.0e6       # page table entries of one plan


def _case(name, op, **kw):
    base = dict(name=name, op=op, given="bf16", hq=32, hkv=8, d=128, page=16, block=16, heads_first=True, decodes=0,
                prompts=0, prompt_lo=1, prompt_hi=1, idle=0, ctx_lo=0, ctx_hi=0, window=0, sinks=0, groups=0,
                prefix_lo=0, prefix_hi=0, rot=128, interleaved=False, over=0, short=0.0, mix=1)
    base.update(kw)
    return base


def listed():
    return [
        # the tables of one decode step of 32 requests: latency
        _case("plan-decode-32", "plan", decodes=32, ctx_lo=16, ctx_hi=500, mix=1),
        # 768 requests of eight adapters behind prefixes: decode rows, prompt pieces, requests that end, and too few
        # free pages for the last ones
        _case("plan-mixed-768", "plan", decodes=600, prompts=48, prompt_lo=20, prompt_hi=1500, idle=20, over=8,
              ctx_lo=0, ctx_hi=4000, groups=8, prefix_lo=500, prefix_hi=2000, short=0.2, mix=2),
        # one decode step of 32 single-token requests on an 8B layer: latency
        _case("append-decode-8b", "append", decodes=32, ctx_lo=16, ctx_hi=500, mix=3),
        # chunked prefill: 64 decode rows and four prompt pieces of 512, fp32 projections, half of each head rotated
        # in neighbouring pairs, pages of 64 tokens in two blocks with the token outside the head
        _case("append-mixed-f32-in", "append", given="f32", decodes=64, prompts=4, prompt_lo=512, prompt_hi=512,
              ctx_lo=1, ctx_hi=700, page=64, block=32, heads_first=False, rot=64, interleaved=True, mix=4),
        # a whole prompt batch on a 70B layer: 16 requests of 128 to 2048 tokens
        _case("append-prefill-70b", "append", prompts=16, prompt_lo=128, prompt_hi=2048, hq=64, mix=5),
        # the smallest attention: odd everything, an idle sequence among them
        _case("window-tiny", "window", hq=12, hkv=4, d=64, page=8, block=4, decodes=4, prompts=1, prompt_lo=37,
              prompt_hi=37, idle=1, ctx_lo=0, ctx_hi=300, window=100, sinks=3, mix=6),
        # the decode step of 32 requests with ordinary contexts
        _case("window-decode-8b", "window", decodes=32, ctx_lo=64, ctx_hi=2047, mix=7),
        # few requests with long contexts: the time is the cache's bytes
        _case("window-decode-long-70b", "window", decodes=8, hq=64, ctx_lo=16000, ctx_hi=60000, page=64, block=64,
              mix=8),
        # chunked prefill on a 70B layer: decode rows and prompt pieces over earlier context, window and sinks
        _case("window-chunk-70b", "window", decodes=16, prompts=4, prompt_lo=512, prompt_hi=512, hq=64, ctx_lo=1,
              ctx_hi=3500, window=2048, sinks=4, page=32, block=16, heads_first=False, mix=9),
        # one long prompt from nothing: the matrix units' case
        _case("window-prefill-8k-8b", "window", prompts=1, prompt_lo=8192, prompt_hi=8192, page=64, block=64, mix=10),
        # 256 requests of eight adapters, each with a prompt of its own, on a 70B layer
        _case("prefix-decode-8-adapters-70b", "prefix", decodes=256, hq=64, ctx_lo=32, ctx_hi=1000, groups=8,
              prefix_lo=1000, prefix_hi=8000, page=32, block=32, mix=11),
        # twelve new prompts behind three shared prefixes
        _case("prefix-prompts-8b", "prefix", prompts=12, prompt_lo=33, prompt_hi=160, groups=3, prefix_lo=1500,
              prefix_hi=2500, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def _propose(rng):
    op = rng.choice(["plan", "append", "window", "window", "prefix"])
    hq, hkv = rng.choice([(32, 8), (32, 8), (64, 8), (64, 8), (16, 16), (12, 4), (8, 1), (5, 1)])
    page = rng.choice([8, 16, 16, 32, 64, 128])
    c = _case("", op, hq=hq, hkv=hkv, d=rng.choice([64, 128, 128, 128]), page=page,
              block=max(4, page // rng.choice([1, 1, 2, 4])), heads_first=rng.random() < 0.6, mix=rng.randrange(1 << 20),
              idle=rng.choice([0, 0, 1]))
    del c["name"]
    kind = rng.choice(["decode", "decode", "mixed", "prompt"])
    if kind != "prompt":
        c["decodes"] = _log(rng, 1, 768 if op == "plan" else 256)
    if kind != "decode":
        c["prompts"] = _log(rng, 1, 48 if op == "plan" else 12)
        c["prompt_hi"] = _log(rng, 2, 2048)
        c["prompt_lo"] = max(1, c["prompt_hi"] // rng.choice([1, 2, 8]))
    c["ctx_hi"] = _log(rng, 4, 30000 if kind == "decode" and c["decodes"] <= 16 and op != "plan" else 6000)
    c["ctx_lo"] = rng.choice([0, c["ctx_hi"] // 8, c["ctx_hi"] // 2])
    c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2])
    c["interleaved"] = rng.random() < 0.4
    if op == "plan":
        c["over"] = rng.choice([0, 1, 3, _log(rng, 1, 100)])
        c["short"] = rng.choice([0.0, 0.0, 0.1, 0.5])
        c["groups"] = rng.choice([0, min(c["decodes"] + c["prompts"], _log(rng, 1, 8))])
    elif op == "append":
        c["given"] = rng.choice(["bf16", "f32"])
        c["ctx_hi"] = min(c["ctx_hi"], 600)
        c["ctx_lo"] = min(c["ctx_lo"], 300)
    elif rng.random() < 0.6 and op == "window":
        c["window"] = _log(rng, 16, 4096)
        c["sinks"] = rng.choice([0, 1, 4, 16])
    if op == "prefix":
        c["ctx_hi"] = min(c["ctx_hi"], 1000)
        c["ctx_lo"] = min(c["ctx_lo"], 500)
        c["groups"] = min(c["decodes"] + c["prompts"] + c["idle"], _log(rng, 1, 8))
    if c["groups"]:
        c["prefix_hi"] = _log(rng, 64, 8000)
        c["prefix_lo"] = rng.choice([c["prefix_hi"], c["prefix_hi"] // 3])
    return c


def _fits(c):
    b = _batch(c)
    rows, longest = sum(b["nq"]), max(b["len"])
    if rows < 1:
        return False
    if c["op"] == "plan":
        return len(b["nq"]) * (longest // c["page"] + 1) <= MOST_TABLE and work(c)["bytes"] <= 6e6
    if len(b["nq"]) * longest * c["hkv"] * c["d"] > MOST_KV:
        return False
    if c["op"] == "append":
        return rows * (c["hq"] + 2 * c["hkv"]) * c["d"] <= MOST_ROWS * 80 * 128 * 0.9
    widest = max(b["nq"])
    scores = len(b["nq"]) * widest * c["hq"] * longest
    if c["groups"]:
        scores += c["groups"] * max(b["group_rows"]) * c["hq"] * max(b["prefix"])
    return scores <= MOST_SCORES and work(c)["flops"] <= 5e11


def draw(rng):
    while True:
        c = _propose(rng)
        if _fits(c):
            return c


def _batch(c):
    """The step's structure, from the case alone: rows and lengths of each sequence, groups and prefix lengths."""
    rng = random.Random(c["mix"])
    kinds = ["d"] * c["decodes"] + ["p"] * c["prompts"] + ["i"] * c["idle"] + ["o"] * c["over"]
    rng.shuffle(kinds)
    nq = [1 if k == "d" else rng.randint(c["prompt_lo"], c["prompt_hi"]) if k == "p" else 0 for k in kinds]
    ctx = [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in kinds]
    out = {"kinds": kinds, "nq": nq, "ctx": ctx, "len": [a + b for a, b in zip(nq, ctx)], "prefix": [],
           "group_of": [0] * len(nq), "group_off": [0]}
    if c["groups"]:
        cuts = sorted(rng.sample(range(1, len(nq)), c["groups"] - 1)) if c["groups"] > 1 else []
        out["group_off"] = [0] + cuts + [len(nq)]
        out["prefix"] = [rng.randint(c["prefix_lo"], c["prefix_hi"]) for _ in range(c["groups"])]
        out["group_of"] = [g for g in range(c["groups"]) for _ in range(out["group_off"][g + 1] - out["group_off"][g])]
    off = out["group_off"]
    out["group_rows"] = [sum(nq[off[g]:off[g + 1]]) for g in range(len(off) - 1)]
    return out


def _new_pages(c, b):
    return sum(-(-n // c["page"]) - -(-before // c["page"]) for n, before in zip(b["len"], b["ctx"]))


def _seen(p, window, sinks):
    """How many of the keys 0 .. p a row at position p sees."""
    if not window or p + 1 <= window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def work(c):
    b = _batch(c)
    rows = sum(b["nq"])
    if c["op"] == "plan":
        # of a sequence: rows, adapter, length, its row offset and new length; of a row: request, adapter, position and
        # a place of 8 bytes; of a page: read from the stack or a table, and written
        back = sum(-(-n // c["page"]) for n, k in zip(b["ctx"], b["kinds"]) if k == "o")
        return {"bytes": 20 * len(b["nq"]) + 20 * rows + 8 * (_new_pages(c, b) + back), "flops": 0}
    kv_row = c["hkv"] * c["d"]
    if c["op"] == "append":
        g = {"bf16": 2, "f32": 4}[c["given"]]
        reach = max(b["len"])
        blocks = sum(-(-n // c["block"]) - before // c["block"] for n, before in zip(b["len"], b["ctx"]) if n > before)
        return {"bytes": rows * (c["hq"] * c["d"] * (g + 2) + 2 * kv_row * (g + 1)) + min(rows, reach) * c["rot"] * 4 +
                blocks * c["hkv"] * 8,
                "flops": rows * (c["hq"] + c["hkv"]) * c["rot"] * 3}
    pairs, keys, blocks = 0, sum(b["prefix"]), sum(-(-n // c["block"]) for n in b["prefix"])
    for s, (n, length) in enumerate(zip(b["nq"], b["len"])):
        before = b["prefix"][b["group_of"][s]] if c["groups"] else 0
        pairs += sum(_seen(before + p, c["window"], c["sinks"]) for p in range(length - n, length))
        seen = 0
        if n and not c["window"]:
            seen = length
        elif n:
            low = max(0, length - n - c["window"] + 1)
            seen = length - low + min(low, c["sinks"])
        keys += seen
        blocks += -(-seen // c["block"])
    return {"bytes": keys * 2 * kv_row + blocks * c["hkv"] * 8 + 4 * rows * c["hq"] * c["d"] + rows * c["hq"] * 4,
            "flops": 4 * pairs * c["hq"] * c["d"]}


# ---- a cache in 8 bits ---------------------------------------------------

def _two_to(e):
    """2^e in 64 bits, from its bits: a power function may be off by one of its last ones."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _power(top):
    """The least power of two (exponent) that brings values up to `top` (64 bits) within e4m3's range."""
    m, e = torch.frexp(top)                      # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = e.to(torch.int32) - 9 + (m > 0.875)
    return torch.where(top > 0, e, LEAST).clamp(LEAST, MOST)


def _to_e4m3(x):
    """x (64 bits, at most 448 in magnitude) rounded to e4m3, to nearest, ties to even: a float8 tensor."""
    step = torch.frexp(x)[1].clamp(min=-5) - 4   # 4 significant bits from 2^-6 on, a fixed step of 2^-9 below
    unit = _two_to(step)
    return (torch.round(x / unit) * unit).float().to(torch.float8_e4m3fn)


def _filled(x, block):
    """x [pages, tokens, heads, d] fp32 as an 8-bit cache: (e4m3, scales [pages, blocks, heads] fp32)."""
    p, t, h, d = x.shape
    top = x.view(p, t // block, block, h, d).abs().amax((2, 4))
    m, e = torch.frexp(top)
    e = (e - 9 + (m > 0.875)).clamp(LEAST, MOST)
    s = _two_to(e).float()
    return (x.view(p, t // block, block, h, d) / s[:, :, None, :, None]).view(p, t, h, d).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    c, b = case, _batch(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    rows = sum(b["nq"])

    def randn(shape, dtype, by=1.0):
        return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * by).to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    s = {"case": c}
    if c["groups"]:
        s.update(group_off=ints(b["group_off"]), prefix_len=ints(b["prefix"]))
    if c["op"] == "plan":
        # what the requests hold before the step, and a stack of the other pages: what the step needs and some more,
        # or less by the share `short`
        held = [-(-n // page) for n in b["ctx"]]
        back = sum(n for n, k in zip(held, b["kinds"]) if k == "o")
        need = _new_pages(c, b)
        spare = max(0, int(need * (1.0 - c["short"])) - back) if c["short"] else need + 64
        n_pages = sum(held) + spare
        order = list(range(n_pages))
        rng.shuffle(order)
        wide = max(-(-n // page) for n in b["len"]) + 2
        table = [[order.pop() for _ in range(n)] + [-1] * (wide - n) for n in held]
        s.update(new_rows=ints([-1 if k == "o" else n for n, k in zip(b["nq"], b["kinds"])]),
                 adapter=ints([rng.randrange(-1, 20) for _ in b["nq"]]), kv_len=ints(b["ctx"]), pages=ints(table),
                 free_pages=ints(order + [-1] * (n_pages - len(order))), n_free=ints([spare]), max_rows=rows + 7,
                 kv_len_out=ints(b["ctx"]), n_free_out=ints([0]), status=ints([0]))
        return s

    need = [-(-n // page) for n in b["len"]]
    need_prefix = [-(-n // page) for n in b["prefix"]]
    n_pages = sum(need) + sum(need_prefix) + 1
    free = list(range(n_pages))
    rng.shuffle(free)

    def table(counts):
        wide = max(counts + [1])
        return ints([[free.pop() for _ in range(n)] + [0] * (wide - n) for n in counts])

    # heads differ in size, and so do tokens a little
    gain = torch.exp(0.5 * randn((2, 1, 1, hkv, 1), torch.float32))
    token = torch.exp(0.3 * randn((n_pages, page, 1, 1), torch.float32))
    halves = []
    for x, by in ((randn((n_pages, page, hkv, d), torch.float32), 1.0), (randn((n_pages, page, hkv, d), torch.float32), 3.0)):
        halves += _filled(x * gain[len(halves) // 2] * (token if by != 1.0 else 1.0) * by, c["block"])
    k, k_scale, v, v_scale = halves
    if c["heads_first"]:
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))   # always seen as [page, token, head, dim]
    starts = [0]
    for n in b["nq"]:
        starts.append(starts[-1] + n)
    s.update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, row_off=ints(starts), kv_len=ints(b["len"]), pages=table(need),
             n_rows=rows, max_rows=max(b["nq"]), max_len=max(b["len"]), max_prefix=max(b["prefix"] + [0]),
             max_group_rows=max(b["group_rows"] + [0]))
    if c["groups"]:
        s["prefix_pages"] = table(need_prefix)
    # where each row is, for the padded plain form
    seq = [i for i, n in enumerate(b["nq"]) for _ in range(n)]
    s["row_seq"] = torch.tensor(seq, device=DEV)
    s["row_at"] = torch.tensor([j for n in b["nq"] for j in range(n)], device=DEV)
    s["row_group"] = torch.tensor([b["group_of"][i] for i in seq], device=DEV)
    first = [starts[o] for o in b["group_off"]]
    s["row_at_group"] = torch.tensor([r - first[b["group_of"][i]] if c["groups"] else 0 for r, i in enumerate(seq)],
                                     device=DEV)
    if c["op"] == "append":
        given = DTYPES[c["given"]]
        half = c["rot"] // 2
        turn = torch.outer(torch.arange(s["max_len"] + s["max_prefix"], device=DEV, dtype=torch.float64),
                           500000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half))
        # new rows are of the cache's sizes: now and then one is larger than what its block holds
        flat = gain.reshape(2, hkv, 1)
        s.update(cos=turn.cos().float(), sin=turn.sin().float(),
                 q_out=torch.empty((rows, hq * d), dtype=torch.bfloat16, device=DEV),
                 xq=randn((rows, hq * d), given), xk=(randn((rows, hkv, d), torch.float32) * flat[0]).view(rows, -1).to(given),
                 xv=(randn((rows, hkv, d), torch.float32, 3.0) * flat[1]).view(rows, -1).to(given))
    else:
        s.update(q=randn((rows, hq * d), torch.bfloat16, 1.3),
                 o=torch.empty((rows, hq * d), dtype=torch.bfloat16, device=DEV),
                 lse=torch.empty((rows, hq), dtype=torch.float32, device=DEV))
    return s


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return _plain_plan(state) if op == "plan" else _plain_append(state) if op == "append" else _plain_attention(state)


def _run_own(s):
    from lora_bgmv_shrink_amd import binding as lb

    c = s["case"]
    groups = dict(group_off=s["group_off"], prefix_len=s["prefix_len"]) if c["groups"] else {}
    if c["op"] == "plan":
        if "handles" not in s:   # what a program keeps over its steps
            s["handles"] = lb.KvPlan(s["kv_len"], s["pages"], s["free_pages"], s["n_free"], c["page"], s["max_rows"],
                                     kv_len_out=s["kv_len_out"], n_free_out=s["n_free_out"], **groups)
        plan = s["handles"]
        lb.lora_kv_plan(plan, s["new_rows"], s["adapter"], status=s["status"])
        return {"row_off": plan.row_off, "row_seq": plan.row_seq, "row_adapter": plan.row_adapter,
                "row_pos": plan.row_pos, "row_slot": plan.row_slot, "kv_len": s["kv_len_out"], "pages": s["pages"],
                "free_pages": s["free_pages"], "n_free": s["n_free_out"], "status": s["status"]}
    if "handles" not in s:   # what a program keeps over its layers and steps
        if c["groups"]:
            groups.update(prefix_pages=s["prefix_pages"], max_prefix_len=s["max_prefix"],
                          max_group_rows=s["max_group_rows"])
        cache = lb.KvCacheQ8(s["k"], s["v"], s["k_scale"], s["v_scale"])
        batch = lb.KvBatch(s["row_off"], s["kv_len"], s["pages"], s["n_rows"], s["max_rows"], s["max_len"], **groups)
        if c["op"] == "append":
            s["handles"] = (cache, batch, lb.Rope(s["cos"], s["sin"], interleaved=c["interleaved"]))
        else:
            s["handles"] = (cache, batch, lb.attn_workspace_q8(cache, batch, c["hq"]))
    cache, batch, third = s["handles"]
    if c["op"] == "append":
        lb.lora_kv_append_q8(cache, batch, s["xq"], s["xk"], s["xv"], third, q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    call = lb.lora_attn_prefix_q8 if c["op"] == "prefix" else lb.lora_attn_paged_q8
    call(cache, batch, s["q"], 1.0 / math.sqrt(c["d"]), window=c["window"], n_sink=c["sinks"], o=s["o"], lse=s["lse"],
         ws=third)
    return {"o": s["o"], "lse": s["lse"]}


# ---- plain forms ---------------------------------------------------------

def _plain_plan(s):
    c = s["case"]
    page, n, wide = c["page"], s["kv_len"].numel(), s["pages"].shape[1]
    want, length = s["new_rows"].long(), s["kv_len"].long()
    held = (length + page - 1) // page
    ends, asks = want < 0, want > 0
    claims = asks & (length + want <= wide * page)
    rows = torch.where(claims, want, 0)
    need = torch.where(claims, (length + want + page - 1) // page - held, 0)
    back = torch.where(ends, held, 0)
    n0 = s["n_free"].long()
    there = n0 + back.sum()
    given = claims & (rows.cumsum(0) <= s["max_rows"]) & ((need == 0) | (need.cumsum(0) <= there))
    rows, need = torch.where(given, rows, 0), torch.where(given, need, 0)
    ends_at, taken, came = rows.cumsum(0), need.cumsum(0), back.cumsum(0)
    # the stack with the pages that come back on top; pages are taken from there
    i = torch.arange(s["free_pages"].numel(), device=DEV)
    giver = torch.searchsorted(came, (i - n0).contiguous(), right=True).clamp(max=n - 1)
    which = (i - n0 - came[giver] + back[giver]).clamp(0, wide - 1)
    stack = torch.where(i < n0, s["free_pages"].long(), s["pages"][giver, which].long())
    left = there - taken[-1]
    free_pages = torch.where((i >= n0) & (i < left), stack, s["free_pages"].long()).int()
    col = torch.arange(wide, device=DEV)
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    from_top = (taken - need)[:, None] + col - held[:, None]
    picked = stack[(there - 1 - from_top).clamp(0, stack.numel() - 1)]
    pages = torch.where(fresh, picked, s["pages"].long())
    r = torch.arange(s["max_rows"], device=DEV)
    there_is = r < ends_at[-1]
    seq = torch.searchsorted(ends_at, r, right=True).clamp(max=n - 1)
    at = length[seq] + r - (ends_at - rows)[seq]
    slot = pages[seq, torch.where(there_is, at // page, 0)] * page + at % page
    before = torch.zeros_like(length)
    if c["groups"]:
        sizes = (s["group_off"][1:] - s["group_off"][:-1]).long()
        before = torch.repeat_interleave(s["prefix_len"].long(), sizes, output_size=n)
    s["pages"].copy_(pages)
    s["free_pages"].copy_(free_pages)
    s["kv_len_out"].copy_(torch.where(ends, 0, length + rows))
    s["n_free_out"].copy_(left)
    s["status"].copy_(s["status"] | (asks & ~given).any())
    return {"row_off": torch.cat((torch.zeros_like(ends_at[:1]), ends_at)).int(),
            "row_seq": torch.where(there_is, seq, -1).int(),
            "row_adapter": torch.where(there_is, s["adapter"][seq].long(), -1).int(),
            "row_pos": torch.where(there_is, before[seq] + at, -1).int(), "row_slot": torch.where(there_is, slot, -1),
            "kv_len": s["kv_len_out"], "pages": s["pages"], "free_pages": s["free_pages"], "n_free": s["n_free_out"],
            "status": s["status"]}


def _turned(x, cos, sin, interleaved):
    """x [rows, heads, d] with its first 2 * half dims rotated by [rows, half] angles."""
    half = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _plain_put(s, x, cache, scale, at, first):
    """x [rows, hkv, d] (64 bits) into the pages; the tokens of a block that were there before are scaled with it."""
    c = s["case"]
    blk, page, hkv, d = c["block"], c["page"], c["hkv"], c["d"]
    # the step's blocks, numbered by their first rows
    opens = (at % blk == 0) | (s["row_at"] == 0)
    unit = torch.cumsum(opens, 0) - 1
    lead = torch.nonzero(opens)[:, 0]
    seq, start = s["row_seq"][lead], at[lead] // blk * blk
    held = s["pages"][seq, start // page].long()
    part = start % page // blk
    top = torch.zeros((lead.numel(), hkv), dtype=torch.float64, device=DEV)
    top = top.index_reduce(0, unit, x.abs().amax(2), "amax")
    power = _power(top)
    old = scale[held, part].double()
    kept = first[seq] > start                    # tokens of earlier steps in the block
    old_power = torch.frexp(old)[1] - 1
    power = torch.where(kept[:, None], torch.maximum(power, old_power), power)
    new = _two_to(power)
    # tokens before the step's, under the new scale
    token = start[:, None] + torch.arange(blk, device=DEV)
    which, i = torch.nonzero(token < first[seq][:, None], as_tuple=True)
    where = (held[which], (start % page)[which] + i)
    raw = cache.view(torch.uint8)
    there = raw[where].view(torch.float8_e4m3fn).double()
    raw[where] = _to_e4m3(there * (old / new)[which][:, :, None]).view(torch.uint8)
    row_page = s["pages"][s["row_seq"], at // page].long()
    raw[row_page, at % page] = _to_e4m3(x / new[unit][:, :, None]).view(torch.uint8)
    scale[held, part] = new.float()


def _plain_append(s):
    c = s["case"]
    rows, d = s["n_rows"], c["d"]
    nq = s["row_off"][1:] - s["row_off"][:-1]
    first = (s["kv_len"] - nq).long()
    at = first[s["row_seq"]] + s["row_at"]
    cos, sin = s["cos"][at], s["sin"][at]
    q = _turned(s["xq"].float().view(rows, c["hq"], d), cos, sin, c["interleaved"])
    k = _turned(s["xk"].double().view(rows, c["hkv"], d), cos.double(), sin.double(), c["interleaved"])
    _plain_put(s, k, s["k"], s["k_scale"], at, first)
    _plain_put(s, s["xv"].double().view(rows, c["hkv"], d), s["v"], s["v_scale"], at, first)
    return {"q": q.reshape(rows, c["hq"] * d).to(torch.bfloat16), "k": s["k"], "v": s["v"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _gathered(cache, scale, pages, longest, c):
    """[tables, hkv, longest, d] in fp32 of the tokens that a page table lists."""
    raw = cache.view(torch.uint8)[pages.long()].contiguous().view(torch.float8_e4m3fn)
    x = raw.float() * scale[pages.long()].repeat_interleave(c["block"], 2)[..., None]   # [tables, pages, page, hkv, d]
    x = x.flatten(1, 2)[:, :longest]
    return x.transpose(1, 2).contiguous()


def _part(q, k, v, at, key_at, there, c):
    """Unnormalised attention of q [n, hkv, rows, d] over k, v [n, hkv, keys, d]: (max, sum, product).
    at [n, rows] and key_at [n, keys]: positions; there [n, keys]: whether the key exists."""
    scores = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(c["d"]))
    sees = (key_at[:, None, :] <= at[:, :, None]) & there[:, None, :]
    if c["window"]:
        sees = sees & ((key_at[:, None, :] > at[:, :, None] - c["window"]) | (key_at[:, None, :] < c["sinks"]))
    scores = scores.masked_fill_(~sees[:, None], -INF)
    top = scores.amax(-1, keepdim=True)
    scores = torch.exp(scores - torch.where(top == -INF, 0.0, top))
    return top, scores.sum(-1, keepdim=True), torch.matmul(scores, v)


def _rows_of(x, which, at, rows, c):
    """[n, hkv, padded rows * share, e] -> [rows, hq, e]."""
    n, hkv, _, e = x.shape
    x = x.view(n, hkv, -1, c["hq"] // hkv, e)
    return x[which, :, at].reshape(rows, c["hq"], e)


def _padded(s, which, at, n, wide):
    """q in [n, hkv, wide * share, d] fp32, share query heads of one key head side by side, and zeros elsewhere."""
    c = s["case"]
    q = torch.zeros((n, wide, c["hq"], c["d"]), device=DEV)
    q[which, at] = s["q"].float().view(-1, c["hq"], c["d"])
    share = c["hq"] // c["hkv"]
    return q.view(n, wide, c["hkv"], share, c["d"]).transpose(1, 2).reshape(n, c["hkv"], wide * share, c["d"])


def _plain_attention(s):
    c = s["case"]
    rows, share = s["n_rows"], c["hq"] // c["hkv"]
    nq = s["row_off"][1:] - s["row_off"][:-1]
    n, wide, longest = nq.numel(), s["max_rows"], s["max_len"]
    before = torch.zeros_like(s["kv_len"])
    if c["groups"]:
        sizes = s["group_off"][1:] - s["group_off"][:-1]
        before = torch.repeat_interleave(s["prefix_len"], sizes, output_size=n)
    at = (before + s["kv_len"] - nq)[:, None] + torch.arange(wide, device=DEV)
    key = torch.arange(longest, device=DEV)
    k = _gathered(s["k"], s["k_scale"], s["pages"], longest, c)
    v = _gathered(s["v"], s["v_scale"], s["pages"], longest, c)
    there = key < s["kv_len"][:, None]
    v = v.masked_fill_(~there[:, None, :, None], 0.0)
    m, l, o = _part(_padded(s, s["row_seq"], s["row_at"], n, wide), k, v, at.repeat_interleave(share, 1),
                    before[:, None] + key, there, c)
    m, l, o = (_rows_of(x, s["row_seq"], s["row_at"], rows, c) for x in (m, l, o))
    if c["groups"]:
        longest = s["max_prefix"]
        key = torch.arange(longest, device=DEV)
        k = _gathered(s["k"], s["k_scale"], s["prefix_pages"], longest, c)
        v = _gathered(s["v"], s["v_scale"], s["prefix_pages"], longest, c)
        there = key < s["prefix_len"][:, None]
        v = v.masked_fill_(~there[:, None, :, None], 0.0)
        at_group = torch.zeros((c["groups"], s["max_group_rows"]), dtype=at.dtype, device=DEV)
        at_group[s["row_group"], s["row_at_group"]] = at[s["row_seq"], s["row_at"]]
        q = _padded(s, s["row_group"], s["row_at_group"], c["groups"], s["max_group_rows"])
        more = _part(q, k, v, at_group.repeat_interleave(share, 1), key.expand(c["groups"], -1), there, c)
        m2, l2, o2 = (_rows_of(x, s["row_group"], s["row_at_group"], rows, c) for x in more)
        top = torch.maximum(m, m2)
        safe = torch.where(top == -INF, 0.0, top)
        a, b = torch.exp(m - safe), torch.exp(m2 - safe)
        m, l, o = top, l * a + l2 * b, o * a + o2 * b
    lse = (m + torch.log(l)).view(rows, c["hq"])
    o = torch.where(l > 0, o / torch.where(l > 0, l, 1.0), 0.0)
    return {"o": o.reshape(rows, c["hq"] * c["d"]).to(torch.bfloat16), "lse": lse}


# ---- from the definition, in 64 bits -------------------------------------

def _exact_plan(c, b, s):
    page, cap, wide = c["page"], s["max_rows"], s["pages"].shape[1]
    want, length, table = s["new_rows"].tolist(), s["kv_len"].tolist(), s["pages"].tolist()
    adapter, free = s["adapter"].tolist(), s["free_pages"].tolist()
    stack = free[:s["n_free"].item()]
    for i, n in enumerate(want):
        if n < 0:
            stack += table[i][:-(-length[i] // page)]
            length[i] = 0
    row_off, rows, asked_rows, asked_pages, most, refused = [0], [], 0, 0, len(stack), 0
    for i, n in enumerate(want):
        take = max(n, 0)
        if take and length[i] + take > wide * page:
            take, refused = 0, 1
        held, need = -(-length[i] // page), -(-(length[i] + take) // page)
        asked_rows, asked_pages = asked_rows + take, asked_pages + need - held
        if take and (asked_rows > cap or (need > held and asked_pages > most)):
            take, need, refused = 0, held, 1
        for j in range(held, need):
            table[i][j] = stack.pop()
        before = b["prefix"][b["group_of"][i]] if c["groups"] else 0
        for t in range(length[i], length[i] + take):
            rows.append((i, adapter[i], before + t, table[i][t // page] * page + t % page))
        length[i] += take
        row_off.append(len(rows))
    left = len(stack)
    free = stack + free[left:]
    rows += [(-1, -1, -1, -1)] * (cap - len(rows))

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=DEV)

    return {"row_off": ints(row_off), "row_seq": ints([r[0] for r in rows]), "row_adapter": ints([r[1] for r in rows]),
            "row_pos": ints([r[2] for r in rows]), "row_slot": ints([r[3] for r in rows], torch.int64),
            "kv_len": ints(length), "pages": ints(table), "free_pages": ints(free), "n_free": ints([left]),
            "status": ints([refused])}


def _nearest_code(x, codes, borders):
    """The e4m3 value next to x: of two equally near ones the one with the even code."""
    at = torch.searchsorted(borders, x.abs().contiguous())           # borders below |x|
    tie = borders[at.clamp(max=borders.numel() - 1)] == x.abs()
    at = at + (tie & (at % 2 == 1))
    return torch.copysign(codes[at], x)


def _exact_append(c, b, s):
    hq, hkv, d, page, blk = c["hq"], c["hkv"], c["d"], c["page"], c["block"]
    starts, half = s["row_off"].tolist(), c["rot"] // 2
    codes = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    borders = (codes[1:] + codes[:-1]) / 2
    powers = torch.tensor([2.0 ** e for e in range(LEAST, MOST + 1)], dtype=torch.float64, device=DEV)
    q_out = s["xq"].double().view(-1, hq, d).clone()
    fresh = [s["xk"].double().view(-1, hkv, d).clone(), s["xv"].double().view(-1, hkv, d)]
    held = [x.view(torch.uint8).contiguous().view(torch.float8_e4m3fn).double() for x in (s["k"], s["v"])]
    scales = [s["k_scale"].double(), s["v_scale"].double()]
    one = torch.arange(half, device=DEV)
    first, second = (2 * one, 2 * one + 1) if c["interleaved"] else (one, one + half)
    for i, (n, length) in enumerate(zip(b["nq"], b["len"])):
        if not n:
            continue
        here = slice(starts[i], starts[i + 1])
        at = torch.arange(length - n, length, device=DEV)
        # a rotation is the product with exp(i * angle)
        unit = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None, :]
        for x in (q_out, fresh[0]):
            z = torch.complex(x[here][..., first], x[here][..., second]) * unit
            x[here][..., first], x[here][..., second] = z.real, z.imag
        table = s["pages"][i].tolist()
        for t0 in range((length - n) // blk * blk, length, blk):
            lo, hi = max(t0, length - n), min(t0 + blk, length)
            pg, cell, before = table[t0 // page], t0 % page, max(0, length - n - t0)
            for x, cache, scale in zip(fresh, held, scales):
                new = x[starts[i] + lo - (length - n):starts[i] + hi - (length - n)]
                # the first power of two under which the block's largest is no more than 448
                power = powers[torch.searchsorted(powers * LARGEST, new.abs().amax((0, 2)).contiguous()).clamp(max=MOST - LEAST)]
                was = scale[pg, cell // blk].clone()
                if before:
                    power = torch.maximum(power, was)
                    old = cache[pg, cell:cell + before] * was[:, None] / power[:, None]
                    cache[pg, cell:cell + before] = _nearest_code(old, codes, borders)
                cache[pg, cell + lo - t0:cell + hi - t0] = _nearest_code(new / power[:, None], codes, borders)
                scale[pg, cell // blk] = power
    return {"q": q_out.reshape(-1, hq * d), "k": held[0], "v": held[1], "k_scale": scales[0], "v_scale": scales[1]}


def exact(case, seed):
    c, b, s = case, _batch(case), prepare(case, seed)
    if c["op"] == "plan":
        return _exact_plan(c, b, s)
    if c["op"] == "append":
        return _exact_append(c, b, s)
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    starts = s["row_off"].tolist()
    pages = s["pages"].tolist()
    share = hq // hkv
    o = torch.zeros((s["n_rows"], hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((s["n_rows"], hq), -INF, dtype=torch.float64, device=DEV)
    prefix_pages = s["prefix_pages"].tolist() if c["groups"] else None

    def tokens(which, listed_pages, length, h):
        at = torch.tensor(listed_pages, device=DEV)
        x = s[which][:, :, h].view(torch.uint8)[at].contiguous().view(torch.float8_e4m3fn).double()
        x = x.view(at.numel(), page // c["block"], -1) * s[which + "_scale"][:, :, h][at].double()[..., None]
        return x.reshape(-1, d)[:length]

    for i, (n, length) in enumerate(zip(b["nq"], b["len"])):
        g = b["group_of"][i]
        before = b["prefix"][g] if c["groups"] else 0
        for h in range(hkv if n else 0):
            k, v = tokens("k", pages[i], length, h), tokens("v", pages[i], length, h)
            if before:
                k = torch.cat((tokens("k", prefix_pages[g], before, h), k))
                v = torch.cat((tokens("v", prefix_pages[g], before, h), v))
            key = torch.arange(before + length, device=DEV)
            for r in range(0, n, 1024):
                m = min(1024, n - r)
                rows = slice(starts[i] + r, starts[i] + r + m)
                p = torch.arange(before + length - n + r, before + length - n + r + m, device=DEV)[:, None]
                hidden = key > p
                if c["window"]:
                    hidden |= (key <= p - c["window"]) & (key >= c["sinks"])
                q = s["q"][rows].double().view(m, hq, d)[:, h * share:(h + 1) * share]
                x = torch.matmul(q.reshape(m * share, d), k.t()).view(m, share, -1) / math.sqrt(d)
                x = x.masked_fill(hidden[:, None, :], -INF)
                lse[rows, h * share:(h + 1) * share] = torch.logsumexp(x, -1)
                weights = torch.softmax(x, -1)
                o[rows, h * share:(h + 1) * share] = torch.matmul(weights.view(m * share, -1), v).view(m, share, d)
    return {"o": o.reshape(-1, hq * d), "lse": lse}
