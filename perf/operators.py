"""Work on the paged key/value cache around the multi-LoRA projections, as cases to measure.

Three operators of one decode or prompt step:

* ``append``: rotate the step's queries and keys by their positions and write keys and values into the pages of
  each sequence (``lora_kv_append``);
* ``window``: attention of the step's rows over those pages, with a sliding window and a few first tokens that
  stay visible (``lora_attn_paged``; window 0 is plain causal attention);
* ``prefix``: the same for groups of sequences that share a long prefix held once (``lora_attn_prefix``).

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits, over the batch padded to its
longest sequence.  Head layouts are those of the 8B (32 query heads on 8) and 70B (64 on 8) layers, 128 wide, and a
few odd ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")
MOST_SCORES = 2.7e9     # padded scores of one attention case
MOST_ROWS = 20000       # rows of an append in the widest layout
MOST_KV = 5.0e8         # padded elements of one attention case's keys


def _case(name, op, **kw):
    base = dict(name=name, op=op, dtype="bf16", given="bf16", hq=32, hkv=8, d=128, page=16, heads_first=True,
                decodes=0, prompts=0, prompt_lo=1, prompt_hi=1, idle=0, ctx_lo=0, ctx_hi=0, window=0, sinks=0,
                groups=0, prefix_lo=0, prefix_hi=0, rot=128, interleaved=False, mix=1)
    base.update(kw)
    return base


def listed():
    return [
        # one decode step of 32 single-token requests on an 8B layer: latency
        _case("append-decode-8b", "append", decodes=32, ctx_lo=16, ctx_hi=500),
        # chunked prefill: 64 decode rows and four prompt pieces of 512, fp32 projections, half of each head rotated
        # in neighbouring pairs, pages of 64 tokens with the token outside the head
        _case("append-mixed-f32-in", "append", given="f32", decodes=64, prompts=4, prompt_lo=512, prompt_hi=512,
              ctx_lo=1, ctx_hi=700, page=64, heads_first=False, rot=64, interleaved=True, mix=2),
        # a whole prompt batch on a 70B layer: 16 requests of 128 to 2048 tokens
        _case("append-prefill-70b", "append", prompts=16, prompt_lo=128, prompt_hi=2048, hq=64, mix=3),
        # the smallest attention: odd everything, fp32, an idle sequence among them
        _case("window-tiny-f32", "window", dtype="f32", hq=12, hkv=4, d=64, page=8, decodes=4, prompts=1, prompt_lo=37,
              prompt_hi=37, idle=1, ctx_lo=0, ctx_hi=300, window=100, sinks=3, mix=4),
        # the decode step of 32 requests with ordinary contexts
        _case("window-decode-8b", "window", decodes=32, ctx_lo=64, ctx_hi=2047, mix=5),
        # 256 requests on a model with a sliding window and sinks
        _case("window-decode-256-sinks", "window", decodes=256, ctx_lo=100, ctx_hi=4000, window=1024, sinks=4, page=32,
              mix=6),
        # few requests with long contexts: the time is the cache's bytes
        _case("window-decode-long-70b", "window", decodes=8, hq=64, ctx_lo=16000, ctx_hi=60000, page=64, mix=7),
        # chunked prefill on a 70B layer: decode rows and prompt pieces over earlier context, window and sinks
        _case("window-chunk-70b", "window", decodes=16, prompts=4, prompt_lo=512, prompt_hi=512, hq=64, ctx_lo=1,
              ctx_hi=3500, window=2048, sinks=4, heads_first=False, mix=8),
        # one long prompt from nothing: the matrix units' case
        _case("window-prefill-8k-8b", "window", prompts=1, prompt_lo=8192, prompt_hi=8192, page=64, mix=9),
        # 32 requests of one tenant behind one system prompt
        _case("prefix-decode-8b", "prefix", decodes=32, ctx_lo=16, ctx_hi=500, groups=1, prefix_lo=4096,
              prefix_hi=4096, mix=10),
        # 256 requests of eight adapters, each with a prompt of its own, on a 70B layer
        _case("prefix-decode-8-adapters-70b", "prefix", decodes=256, hq=64, ctx_lo=32, ctx_hi=1000, groups=8,
              prefix_lo=1000, prefix_hi=8000, page=32, mix=11),
        # twelve new prompts behind three shared prefixes
        _case("prefix-prompts-8b", "prefix", prompts=12, prompt_lo=33, prompt_hi=160, groups=3, prefix_lo=1500,
              prefix_hi=2500, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def _propose(rng):
    op = rng.choice(["append", "window", "window", "prefix"])
    hq, hkv = rng.choice([(32, 8), (32, 8), (64, 8), (64, 8), (16, 16), (12, 4), (8, 1), (5, 1)])
    d = rng.choice([64, 128, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    c = _case("", op, dtype=dtype, hq=hq, hkv=hkv, d=d, page=rng.choice([8, 16, 16, 32, 64, 128]),
              heads_first=rng.random() < 0.6, mix=rng.randrange(1 << 20), idle=rng.choice([0, 0, 1]))
    del c["name"]
    kind = rng.choice(["decode", "decode", "mixed", "prompt"])
    if kind != "prompt":
        c["decodes"] = _log(rng, 1, 256)
    if kind != "decode":
        c["prompts"] = _log(rng, 1, 12)
        c["prompt_hi"] = _log(rng, 2, 2048)
        c["prompt_lo"] = max(1, c["prompt_hi"] // rng.choice([1, 2, 8]))
    c["ctx_hi"] = _log(rng, 4, 30000 if kind == "decode" and c["decodes"] <= 16 else 6000)
    c["ctx_lo"] = rng.choice([0, c["ctx_hi"] // 8, c["ctx_hi"] // 2])
    c["rot"] = rng.choice([d, d, d // 2])
    c["interleaved"] = rng.random() < 0.4
    if op == "append":
        c["given"] = rng.choice(["bf16", "f32"])
        c["ctx_hi"] = min(c["ctx_hi"], 600)
        c["ctx_lo"] = min(c["ctx_lo"], 300)
        c["groups"] = 0
    elif rng.random() < 0.6 and op == "window":
        c["window"] = _log(rng, 16, 4096)
        c["sinks"] = rng.choice([0, 1, 4, 16])
    if op == "prefix":
        c["ctx_hi"] = min(c["ctx_hi"], 1000)
        c["ctx_lo"] = min(c["ctx_lo"], 500)
        c["groups"] = min(c["decodes"] + c["prompts"] + c["idle"], _log(rng, 1, 8))
        c["prefix_hi"] = _log(rng, 64, 8000)
        c["prefix_lo"] = rng.choice([c["prefix_hi"], c["prefix_hi"] // 3])
    return c


def _fits(c):
    b = _batch(c)
    rows, longest = sum(b["nq"]), max(b["len"])
    if rows < 1 or len(b["nq"]) * longest * c["hkv"] * c["d"] > MOST_KV:
        return False
    if c["op"] == "append":
        return rows * (c["hq"] + 2 * c["hkv"]) * c["d"] <= MOST_ROWS * 80 * 128 * 0.9
    widest = max(b["nq"])
    scores = len(b["nq"]) * widest * c["hq"] * longest
    if c["groups"]:
        scores += c["groups"] * max(b["group_rows"]) * c["hq"] * max(b["prefix"])
    return scores <= MOST_SCORES and work(c)["flops"] <= (6e11 if c["dtype"] == "bf16" else 2e11)


def draw(rng):
    while True:
        c = _propose(rng)
        if _fits(c):
            return c


def _batch(c):
    """The step's structure, from the case alone: rows and lengths of each sequence, groups and prefix lengths."""
    rng = random.Random(c["mix"])
    kinds = ["d"] * c["decodes"] + ["p"] * c["prompts"] + ["i"] * c["idle"]
    rng.shuffle(kinds)
    nq = [1 if k == "d" else 0 if k == "i" else rng.randint(c["prompt_lo"], c["prompt_hi"]) for k in kinds]
    ctx = [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in kinds]
    out = {"nq": nq, "len": [a + b for a, b in zip(nq, ctx)], "prefix": [], "group_of": [0] * len(nq), "group_off": [0]}
    if c["groups"]:
        cuts = sorted(rng.sample(range(1, len(nq)), c["groups"] - 1)) if c["groups"] > 1 else []
        out["group_off"] = [0] + cuts + [len(nq)]
        out["prefix"] = [rng.randint(c["prefix_lo"], c["prefix_hi"]) for _ in range(c["groups"])]
        out["group_of"] = [g for g in range(c["groups"]) for _ in range(out["group_off"][g + 1] - out["group_off"][g])]
    off = out["group_off"]
    out["group_rows"] = [sum(nq[off[g]:off[g + 1]]) for g in range(len(off) - 1)]
    return out


def _seen(p, window, sinks):
    """How many of the keys 0 .. p a row at position p sees."""
    if not window or p + 1 <= window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def work(c):
    b = _batch(c)
    rows = sum(b["nq"])
    e = {"bf16": 2, "f32": 4}[c["dtype"]]
    kv_row = c["hkv"] * c["d"]
    if c["op"] == "append":
        g = {"bf16": 2, "f32": 4}[c["given"]]
        per = (c["hq"] + 2 * c["hkv"]) * c["d"]
        reach = max(b["len"])
        return {"bytes": rows * per * (g + e) + min(rows, reach) * c["rot"] * 4,
                "flops": rows * (c["hq"] + c["hkv"]) * c["rot"] * 3}
    pairs, keys = 0, sum(b["prefix"])
    for s, (n, length) in enumerate(zip(b["nq"], b["len"])):
        before = b["prefix"][b["group_of"][s]] if c["groups"] else 0
        pairs += sum(_seen(before + p, c["window"], c["sinks"]) for p in range(length - n, length))
        if n and not c["window"]:
            keys += length
        elif n:
            low = max(0, length - n - c["window"] + 1)
            keys += length - low + min(low, c["sinks"])
    return {"bytes": keys * 2 * kv_row * e + 2 * rows * c["hq"] * c["d"] * e + rows * c["hq"] * 4,
            "flops": 4 * pairs * c["hq"] * c["d"]}


def prepare(case, seed):
    c, b = case, _batch(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    dt, given = DTYPES[c["dtype"]], DTYPES[c["given"]]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    rows = sum(b["nq"])

    def randn(shape, dtype, by=1.0):
        return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * by).to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    need = [-(-n // page) for n in b["len"]]
    need_prefix = [-(-n // page) for n in b["prefix"]]
    n_pages = sum(need) + sum(need_prefix) + 1
    free = list(range(n_pages))
    rng.shuffle(free)

    def table(counts):
        wide = max(counts + [1])
        return ints([[free.pop() for _ in range(n)] + [0] * (wide - n) for n in counts])

    shape = (n_pages, hkv, page, d) if c["heads_first"] else (n_pages, page, hkv, d)
    k, v = randn(shape, dt, 1.3), randn(shape, dt)
    if c["heads_first"]:
        k, v = k.transpose(1, 2), v.transpose(1, 2)   # always seen as [page, token, head, dim]
    starts = [0]
    for n in b["nq"]:
        starts.append(starts[-1] + n)
    s = {"case": c, "k": k, "v": v, "row_off": ints(starts), "kv_len": ints(b["len"]), "pages": table(need),
         "n_rows": rows, "max_rows": max(b["nq"]), "max_len": max(b["len"]), "max_prefix": max(b["prefix"] + [0]),
         "max_group_rows": max(b["group_rows"] + [0])}
    if c["groups"]:
        s.update(group_off=ints(b["group_off"]), prefix_len=ints(b["prefix"]), prefix_pages=table(need_prefix))
    # where each row is, for the padded plain form
    seq = [i for i, n in enumerate(b["nq"]) for _ in range(n)]
    s["row_seq"] = torch.tensor(seq, device=DEV)
    s["row_at"] = torch.tensor([j for n in b["nq"] for j in range(n)], device=DEV)
    s["row_group"] = torch.tensor([b["group_of"][i] for i in seq], device=DEV)
    first = [starts[o] for o in b["group_off"]]
    s["row_at_group"] = torch.tensor([r - first[b["group_of"][i]] if c["groups"] else 0 for r, i in enumerate(seq)],
                                     device=DEV)
    if c["op"] == "append":
        half = c["rot"] // 2
        turn = torch.outer(torch.arange(s["max_len"] + s["max_prefix"], device=DEV, dtype=torch.float64),
                           500000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half))
        s.update(cos=turn.cos().float(), sin=turn.sin().float(), q_out=torch.empty((rows, hq * d), dtype=dt, device=DEV),
                 xq=randn((rows, hq * d), given), xk=randn((rows, hkv * d), given), xv=randn((rows, hkv * d), given))
    else:
        s.update(q=randn((rows, hq * d), dt, 1.3), o=torch.empty((rows, hq * d), dtype=dt, device=DEV),
                 lse=torch.empty((rows, hq), dtype=torch.float32, device=DEV))
    return s


def run(state):
    if own:
        return _run_own(state)
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attention(state)


def _run_own(s):
    from lora_bgmv_shrink_amd import binding as lb

    c = s["case"]
    if "handles" not in s:   # what a program keeps over its layers and steps
        groups = {}
        if c["groups"]:
            groups = dict(group_off=s["group_off"], prefix_len=s["prefix_len"], prefix_pages=s["prefix_pages"],
                          max_prefix_len=s["max_prefix"], max_group_rows=s["max_group_rows"])
        cache = lb.KvCache(s["k"], s["v"])
        batch = lb.KvBatch(s["row_off"], s["kv_len"], s["pages"], s["n_rows"], s["max_rows"], s["max_len"], **groups)
        if c["op"] == "append":
            s["handles"] = (cache, batch, lb.Rope(s["cos"], s["sin"], interleaved=c["interleaved"]))
        else:
            s["handles"] = (cache, batch, lb.attn_workspace(cache, batch, c["hq"]))
    cache, batch, third = s["handles"]
    if c["op"] == "append":
        lb.lora_kv_append(cache, batch, s["xq"], s["xk"], s["xv"], third, q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    call = lb.lora_attn_prefix if c["op"] == "prefix" else lb.lora_attn_paged
    call(cache, batch, s["q"], 1.0 / math.sqrt(c["d"]), window=c["window"], n_sink=c["sinks"], o=s["o"], lse=s["lse"],
         ws=third)
    return {"o": s["o"], "lse": s["lse"]}


# ---- plain forms ---------------------------------------------------------

def _turned(x, cos, sin, interleaved):
    """x [rows, heads, d] fp32 with its first 2 * half dims rotated by [rows, half] angles."""
    half = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _plain_append(s):
    c = s["case"]
    rows, d = s["n_rows"], c["d"]
    nq = s["row_off"][1:] - s["row_off"][:-1]
    at = (s["kv_len"] - nq)[s["row_seq"]] + s["row_at"]
    cos, sin = s["cos"][at], s["sin"][at]
    q = _turned(s["xq"].float().view(rows, c["hq"], d), cos, sin, c["interleaved"])
    k = _turned(s["xk"].float().view(rows, c["hkv"], d), cos, sin, c["interleaved"])
    where = (s["pages"][s["row_seq"], at // c["page"]].long(), at % c["page"])
    s["k"][where] = k.to(s["k"].dtype)
    s["v"][where] = s["xv"].view(rows, c["hkv"], d).to(s["v"].dtype)
    return {"q": q.reshape(rows, c["hq"] * d).to(s["k"].dtype), "k": s["k"], "v": s["v"]}


def _gathered(cache, pages, longest, c):
    """[tables, hkv, longest, d] in fp32 of the tokens that a page table lists."""
    x = cache[pages.long()].float()                       # [tables, pages, page, hkv, d]
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
    k, v = _gathered(s["k"], s["pages"], longest, c), _gathered(s["v"], s["pages"], longest, c)
    there = key < s["kv_len"][:, None]
    v = v.masked_fill_(~there[:, None, :, None], 0.0)
    m, l, o = _part(_padded(s, s["row_seq"], s["row_at"], n, wide), k, v, at.repeat_interleave(share, 1),
                    before[:, None] + key, there, c)
    m, l, o = (_rows_of(x, s["row_seq"], s["row_at"], rows, c) for x in (m, l, o))
    if c["groups"]:
        longest = s["max_prefix"]
        key = torch.arange(longest, device=DEV)
        k, v = (_gathered(x, s["prefix_pages"], longest, c) for x in (s["k"], s["v"]))
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
    return {"o": o.reshape(rows, c["hq"] * c["d"]).to(s["k"].dtype), "lse": lse}


# ---- from the definition, in 64 bits -------------------------------------

def exact(case, seed):
    c, b, s = case, _batch(case), prepare(case, seed)
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    starts = s["row_off"].tolist()
    pages = s["pages"].tolist()
    if c["op"] == "append":
        keys, values, half = s["k"].double(), s["v"].double(), c["rot"] // 2
        q_out = s["xq"].double().view(-1, hq, d).clone()
        k_new, v_new = s["xk"].double().view(-1, hkv, d).clone(), s["xv"].double().view(-1, hkv, d)
        one = torch.arange(half, device=DEV)
        first, second = (2 * one, 2 * one + 1) if c["interleaved"] else (one, one + half)
        for i, (n, length) in enumerate(zip(b["nq"], b["len"])):
            if not n:
                continue
            here = slice(starts[i], starts[i + 1])
            at = torch.arange(length - n, length, device=DEV)
            # a rotation is the product with exp(i * angle)
            unit = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None, :]
            for x in (q_out, k_new):
                z = torch.complex(x[here][..., first], x[here][..., second]) * unit
                x[here][..., first], x[here][..., second] = z.real, z.imag
            slot = torch.tensor(pages[i], device=DEV)[at // page] * page + at % page
            keys[slot // page, slot % page] = k_new[here]
            values[slot // page, slot % page] = v_new[here]
        return {"q": q_out.reshape(-1, hq * d), "k": keys, "v": values}
    share = hq // hkv
    o = torch.zeros((s["n_rows"], hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((s["n_rows"], hq), -INF, dtype=torch.float64, device=DEV)
    prefix_pages = s["prefix_pages"].tolist() if c["groups"] else None

    def tokens(cache, listed_pages, length, h):
        return cache[:, :, h][torch.tensor(listed_pages, device=DEV)].reshape(-1, d)[:length].double()

    for i, (n, length) in enumerate(zip(b["nq"], b["len"])):
        g = b["group_of"][i]
        before = b["prefix"][g] if c["groups"] else 0
        for h in range(hkv if n else 0):
            k, v = tokens(s["k"], pages[i], length, h), tokens(s["v"], pages[i], length, h)
            if before:
                k = torch.cat((tokens(s["k"], prefix_pages[g], before, h), k))
                v = torch.cat((tokens(s["v"], prefix_pages[g], before, h), v))
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
