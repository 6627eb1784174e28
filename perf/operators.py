"""The operators of a decode step over a paged key-value cache: what is measured, and their plain forms.

A hybrid decoder's softmax-attention layers keep keys and values in pages of a fixed number of tokens.  Four operators
make one step of such a program: block tables and slot maps from the requests' lengths (`tables`), the new tokens' keys
and values written through the slot map (`append`), attention of one new token per request over its pages (`attend`),
and the next token from the logits (`sample`).
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0


# ---- the cases ------------------------------------------------------------------------------------------------------
def listed():
    return [
        # every running request of a small server adds one token: pure latency, once per step
        {"name": "tables_step", "op": "tables", "requests": 64, "page": 16, "cached": 8192, "new": 1, "max_pages": 640},
        # many requests add a prompt chunk each, some nothing: a long slot map
        {"name": "tables_chunk", "op": "tables", "requests": 1021, "page": 64, "cached": 20000, "new": 511, "max_pages": 512},
        # one new token per request, written in every attention layer of every step
        {"name": "append_step", "op": "append", "tokens": 64, "kv_heads": 8, "dim": 128, "page": 16, "type": "bf16", "cache": "bf16",
         "head_major": False},
        # the keys and values of a whole prompt go into an 8-bit cache
        {"name": "append_prompt_e4m3", "op": "append", "tokens": 32805, "kv_heads": 8, "dim": 128, "page": 64, "type": "bf16", "cache": "e4m3",
         "head_major": True},
        # the first tokens of a single chat: one short row
        {"name": "attend_first", "op": "attend", "requests": 1, "longest": 37, "fill": "full", "q_heads": 16, "kv_heads": 2, "dim": 128, "page": 16,
         "cache": "bf16", "head_major": False, "window": 0},
        # a busy server's ordinary step: ragged lengths, one of them empty
        {"name": "attend_step", "op": "attend", "requests": 64, "longest": 8192, "fill": "ragged", "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "cache": "bf16", "head_major": False, "window": 0},
        # one very long document: few rows, the cache's length has to fill the GPU
        {"name": "attend_long", "op": "attend", "requests": 1, "longest": 131072, "fill": "full", "q_heads": 16, "kv_heads": 4, "dim": 128, "page": 64,
         "cache": "bf16", "head_major": True, "window": 0},
        # long contexts in an 8-bit cache, the type that lets them fit
        {"name": "attend_e4m3", "op": "attend", "requests": 32, "longest": 32768, "fill": "ragged", "q_heads": 32, "kv_heads": 4, "dim": 128, "page": 64,
         "cache": "e4m3", "head_major": True, "window": 0},
        # wide heads with a sliding window: every row reads the window's tail only
        {"name": "attend_window", "op": "attend", "requests": 48, "longest": 16384, "fill": "ragged", "q_heads": 16, "kv_heads": 2, "dim": 256, "page": 32,
         "cache": "bf16", "head_major": False, "window": 4096},
        # 32-bit storage, as a parity run keeps it; pages that are no power of two
        {"name": "attend_f32", "op": "attend", "requests": 9, "longest": 4099, "fill": "ragged", "q_heads": 12, "kv_heads": 4, "dim": 64, "page": 48,
         "cache": "f32", "head_major": False, "window": 0},
        # one chat's next token with the usual filters
        {"name": "sample_one", "op": "sample", "rows": 1, "vocab": 131072, "type": "bf16", "filters": "usual"},
        # a large batch in which every request brings its own settings, greedy and unfiltered ones among them
        {"name": "sample_batch", "op": "sample", "rows": 256, "vocab": 100003, "type": "f32", "filters": "mixed"},
    ]


def _log(rng, low, high):
    """A whole number in [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "attend", "sample"])
    if op == "tables":
        page, requests = rng.choice([1, 8, 16, 32, 48, 64, 128]), _log(rng, 1, 1021)
        new = rng.choice([1, _log(rng, 1, 511)])
        cached = _log(rng, 1, min(20000, 512 * page))
        return {"op": op, "requests": requests, "page": page, "cached": cached, "new": new, "max_pages": (cached + new) // page + 1 + rng.randrange(8)}
    if op == "append":
        cache = rng.choice(["bf16", "bf16", "f32", "e4m3"])
        heads, dim = rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([64, 128, 256])
        tokens = _log(rng, 1, 32805 * 1024 // (heads * dim * (2 if cache == "f32" else 1)))
        return {"op": op, "tokens": tokens, "kv_heads": heads, "dim": dim, "page": rng.choice([1, 16, 24, 32, 64, 128]),
                "type": rng.choice(["bf16", "f32"]) if cache == "e4m3" else cache, "cache": cache, "head_major": rng.random() < 0.5}
    if op == "attend":
        cache, dim = rng.choice(["bf16", "bf16", "e4m3", "f32"]), rng.choice([64, 128, 128, 256])
        heads, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
        requests = _log(rng, 1, 256)
        # values of K, were every row as long as the longest: no more than the largest listed case reads
        most = (130_000_000 if cache == "f32" else 260_000_000) // (requests * heads * dim)
        longest = _log(rng, 1, max(1, min(131072, most)))
        return {"op": op, "requests": requests, "longest": longest, "fill": rng.choice(["ragged", "ragged", "full"]), "q_heads": heads * group,
                "kv_heads": heads, "dim": dim, "page": rng.choice([1, 16, 24, 32, 64, 128]), "cache": cache, "head_major": rng.random() < 0.5,
                "window": rng.choice([0, 0, _log(rng, 1, longest)])}
    vocab = _log(rng, 1000, 160000)
    return {"op": op, "rows": _log(rng, 1, min(256, 256 * 100003 // vocab)), "vocab": vocab, "type": rng.choice(["bf16", "f32"]),
            "filters": rng.choice(["usual", "mixed", "none"])}


def _lengths(case, longest, some_empty=True):
    """The requests' lengths: the case's own, whatever the seed."""
    n = case["requests"]
    if case.get("fill", "ragged") == "full":
        return [longest] * n
    r = random.Random(n * 1000003 + longest)
    got = [r.randint(1, longest) for _ in range(n)]
    got[r.randrange(n)] = longest
    if some_empty and n >= 8:
        got[r.choice([i for i in range(n) if got[i] != longest] or [0])] = 0
    return got


# ---- what a program has in hand --------------------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    return {"tables": _prepare_tables, "append": _prepare_append, "attend": _prepare_attend, "sample": _prepare_sample}[case["op"]](case, seed, dev, gen)


def _table_lengths(case):
    n = case["requests"]
    cached = _lengths(case, case["cached"])
    if case["new"] == 1:
        return cached, [1] * n
    r = random.Random(n * 7919 + case["new"])
    return cached, [r.choice([0, r.randint(1, case["new"]), case["new"]]) for _ in range(n)]


def _prepare_tables(case, seed, dev, gen):
    page, wide = case["page"], case["max_pages"]
    cached, new = _table_lengths(case)
    old = torch.tensor([-(-c // page) for c in cached], device=dev)
    total = int(old.sum())
    need = sum(-(-(c + n) // page) for c, n in zip(cached, new)) - total
    ids = torch.randperm(total + need + 64, device=dev, generator=gen).to(torch.int32)
    # the pages that the requests hold already are dealt out in order; the rest are free
    at = torch.cumsum(old, 0)[:, None] - old[:, None] + torch.arange(wide, device=dev)
    held = torch.arange(wide, device=dev) < old[:, None]
    table = torch.where(held, ids[torch.where(held, at, 0)], -1).to(torch.int32)
    # a step's slot map has room for every token that the batch may add; a captured step keeps this length
    return {"op": "tables", "page": page, "cached": torch.tensor(cached, dtype=torch.int32, device=dev),
            "new": torch.tensor(new, dtype=torch.int32, device=dev), "free": ids[total:].contiguous(), "table": table,
            "n_slots": case["requests"] * case["new"]}


def _cache(case, pages, dev, gen):
    """Keys and values [pages, page, kv_heads, dim], in either storage order, and the 8-bit cache's scales."""
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    shape = (pages, heads, page, dim) if case["head_major"] else (pages, page, heads, dim)

    def values():
        if case["cache"] != "e4m3":
            return torch.randn(shape, device=dev, generator=gen, dtype=TYPES[case["cache"]])
        # calibrated: the largest value met is a little below the format's largest
        return (torch.randn(shape, device=dev, generator=gen, dtype=torch.bfloat16) * 80.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)

    def scale():
        return 0.01 + 0.004 * torch.rand(heads, device=dev, generator=gen) if case["cache"] == "e4m3" else None

    k, v = values(), values()
    return (k.transpose(1, 2), v.transpose(1, 2), scale(), scale()) if case["head_major"] else (k, v, scale(), scale())


def _prepare_append(case, seed, dev, gen):
    n, heads, dim, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    pages = -(-n // page) + 8
    k_cache, v_cache, k_scale, v_scale = _cache(case, pages, dev, gen)
    # keys and values are slices of one projection's output, as a layer makes them
    kv = torch.randn((n, 2 * heads, dim), device=dev, generator=gen, dtype=TYPES[case["type"]])
    slots = torch.randperm(pages, device=dev, generator=gen)[:, None] * page + torch.arange(page, device=dev)
    slots = slots.reshape(-1)[:n].contiguous()
    if n >= 16:
        slots[n - 1 - n // 16:] = -1  # the padding of a captured step
    return {"op": "append", "k": kv[:, :heads], "v": kv[:, heads:], "slots": slots, "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale,
            "v_scale": v_scale, "page": page}


def _prepare_attend(case, seed, dev, gen):
    page, b = case["page"], case["requests"]
    lengths = _lengths(case, case["longest"])
    wide = -(-case["longest"] // page)
    need = torch.tensor([-(-n // page) for n in lengths], device=dev)
    pages = int(need.sum()) + 3
    k_cache, v_cache, k_scale, v_scale = _cache(case, pages, dev, gen)
    ids = torch.randperm(pages, device=dev, generator=gen).to(torch.int32)
    held = torch.arange(wide, device=dev) < need[:, None]
    at = torch.cumsum(need, 0)[:, None] - need[:, None] + torch.arange(wide, device=dev)
    table = torch.where(held, ids[torch.where(held, at, 0)], -1).to(torch.int32)
    kind = torch.float32 if case["cache"] == "f32" else torch.bfloat16
    q = (2.0 * torch.randn((b, case["q_heads"], case["dim"]), device=dev, generator=gen)).to(kind)
    return {"op": "attend", "q": q, "k_cache": k_cache, "v_cache": v_cache, "table": table, "lengths": torch.tensor(lengths, dtype=torch.int32, device=dev),
            "k_scale": k_scale, "v_scale": v_scale, "window": case["window"]}


def _prepare_sample(case, seed, dev, gen):
    rows, vocab = case["rows"], case["vocab"]
    logits = 2.5 * torch.randn((rows, vocab), device=dev, generator=gen)
    # a few tokens stand out, as they do after a trained model's last layer
    peak = torch.randint(0, vocab // 8, (rows, 8), device=dev, generator=gen) + vocab // 8 * torch.arange(8, device=dev)
    logits.scatter_add_(1, peak, 8.0 * torch.rand((rows, 8), device=dev, generator=gen))
    banned = torch.randint(0, vocab, (rows, 5), device=dev, generator=gen)
    logits.scatter_(1, banned, float("-inf"))
    noise = torch.rand((rows, vocab), device=dev, generator=gen)
    r = random.Random(seed)
    given = {"temperature": [0.8] * rows, "top_k": [50] * rows, "top_p": [0.9] * rows, "min_p": [0.02] * rows}
    if case["filters"] == "mixed":
        given = {"temperature": [r.choice([0.0, 0.3, 0.7, 1.0, 1.3]) for _ in range(rows)], "top_k": [r.choice([0, 0, 1, 20, 200, 5000]) for _ in range(rows)],
                 "top_p": [r.choice([1.0, 1.0, 0.5, 0.9, 0.95]) for _ in range(rows)], "min_p": [r.choice([0.0, 0.0, 0.05]) for _ in range(rows)]}
    state = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device=dev) for k, v in given.items()}
    if case["filters"] == "none":
        state = {"temperature": state["temperature"], "top_k": None, "top_p": None, "min_p": None}
    return {"op": "sample", "logits": logits.to(TYPES[case["type"]]), "noise": noise, **state}


# ---- one pass ----------------------------------------------------------------------------------------------------------
def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


def _own_tables(s):
    import gated_delta_rule_16_gb300 as gdn
    slots, positions, seq_lens, cu_new, counts = gdn.gdn_page_tables(s["new"], s["free"], s["table"], page=s["page"], cached_lens=s["cached"],
                                                                     n_slots=s["n_slots"])
    return {"table": s["table"], "slots": slots, "positions": positions, "seq_lens": seq_lens, "cu_new": cu_new, "counts": counts}


def _own_append(s):
    import gated_delta_rule_16_gb300 as gdn
    gdn.gdn_kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    import gated_delta_rule_16_gb300 as gdn
    o, lse = gdn.gdn_paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                  window=s["window"])
    return {"o": o, "lse": lse}


def _own_sample(s):
    import gated_delta_rule_16_gb300 as gdn
    tokens, logprobs = gdn.gdn_sample(s["logits"], s["noise"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    return {"tokens": tokens, "logprobs": logprobs}


def _plain_tables(s):
    page, table, cached, new, free, n = s["page"], s["table"], s["cached"].long(), s["new"].long(), s["free"], s["n_slots"]
    dev, wide = table.device, table.shape[1]
    length = cached + new
    old = (cached + page - 1) // page
    need = ((length + page - 1) // page).clamp(max=wide)
    more = (need - old).clamp(min=0)
    first = torch.cumsum(more, 0) - more
    j = torch.arange(wide, device=dev)
    at = first[:, None] + j - old[:, None]
    fresh = (j >= old[:, None]) & (j < need[:, None])
    ids = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where(fresh, ids, torch.where(j < old[:, None], table, -1)))
    cu = torch.zeros(new.numel() + 1, dtype=torch.int64, device=dev)
    cu[1:] = torch.cumsum(new, 0)
    t = torch.arange(n, device=dev)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=new.numel() - 1)
    real = t < cu[-1]
    pos = torch.where(real, cached[b] + t - cu[b], 0)
    cell = pos // page
    held = torch.where(real & (cell < wide), table[b, cell.clamp(max=wide - 1)], -1).long()
    slots = torch.where(held >= 0, held * page + pos % page, -1)
    taken = more.sum()
    status = (taken > free.numel()).long() + 2 * ((length + page - 1) // page > wide).any().long() + 4 * (cu[-1] > n).long()
    counts = torch.stack([cu[-1], taken, status, length.max()])
    return {"table": table, "slots": slots, "positions": pos.to(torch.int32), "seq_lens": length.to(torch.int32), "cu_new": cu.to(torch.int32),
            "counts": counts.to(torch.int32)}


def _written(cache, x, scale, page, cell):
    x = x.float()
    if scale is not None:
        x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype).view(torch.uint8)
        cache.view(torch.uint8)[page, cell] = x
    else:
        cache[page, cell] = x.to(cache.dtype)
    return cache


def _plain_append(s):
    slots, page = s["slots"], s["page"]
    keep = slots >= 0
    # a padded row writes once more what the first kept row writes: no row count leaves the GPU
    src = torch.where(keep, torch.arange(slots.numel(), device=slots.device), torch.argmax(keep.to(torch.int32)))
    at, cell = slots[src] // page, slots[src] % page
    return {"k_cache": _written(s["k_cache"], s["k"][src], s["k_scale"], at, cell), "v_cache": _written(s["v_cache"], s["v"][src], s["v_scale"], at, cell)}


def _gathered(cache, scale, at, cell, ok):
    """The cached rows of every request, in 32 bits [requests, longest, kv_heads, dim]; zero where there is none."""
    x = (cache.view(torch.uint8)[at, cell].view(cache.dtype) if scale is not None else cache[at, cell]).float()
    if scale is not None:
        x.mul_(scale[:, None])
    return x.masked_fill_(~ok[:, :, None, None], 0.0)


def _plain_attend(s):
    q, table, lengths, window, page = s["q"], s["table"], s["lengths"].long(), s["window"], s["k_cache"].shape[1]
    b, heads, dim = q.shape
    kv_heads, wide = s["k_cache"].shape[2], table.shape[1]
    j = torch.arange(wide * page, device=q.device)
    at = table.long()[:, j // page]
    ok = (j < lengths[:, None]) & (at >= 0)
    if window:
        ok &= j >= lengths[:, None] - window
    at, cell = at.clamp(min=0), j % page
    x = q.float().view(b, kv_heads, heads // kv_heads, dim) * dim ** -0.5
    score = torch.einsum("bhgd,blhd->bhgl", x, _gathered(s["k_cache"], s["k_scale"], at, cell, ok))
    score.masked_fill_(~ok[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgl,blhd->bhgd", p, _gathered(s["v_cache"], s["v_scale"], at, cell, ok)) / torch.where(total == 0, 1.0, total)
    return {"o": o.reshape(b, heads, dim).to(q.dtype), "lse": (top + torch.log(total)).reshape(b, heads)}


def _plain_sample(s):
    x, u = s["logits"].float(), s["noise"]
    rows, vocab = x.shape
    t = s["temperature"][:, None]
    greedy = t <= 0
    top = x.amax(1, keepdim=True)
    y = (x - top) / torch.where(greedy, 1.0, t)
    w = torch.exp(y)
    keep = w > 0
    if s["top_k"] is not None:
        k = s["top_k"][:, None].long()
        k = torch.where((k <= 0) | (k > vocab), vocab, k)
        sorted_x, order = torch.sort(x, dim=1, descending=True, stable=True)
        ws = torch.where(torch.arange(vocab, device=x.device) < k, torch.gather(w, 1, order), 0.0)
        before = torch.cumsum(ws, 1) - ws
        # the shortest prefix that holds top_p of the mass: a token stays while what is before it holds less
        stay = (torch.arange(vocab, device=x.device) < k) & ((s["top_p"][:, None] >= 1) | (before < s["top_p"][:, None] * ws.sum(1, keepdim=True)))
        stay[:, 0] = True
        keep &= torch.zeros_like(keep).scatter_(1, order, stay) & (w >= s["min_p"][:, None])
    gumbel = -torch.log(-torch.log(u.clamp(2.0 ** -32, 1 - 2.0 ** -24)))
    race = torch.where(keep, y + gumbel, float("-inf"))
    tokens = torch.where(greedy[:, 0], torch.argmax(x, 1), torch.argmax(race, 1))
    logprobs = torch.gather(y, 1, tokens[:, None])[:, 0] - torch.log(w.sum(1))
    return {"tokens": tokens.to(torch.int32), "logprobs": torch.where(greedy[:, 0], 0.0, logprobs)}


PLAIN = {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}
OWN = {"tables": _own_tables, "append": _own_append, "attend": _own_attend, "sample": _own_sample}


# ---- what a pass cannot do without ----------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "tables":
        cached, new = _table_lengths(case)
        page, n = case["page"], case["requests"]
        old, need = [-(-c // page) for c in cached], [-(-(c + m) // page) for c, m in zip(cached, new)]
        tail = sum(case["max_pages"] - o for o in old)  # entries that are written: new ids, and -1 beyond them
        slots = n * case["new"]
        # a slot and a position for every token and for the padding; lengths, offsets; the ids of the pages taken; the
        # entry of a page that a request fills up
        return {"bytes": 8 * n + 4 * (sum(need) - sum(old)) + 4 * n + 4 * tail + 12 * slots + 4 * n + 4 * (n + 1) + 16, "flops": 0}
    if op == "append":
        n = case["tokens"]
        kept = n - (1 + n // 16 if n >= 16 else 0)
        values = 2 * kept * case["kv_heads"] * case["dim"]
        return {"bytes": values * (BYTES[case["type"]] + BYTES[case["cache"]]) + 8 * n, "flops": values if case["cache"] == "e4m3" else 0}
    if op == "attend":
        lengths = _lengths(case, case["longest"])
        read = [min(n, case["window"]) if case["window"] else n for n in lengths]
        page = case["page"]
        pages = sum(-(-n // page) - (n - m) // page for n, m in zip(lengths, read))
        q = 4 if case["cache"] == "f32" else 2
        b, heads, dim = case["requests"], case["q_heads"], case["dim"]
        return {"bytes": 2 * sum(read) * case["kv_heads"] * dim * BYTES[case["cache"]] + 2 * b * heads * dim * q + 4 * (pages + b + b * heads),
                "flops": 4 * sum(read) * heads * dim}
    # the noise of tokens that the filters remove need not be read; how many stay depends on the values, so only the
    # unfiltered case counts it
    values = case["rows"] * case["vocab"]
    return {"bytes": values * BYTES[case["type"]] + (4 * values if case["filters"] == "none" else 0) + 24 * case["rows"], "flops": 4 * values}


# ---- the definition, in 64 bits ----------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None  # whole numbers throughout
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s) if case["op"] == "attend" else _exact_sample(s)


def _exact_append(s):
    slots, page, got = s["slots"].cpu().numpy(), s["page"], {}
    real = slots >= 0
    for name in ("k", "v"):
        cache = s[name + "_cache"].double().cpu().numpy().copy()
        x = s[name].double().cpu().numpy()
        if s[name + "_scale"] is not None:
            x = x / s[name + "_scale"].double().cpu().numpy()[:, None]
            size = np.abs(x)
            # 3 bits after the leading one, no exponent below -6; numpy's rint takes ties to even
            step = np.exp2(np.floor(np.log2(np.maximum(size, 2.0 ** -6))) - 3)
            x = np.copysign(np.minimum(np.rint(size / step) * step, E4M3_MAX), x)
        cache[slots[real] // page, slots[real] % page] = x[real]
        got[name + "_cache"] = cache
    return got


def _exact_attend(s):
    """Request by request and KV head by KV head, with the base-2 exponential of shifted scores."""
    q, window, page = s["q"].double(), s["window"], s["k_cache"].shape[1]
    b, heads, dim = q.shape
    kv_heads = s["k_cache"].shape[2]
    group = heads // kv_heads
    o, lse = torch.zeros_like(q), torch.full((b, heads), float("-inf"), dtype=torch.float64, device=q.device)
    table, log2e = s["table"].long(), 1.0 / math.log(2.0)
    for r, n in enumerate(s["lengths"].tolist()):
        start = max(0, n - window) if window else 0
        if n == 0:
            continue
        j = torch.arange(start, n, device=q.device)
        page_of, cell = table[r, j // page], j % page
        for h in range(kv_heads):
            k, v = (c[page_of, cell, h].double() if f is None else c.view(torch.uint8)[page_of, cell, h].view(c.dtype).double() * f[h].double()
                    for c, f in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            mine = slice(h * group, (h + 1) * group)
            z = (k @ q[r, mine].T) * (log2e / math.sqrt(dim))
            top = z.max(0).values
            e = torch.exp2(z - top)
            total = e.sum(0)
            o[r, mine] = ((v.T @ e) / total).T
            lse[r, mine] = (top + torch.log2(total)) / log2e
    return {"o": o, "lse": lse}


def _exact_sample(s):
    logits, noise = s["logits"].double().cpu().numpy(), s["noise"].double().cpu().numpy()
    rows, vocab = logits.shape
    tokens, logprobs = np.zeros(rows, dtype=np.int32), np.zeros(rows)
    host = {k: None if s[k] is None else s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p")}
    for r in range(rows):
        x, t = logits[r], float(host["temperature"][r])
        if t <= 0:
            tokens[r] = np.argmax(x)
            continue
        w = np.exp((x - x.max()) / t)
        total = w.sum()
        kept = np.arange(vocab)
        if host["top_k"] is not None:
            k, p, least = int(host["top_k"][r]), float(host["top_p"][r]), float(host["min_p"][r])
            kept = np.lexsort((np.arange(vocab), -x))[: k if 0 < k <= vocab else vocab]
            if p < 1:
                mass = np.cumsum(w[kept])
                kept = kept[: 1 + int(np.searchsorted(mass, p * mass[-1], side="left"))]
            kept = kept[(w[kept] >= least)]
        kept = np.sort(kept[w[kept] > 0])
        # an exponential race: the first of clocks with rates w to ring
        clock = -np.log(np.clip(noise[r, kept], 2.0 ** -32, 1 - 2.0 ** -24)) / w[kept]
        tokens[r] = kept[np.argmin(clock)]
        logprobs[r] = math.log(w[tokens[r]] / total)
    return {"tokens": tokens, "logprobs": logprobs}
