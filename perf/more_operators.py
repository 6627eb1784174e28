"""The operators of a prompt chunk through softmax-attention layers: what is measured, and their plain forms.

A hybrid decoder's softmax-attention layers take a prompt in chunks of new tokens.  Queries and keys are normalised per
head and rotated by their positions (`rope`), the chunk's queries attend to everything that the paged cache holds of
their request up to themselves (`attend`), and a scored prompt's logits become log probabilities of its own tokens, with
the distribution's entropy and the likeliest alternatives (`score`).
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
        # one new token of each running request, far into their contexts: pure latency, once per layer and step
        {"name": "rope_step", "op": "rope", "tokens": 64, "q_heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128, "interleaved": False, "norm": True,
         "longest": 131072, "factor": 4.0, "type": "bf16"},
        # a long prompt's queries and keys, slices of one projection
        {"name": "rope_prompt", "op": "rope", "tokens": 16411, "q_heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128, "interleaved": False,
         "norm": True, "longest": 16411, "factor": 1.0, "type": "bf16"},
        # a quarter of each head is rotated, in neighbouring pairs, without a norm; 32-bit storage of a parity run
        {"name": "rope_partial_f32", "op": "rope", "tokens": 2001, "q_heads": 16, "kv_heads": 2, "dim": 256, "rotary": 64, "interleaved": True,
         "norm": False, "longest": 1000003, "factor": 1.0, "type": "f32"},
        # the first prompt of a chat: a few rows, latency
        {"name": "attend_first", "op": "attend", "requests": 1, "new": 37, "cached": 0, "mix": "full", "pad": False, "q_heads": 16, "kv_heads": 2,
         "dim": 128, "page": 16, "cache": "bf16", "head_major": False, "window": 0},
        # one prompt prefilled at once
        {"name": "attend_prompt", "op": "attend", "requests": 1, "new": 8192, "cached": 0, "mix": "full", "pad": False, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "cache": "bf16", "head_major": False, "window": 0},
        # the last chunk of a very long document: few rows against a long cache
        {"name": "attend_chunk", "op": "attend", "requests": 1, "new": 2048, "cached": 129024, "mix": "full", "pad": False, "q_heads": 16,
         "kv_heads": 4, "dim": 128, "page": 64, "cache": "bf16", "head_major": True, "window": 0},
        # a server's mixed step: most requests add one token, some a piece of a prompt; padded rows behind the last
        {"name": "attend_mixed", "op": "attend", "requests": 32, "new": 384, "cached": 4096, "mix": "steps", "pad": True, "q_heads": 16,
         "kv_heads": 4, "dim": 128, "page": 16, "cache": "bf16", "head_major": False, "window": 0},
        # chunks over long contexts in an 8-bit cache
        {"name": "attend_e4m3", "op": "attend", "requests": 8, "new": 512, "cached": 16000, "mix": "ragged", "pad": False, "q_heads": 32,
         "kv_heads": 4, "dim": 128, "page": 64, "cache": "e4m3", "head_major": True, "window": 0},
        # wide heads with a sliding window
        {"name": "attend_window", "op": "attend", "requests": 4, "new": 2048, "cached": 6000, "mix": "ragged", "pad": False, "q_heads": 16,
         "kv_heads": 2, "dim": 256, "page": 32, "cache": "bf16", "head_major": False, "window": 4096},
        # 32-bit storage, pages that are no power of two
        {"name": "attend_f32", "op": "attend", "requests": 3, "new": 1031, "cached": 1000, "mix": "ragged", "pad": False, "q_heads": 12,
         "kv_heads": 4, "dim": 64, "page": 48, "cache": "f32", "head_major": False, "window": 0},
        # log probabilities of the sampled tokens of a small batch, with the usual five alternatives
        {"name": "score_step", "op": "score", "rows": 4, "vocab": 131072, "type": "bf16", "top": 5},
        # a whole prompt scored against its own next tokens
        {"name": "score_prompt", "op": "score", "rows": 2047, "vocab": 100003, "type": "f32", "top": 20},
    ]


def _log(rng, low, high):
    """A whole number in [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "attend", "score"])
    if op == "rope":
        dim, heads = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 5, 8])
        group, kind = rng.choice([1, 2, 4, 5, 8]), rng.choice(["bf16", "bf16", "f32"])
        tokens = _log(rng, 1, 16411 * 40 * 128 // (heads * (group + 1) * dim * (2 if kind == "f32" else 1)))
        return {"op": op, "tokens": tokens, "q_heads": heads * group, "kv_heads": heads, "dim": dim,
                "rotary": rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)]), "interleaved": rng.random() < 0.5,
                "norm": rng.random() < 0.6, "longest": max(tokens, _log(rng, 1, 1000003)), "factor": rng.choice([1.0, 1.0, 4.0, 32.0]), "type": kind}
    if op == "attend":
        cache, dim = rng.choice(["bf16", "bf16", "e4m3", "f32"]), rng.choice([64, 128, 128, 256])
        heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        requests = _log(rng, 1, 64)
        # scores, were every request as large as the largest: a plain form has them all in memory
        most = (60_000_000 if cache == "f32" else 800_000_000) // (requests * heads * group)
        new = _log(rng, 1, min(8192, math.isqrt(most) // 2))
        longest = max(new, min(131072, most // new, 100_000_000 // (requests * heads * dim)))
        cached = rng.choice([0, _log(rng, 1, max(1, longest - new))])
        return {"op": op, "requests": requests, "new": new, "cached": cached, "mix": rng.choice(["full", "ragged", "ragged", "steps"]),
                "pad": rng.random() < 0.3, "q_heads": heads * group, "kv_heads": heads, "dim": dim, "page": rng.choice([1, 16, 24, 32, 64, 128]),
                "cache": cache, "head_major": rng.random() < 0.5, "window": rng.choice([0, 0, _log(rng, 1, new + cached)])}
    vocab = _log(rng, 1000, 160000)
    return {"op": op, "rows": _log(rng, 1, min(2047, 2047 * 100003 // vocab)), "vocab": vocab, "type": rng.choice(["bf16", "f32"]),
            "top": rng.choice([0, 1, 5, 20, 32])}


def _lengths(case):
    """(new, cached) tokens of the requests: the case's own, whatever the seed."""
    n, new, cached = case["requests"], case["new"], case["cached"]
    if case["mix"] == "full":
        return [new] * n, [cached] * n
    r = random.Random(n * 1000003 + new * 101 + cached)
    have = [r.randint(0, cached) for _ in range(n)]
    add = [1 if case["mix"] == "steps" and i % 8 else r.randint(1, new) for i in range(n)]
    at = r.randrange(n)
    add[at], have[at] = new, cached
    if n >= 4:
        add[(at + 1) % n] = 0  # a request that waits in this step
    if n >= 8:
        have[(at + 2) % n] = 0
    return add, have


# ---- what a program has in hand --------------------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    return {"rope": _prepare_rope, "attend": _prepare_attend, "score": _prepare_score}[case["op"]](case, dev, gen)


def _frequencies(case):
    """Radians per token of each pair, in 64 bits: a base of 10000, stretched for long contexts by its factor."""
    r = case["rotary"]
    base = 10000.0 * case["factor"] ** (r / (r - 2) if r > 2 else 1.0)
    return base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)


def _prepare_rope(case, dev, gen):
    n, hq, hk, dim = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    # slices of one projection's output, as a layer makes them
    qkv = torch.randn((n, hq + 2 * hk, dim), device=dev, generator=gen).mul_(3.0).to(TYPES[case["type"]])
    if n == case["longest"]:
        positions = torch.arange(n, device=dev, dtype=torch.int32)
    else:
        positions = torch.randint(0, case["longest"], (n,), device=dev, generator=gen, dtype=torch.int32)
    weight = [0.5 + torch.rand(dim, device=dev, generator=gen) if case["norm"] else None for _ in range(2)]
    return {"op": "rope", "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "positions": positions, "freqs": _frequencies(case).to(dev), "q_weight": weight[0],
            "k_weight": weight[1], "eps": 1e-6, "interleaved": case["interleaved"], "mscale": 0.1 * math.log(case["factor"]) + 1.0}


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


def _prepare_attend(case, dev, gen):
    page, b = case["page"], case["requests"]
    new, cached = _lengths(case)
    lengths = [n + c for n, c in zip(new, cached)]
    wide = max(1, -(-max(lengths) // page))
    need = torch.tensor([-(-n // page) for n in lengths], device=dev)
    pages = int(need.sum()) + 3
    k_cache, v_cache, k_scale, v_scale = _cache(case, pages, dev, gen)
    ids = torch.randperm(pages, device=dev, generator=gen).to(torch.int32)
    held = torch.arange(wide, device=dev) < need[:, None]
    at = torch.cumsum(need, 0)[:, None] - need[:, None] + torch.arange(wide, device=dev)
    table = torch.where(held, ids[torch.where(held, at, 0)], -1).to(torch.int32)
    kind = torch.float32 if case["cache"] == "f32" else torch.bfloat16
    rows = sum(new) + (13 if case["pad"] else 0)
    q = (2.0 * torch.randn((rows, case["q_heads"], case["dim"]), device=dev, generator=gen)).to(kind)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    # a captured step's outputs have rows behind the last request, which stay as they are
    out = {"o": torch.zeros_like(q), "lse": torch.zeros(q.shape[:2], device=dev)} if case["pad"] else {"o": None, "lse": None}
    return {"op": "attend", "q": q, "k_cache": k_cache, "v_cache": v_cache, "table": table, "seq_lens": i32(lengths), "cu_new": i32(cu), "k_scale": k_scale,
            "v_scale": v_scale, "window": case["window"], "most_new": max(new), **out}


def _prepare_score(case, dev, gen):
    rows, vocab = case["rows"], case["vocab"]
    logits = torch.randn((rows, vocab), device=dev, generator=gen).mul_(2.5)
    # a few tokens stand out, as they do after a trained model's last layer, and the given token is often one of them
    peak = torch.randint(0, vocab // 8, (rows, 8), device=dev, generator=gen) + vocab // 8 * torch.arange(8, device=dev)
    logits.scatter_add_(1, peak, 12.0 * torch.rand((rows, 8), device=dev, generator=gen))
    logits.scatter_(1, torch.randint(0, vocab, (rows, 5), device=dev, generator=gen), float("-inf"))
    other = torch.randint(0, vocab, (rows,), device=dev, generator=gen)
    tokens = torch.where(torch.rand(rows, device=dev, generator=gen) < 0.7, peak[:, 0], other).to(torch.int32)
    if rows >= 16:
        tokens[-1] = -1  # nothing follows a prompt's last token
    return {"op": "score", "logits": logits.to(TYPES[case["type"]]), "tokens": tokens, "top": case["top"]}


# ---- one pass ----------------------------------------------------------------------------------------------------------
def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


def _own_rope(s):
    import gated_delta_rule_16_gb300 as gdn
    q, k = gdn.gdn_qk_rope(s["q"], s["k"], s["positions"], s["freqs"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                           interleaved=s["interleaved"], mscale=s["mscale"])
    return {"q": q, "k": k}


def _own_attend(s):
    import gated_delta_rule_16_gb300 as gdn
    o, lse = gdn.gdn_paged_prefill(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["cu_new"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"], window=s["window"], o=s["o"], lse=s["lse"])
    return {"o": o, "lse": lse}


def _own_score(s):
    import gated_delta_rule_16_gb300 as gdn
    logprobs, entropy, top_tokens, top_logprobs = gdn.gdn_logprobs(s["logits"], s["tokens"], top=s["top"])
    return {"logprobs": logprobs, "entropy": entropy, "top_tokens": top_tokens, "top_logprobs": top_logprobs}


def _rotated(x, weight, cos, sin, s):
    y, r = x.float(), 2 * s["freqs"].numel()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * weight
    turn, rest = y[..., :r], y[..., r:]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if s["interleaved"] else (turn[..., :r // 2], turn[..., r // 2:])
    c, d = a * cos - b * sin, a * sin + b * cos
    turn = torch.stack((c, d), -1).flatten(-2) if s["interleaved"] else torch.cat((c, d), -1)
    return torch.cat((turn, rest), -1).to(x.dtype)


def _plain_rope(s):
    # angles in 64 bits: a far position's has lost its fraction of a turn in 32
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = ((s["mscale"] * f(angle)).float()[:, None] for f in (torch.cos, torch.sin))
    return {"q": _rotated(s["q"], s["q_weight"], cos, sin, s), "k": _rotated(s["k"], s["k_weight"], cos, sin, s)}


def _gathered(cache, scale, at, cell, ok):
    """The cached rows of every request, in 32 bits [requests, longest, kv_heads, dim]; zero where there is none."""
    x = (cache.view(torch.uint8)[at, cell].view(cache.dtype) if scale is not None else cache[at, cell]).float()
    if scale is not None:
        x.mul_(scale[:, None])
    return x.masked_fill_(~ok[:, :, None, None], 0.0)


def _plain_attend(s):
    q, table, lengths, cu, window, page = s["q"], s["table"], s["seq_lens"].long(), s["cu_new"].long(), s["window"], s["k_cache"].shape[1]
    n, heads, dim = q.shape
    kv_heads, b, wide = s["k_cache"].shape[2], table.shape[0], table.shape[1]
    o = torch.empty_like(q) if s["o"] is None else s["o"]
    lse = torch.empty((n, heads), device=q.device) if s["lse"] is None else s["lse"]
    # every request's new tokens, padded to the largest request's
    i = torch.arange(s["most_new"], device=q.device)
    row = cu[:-1, None] + i
    real = row < cu[1:, None]
    pos = lengths[:, None] - cu[1:, None] + row
    x = q[row.clamp(max=n - 1)].float().view(b, -1, kv_heads, heads // kv_heads, dim) * dim ** -0.5
    j = torch.arange(wide * page, device=q.device)
    at = table.long()[:, j // page]
    ok = (j < lengths[:, None]) & (at >= 0)
    at, cell = at.clamp(min=0), j % page
    score = torch.einsum("bnhgd,blhd->bhgnl", x, _gathered(s["k_cache"], s["k_scale"], at, cell, ok))
    seen = ok[:, None, :] & (j <= pos[:, :, None])
    if window:
        seen &= j > pos[:, :, None] - window
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    got = torch.einsum("bhgnl,blhd->bhgnd", p, _gathered(s["v_cache"], s["v_scale"], at, cell, ok)) / torch.where(total == 0, 1.0, total)
    # a padded row writes once more what the first real row writes: no row count leaves the GPU
    real, row = real.flatten(), row.flatten()
    src = torch.where(real, torch.arange(real.numel(), device=q.device), torch.argmax(real.to(torch.int32)))
    o[row[src]] = got.permute(0, 3, 1, 2, 4).reshape(-1, heads, dim)[src].to(q.dtype)
    lse[row[src]] = (top + torch.log(total)).permute(0, 3, 1, 2, 4).reshape(-1, heads)[src]
    return {"o": o, "lse": lse}


def _plain_score(s):
    x, tokens, top = s["logits"].float(), s["tokens"].long(), s["top"]
    rows, vocab = x.shape
    most = x.amax(1, keepdim=True)
    y = x - most
    w = torch.exp(y)
    log_z = torch.log(w.sum(1, keepdim=True))
    entropy = log_z[:, 0] - (w * y.clamp(min=-200.0)).sum(1) / w.sum(1)
    real = (tokens >= 0) & (tokens < vocab)
    logprobs = torch.where(real, (torch.gather(y, 1, tokens.clamp(0, vocab - 1)[:, None]) - log_z)[:, 0], 0.0)
    # a whole number that orders logits, and equal ones by their index, lowest first
    bits = x.view(torch.int32).long()
    key = (torch.where(bits < 0, -(bits & 0x7fffffff), bits) << 32) + (vocab - 1 - torch.arange(vocab, device=x.device))
    ids = vocab - 1 - (torch.topk(key, top, dim=1).values & 0xffffffff)
    return {"logprobs": logprobs, "entropy": entropy, "top_tokens": ids.to(torch.int32), "top_logprobs": torch.gather(y, 1, ids) - log_z}


PLAIN = {"rope": _plain_rope, "attend": _plain_attend, "score": _plain_score}
OWN = {"rope": _own_rope, "attend": _own_attend, "score": _own_score}


# ---- what a pass cannot do without ----------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "rope":
        n, heads, dim = case["tokens"], case["q_heads"] + case["kv_heads"], case["dim"]
        return {"bytes": 2 * n * heads * dim * BYTES[case["type"]] + 4 * n + 4 * case["rotary"] + (8 * dim if case["norm"] else 0),
                "flops": n * heads * (3 * case["rotary"] + (4 * dim if case["norm"] else 0))}
    if op == "attend":
        new, cached = _lengths(case)
        window, page, heads, dim = case["window"], case["page"], case["q_heads"], case["dim"]
        keys = pages = pairs = 0
        for n, c in zip(new, cached):
            if n:
                first = max(0, c - window + 1) if window else 0
                keys += c + n - first
                pages += -(-(c + n) // page) - first // page
                whole = n if not window else min(n, max(0, window - c))  # tokens that see all before them
                pairs += whole * c + whole * (whole + 1) // 2 + (n - whole) * window
        rows, q = sum(new), 4 if case["cache"] == "f32" else 2
        return {"bytes": 2 * keys * case["kv_heads"] * dim * BYTES[case["cache"]] + 2 * rows * heads * dim * q + 4 * (pages + 2 * len(new) + 1 + rows * heads),
                "flops": 4 * pairs * heads * dim}
    values = case["rows"] * case["vocab"]
    return {"bytes": values * BYTES[case["type"]] + case["rows"] * (12 + 8 * case["top"]), "flops": 5 * values}


# ---- the definition, in 64 bits ----------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attend": _exact_attend, "score": _exact_score}[case["op"]](s)


def _exact_rope(s):
    """Pairs as complex numbers, turned by a product."""
    turn = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device=s["q"].device).expand(s["positions"].numel(), s["freqs"].numel()).contiguous(),
                       torch.outer(s["positions"].double(), s["freqs"]))[:, None]
    got = {}
    for name in ("q", "k"):
        x, half = s[name].double(), s["freqs"].numel()
        if s[name + "_weight"] is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * s[name + "_weight"].double()
        x = x.clone(memory_format=torch.contiguous_format)
        pairs = x[..., :2 * half].unflatten(-1, (half, 2) if s["interleaved"] else (2, half))
        if not s["interleaved"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * turn)
        x[..., :2 * half] = (z if s["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        got[name] = x
    return got


def _exact_attend(s):
    """Request by request, KV head by KV head and some tokens at a time, with the base-2 exponential of shifted scores."""
    q, window, page = s["q"], s["window"], s["k_cache"].shape[1]
    n, heads, dim = q.shape
    kv_heads = s["k_cache"].shape[2]
    group, log2e = heads // kv_heads, 1.0 / math.log(2.0)
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros((n, heads), dtype=torch.float64, device=q.device)
    table, cu, lengths = s["table"].long(), s["cu_new"].tolist(), s["seq_lens"].tolist()
    for b, length in enumerate(lengths):
        j = torch.arange(length, device=q.device)
        page_of, cell = table[b, j // page], j % page
        for h in range(kv_heads if cu[b + 1] > cu[b] else 0):
            k, v = (c[page_of, cell, h].double() if f is None else c.view(torch.uint8)[page_of, cell, h].view(c.dtype).double() * f[h].double()
                    for c, f in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            mine, step = slice(h * group, (h + 1) * group), max(1, 200_000_000 // (group * length))
            for t in range(cu[b], cu[b + 1], step):
                rows = torch.arange(t, min(t + step, cu[b + 1]), device=q.device)
                pos = rows - cu[b + 1] + length
                # keys before `first` are outside the window of all of these tokens, keys from `last` on behind them
                first, last = max(0, int(pos[0]) - window + 1) if window else 0, int(pos[-1]) + 1
                z = (q[rows, mine].double().reshape(-1, dim) @ k[first:last].T) * (log2e / math.sqrt(dim))
                behind = pos.repeat_interleave(group)[:, None] - j[first:last]
                z.masked_fill_((behind < 0) | (behind >= window) if window else behind < 0, float("-inf"))
                most = z.amax(1, keepdim=True)
                e = torch.exp2(z.sub_(most))
                total = e.sum(1, keepdim=True)
                o[rows, mine] = ((e @ v[first:last]) / total).view(-1, group, dim)
                lse[rows, mine] = ((most + torch.log2(total)) / log2e).view(-1, group)
    return {"o": o, "lse": lse}


def _exact_score(s):
    rows, vocab = s["logits"].shape
    got = {"logprobs": np.zeros(rows), "entropy": np.zeros(rows), "top_tokens": np.zeros((rows, s["top"]), dtype=np.int32), "top_logprobs": np.zeros((rows, s["top"]))}
    tokens = s["tokens"].tolist()
    for r in range(rows):
        x = s["logits"][r].double().cpu().numpy()
        p = np.exp(x - x.max())
        total = p.sum()
        logp = x - (x.max() + math.log(total))
        p /= total
        live = p > 0
        got["entropy"][r] = -np.sum(p[live] * logp[live])
        got["logprobs"][r] = logp[tokens[r]] if 0 <= tokens[r] < vocab else 0.0
        if s["top"]:
            near = np.flatnonzero(x >= np.partition(x, vocab - s["top"])[vocab - s["top"]])
            best = near[np.lexsort((near, -x[near]))][:s["top"]]
            got["top_tokens"][r], got["top_logprobs"][r] = best, logp[best]
    return got
