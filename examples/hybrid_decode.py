"""A toy hybrid decoder served from end to end: one gated delta layer, one softmax-attention layer over a paged cache.

    python examples/hybrid_decode.py [--steps N] [--cache bf16|f32|e4m3] [--temperature T]

Prompts of different lengths are prefilled (gdn_prefill_dense per request; the attention layer writes all prompts' keys
and values with one gdn_kv_append and attends all prompts' tokens with one gdn_paged_prefill), then
every step adds one token to each request: gdn_page_tables, gdn_decode_step, gdn_kv_append, gdn_paged_decode and
gdn_sample.  Weights are random; projections are plain matrix products.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_16_gb300 as gdn  # noqa: E402

CHUNK = 64  # tokens over which a prefill's gates accumulate


class ToyHybrid:
    """Weights and sizes: hidden 256; gated delta layer of 2 query/key heads (4 value heads) of 128; attention of 8 query
    and 2 KV heads of 64; vocabulary 1000."""

    hidden, nq, dim, heads, kv_heads, head_dim, vocab = 256, 2, 128, 8, 2, 64, 1000

    def __init__(self, dtype, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *shape: (torch.randn(shape, device=device, generator=g) / shape[0] ** 0.5).to(dtype)
        h, nv = self.hidden, 2 * self.nq
        self.embed = torch.randn((self.vocab, h), device=device, generator=g).to(dtype)
        self.gq, self.gk, self.gv = rand(h, self.nq * self.dim), rand(h, self.nq * self.dim), rand(h, nv * self.dim)
        self.gbeta, self.ga, self.go = rand(h, nv), rand(h, nv), rand(nv * self.dim, h)
        self.aqkv = rand(h, (self.heads + 2 * self.kv_heads) * self.head_dim)
        self.ao, self.out = rand(self.heads * self.head_dim, h), rand(h, self.vocab)

    def delta_inputs(self, x):
        """q, k [n, Nq, 128] of unit length, v [n, Nv, 128], beta and the tokens' log2 retention [n, Nv] fp32."""
        unit = lambda t: torch.nn.functional.normalize(t.float().view(-1, self.nq, self.dim), dim=-1).to(x.dtype)
        return (unit(x @ self.gq), unit(x @ self.gk), (x @ self.gv).view(-1, 2 * self.nq, self.dim),
                torch.sigmoid((x @ self.gbeta).float()), -0.1 * torch.nn.functional.softplus((x @ self.ga).float()))

    def attention_inputs(self, x):
        """q [n, heads, 64], k and v [n, kv_heads, 64]: slices of one product."""
        qkv = (x @ self.aqkv).view(-1, self.heads + 2 * self.kv_heads, self.head_dim)
        return qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def add_delta(self, x, o):
        return x + o.reshape(len(x), -1) @ self.go

    def add_attention(self, x, o):
        return x + o.reshape(len(x), -1) @ self.ao


def serve(model, prompts, steps, cache="bf16", page=16, temperature=0.0, top_k=50, top_p=0.95, seed=0):
    """Generates `steps` tokens for each prompt (lists of token ids).  Returns (tokens [B, steps], logits [B, steps, vocab])."""
    dev, dtype = model.embed.device, model.embed.dtype
    B, lens = len(prompts), [len(p) for p in prompts]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    max_pages = -(-(max(lens) + steps) // page)
    pages = sum(-(-(n + steps) // page) for n in lens)
    kind = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[cache]
    k_cache, v_cache = (torch.zeros((pages, page, model.kv_heads, model.head_dim), dtype=kind, device=dev) for _ in range(2))
    # an 8-bit cache stores x / scale: here values of up to 8 are kept
    scales = {} if cache != "e4m3" else {n: torch.full((model.kv_heads,), 8.0 / 448.0, device=dev) for n in ("k_scale", "v_scale")}
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    free = torch.arange(pages, dtype=torch.int32, device=dev)
    settings = dict(temperature=torch.full((B,), temperature, device=dev), top_k=torch.full((B,), top_k, dtype=torch.int32, device=dev),
                    top_p=torch.full((B,), top_p, device=dev))
    noise = torch.Generator(device=dev).manual_seed(seed)

    # ---- prompts: all requests' tokens in one list
    x = model.embed[torch.tensor([t for p in prompts for t in p], device=dev)]
    slots, _, seq_lens, cu_new, counts = gdn.gdn_page_tables(i32(lens), free, table, page=page, n_slots=sum(lens))
    q, k, v, beta, a = model.delta_inputs(x)
    states, outs, at = [], [], 0
    for n in lens:
        one = slice(at, at + n)
        gate = torch.cat([c.cumsum(0) for c in a[one].split(CHUNK)])  # log2 retention, accumulated inside each chunk
        o, s = gdn.gdn_prefill_dense(*(t[one][None].contiguous() for t in (q, k, v, beta)), gate[None])
        outs.append(o[0])
        states.append(s)
        at += n
    state = torch.cat(states)
    x = model.add_delta(x, torch.cat(outs))
    q, k, v = model.attention_inputs(x)
    gdn.gdn_kv_append(k, v, slots, k_cache, v_cache, **scales)
    o, _ = gdn.gdn_paged_prefill(q, k_cache, v_cache, table, seq_lens, cu_new, **scales)
    x = model.add_attention(x, o)
    x = x[torch.tensor(lens, device=dev).cumsum(0) - 1]

    tokens, logits = [], []
    ones = torch.ones(B, dtype=torch.int32, device=dev)
    taken = sum(-(-n // page) for n in lens)  # the host knows the lengths: no page count is read back
    for step in range(steps):
        y = x @ model.out
        u = torch.rand(y.shape, device=dev, generator=noise)
        token, _ = gdn.gdn_sample(y, u, **settings)
        tokens.append(token)
        logits.append(y)
        if step == steps - 1:
            break
        x = model.embed[token]
        slots, _, seq_lens, _, counts = gdn.gdn_page_tables(ones, free[taken:], table, page=page, cached_lens=seq_lens, n_slots=B)
        taken += sum((n + step) % page == 0 for n in lens)
        x = model.add_delta(x, gdn.gdn_decode_step(*(t.contiguous() for t in model.delta_inputs(x)), state))
        q, k, v = model.attention_inputs(x)
        gdn.gdn_kv_append(k, v, slots, k_cache, v_cache, **scales)
        o, _ = gdn.gdn_paged_decode(q, k_cache, v_cache, table, seq_lens, **scales)
        x = model.add_attention(x, o)
    if gdn.gdn_page_tables_status(counts):
        raise RuntimeError("the page pool was too small")
    return torch.stack(tokens, 1), torch.stack(logits, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--cache", choices=("bf16", "f32", "e4m3"), default="bf16")
    ap.add_argument("--temperature", type=float, default=0.8)
    args = ap.parse_args()
    model = ToyHybrid(torch.float32 if args.cache == "f32" else torch.bfloat16)
    prompts = [[(7 * i + 3 * j) % model.vocab for j in range(n)] for i, n in enumerate((5, 100, 33, 64))]
    tokens, _ = serve(model, prompts, args.steps, cache=args.cache, temperature=args.temperature)
    for n, row in zip(map(len, prompts), tokens.tolist()):
        print(f"prompt of {n:3d}: {row}")


if __name__ == "__main__":
    main()
