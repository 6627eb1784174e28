"""The toy hybrid decoder of examples/hybrid_decode.py, prefill and decode through every operator, against the
same model token by token in 64 bits: the delta rule as a recurrence, attention over a plain list.

Each step of the reference takes the tokens that the example chose, so that its logits can be compared
step by step.  fp32: two layers of sums held to the library's 1e-5 each, then a product: 1e-4 of a row's norm.
bf16 and an 8-bit cache: every activation is rounded to 2^-9 about ten times on the way (cached values to 2^-4 of their
size each, averaged over a softmax): 5e-2.
"""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_delta_rule_16_gb300 import build
    build.build()


def reference(model, prompt, chosen):
    """Logits [steps, vocab] in 64 bits for a prompt continued by the chosen tokens."""
    w = {n: t.double() for n, t in vars(model).items()}
    nv, d, hd, group = 2 * model.nq, model.dim, model.head_dim, model.heads // model.kv_heads
    S, keys, values, logits = torch.zeros(nv, d, d, dtype=torch.float64, device=model.embed.device), [], [], []
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    for n, token in enumerate(prompt + chosen[:-1]):
        x = w["embed"][token]
        q, k = (unit((x @ w[m]).view(model.nq, d)).repeat_interleave(2, 0) for m in ("gq", "gk"))
        v, beta = (x @ w["gv"]).view(nv, d), torch.sigmoid(x @ w["gbeta"])
        keep = torch.exp2(-0.1 * torch.nn.functional.softplus(x @ w["ga"]))
        S = keep[:, None, None] * S
        S = S + k[:, :, None] * (beta[:, None] * (v - torch.einsum("hkv,hk->hv", S, k)))[:, None, :]
        x = x + (torch.einsum("hkv,hk->hv", S, q) / math.sqrt(d)).reshape(-1) @ w["go"]
        qkv = (x @ w["aqkv"]).view(-1, hd)
        q, k, v = qkv.split([model.heads, model.kv_heads, model.kv_heads])
        keys.append(k)
        values.append(v)
        K, V = (torch.stack(t).repeat_interleave(group, 1) for t in (keys, values))
        p = torch.softmax(torch.einsum("hd,nhd->hn", q, K) / math.sqrt(hd), 1)
        x = x + torch.einsum("hn,nhd->hd", p, V).reshape(-1) @ w["ao"]
        if n >= len(prompt) - 1:
            logits.append(x @ w["out"])
    return torch.stack(logits)


@pytest.mark.parametrize("cache,page,tol", [("f32", 16, 1e-4), ("f32", 7, 1e-4), ("bf16", 32, 5e-2), ("e4m3", 16, 5e-2)])
def test_example_matches_the_model(cache, page, tol):
    import hybrid_decode as ex
    model = ex.ToyHybrid(torch.float32 if cache == "f32" else torch.bfloat16)
    prompts = [[(11 * i + 5 * j) % model.vocab for j in range(n)] for i, n in enumerate((1, 16, 70, 31))]
    tokens, logits = ex.serve(model, prompts, 24, cache=cache, page=page)
    for b, prompt in enumerate(prompts):
        chosen = tokens[b].tolist()
        want = reference(model, prompt, chosen)
        err = (logits[b].double() - want).norm(dim=1) / want.norm(dim=1)
        assert err.max() <= tol, (b, err.max().item())
        assert chosen == logits[b].argmax(1).tolist()   # greedy: the largest of the logits that it was given


def test_example_samples_with_its_settings():
    import hybrid_decode as ex
    model = ex.ToyHybrid(torch.bfloat16)
    run = lambda seed: ex.serve(model, [[1, 2, 3], [4] * 40], 12, temperature=1.0, top_k=5, seed=seed)
    a, b, c = run(1), run(1), run(2)
    assert torch.equal(a[0], b[0]) and not torch.equal(a[0], c[0])
    rank = (a[1].float() > a[1].float().gather(2, a[0].long()[..., None])).sum(2)
    assert (rank < 5).all()
