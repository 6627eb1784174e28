"""Rows of logits that several CTAs share, of which some gather more of the likeliest tokens than their lists hold and others do not.
References and tolerances are those of test_gpu_prompt.py."""
import pytest
import torch

from test_gpu_prompt import TYPES, _built, check_logprobs, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,shares", [(1, 2), (1, 3), (1, 7), (3, 2), (3, 6), (50, 2), (50, 3), (100, 1), (1, 1), (300, 3)])
@pytest.mark.parametrize("rest", [1, 700, 1100, 1235, 1700, 2040, 2100])
def test_last_share_of_few_logits(kind, B, shares, rest):
    # a CTA whose threads do not all have a logit starts without a threshold, and gathers all it has
    V = shares * (8192 if kind == "bf16" else 4096) + rest
    for top in (1, 5, 32):
        for off in (0, 3):
            x = (torch.randn((B, V + 3), device=dev(), generator=gen(rest + off)) * 5).to(TYPES[kind])[:, off:][:, :V]
            check_logprobs(x, [i % V for i in range(B)], top)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B", [1, 3, 60])
@pytest.mark.parametrize("which", [[0], [2], [1, 3], [0, 1, 2, 3, 4, 5, 6], [7]])
def test_some_shares_rise(kind, B, which):
    # in the shares named every batch passes the one before; the others' logits lie among them
    batch, V = (8192 if kind == "bf16" else 4096), 300007
    i = torch.arange(V, device=dev())
    ctas = 4 if B == 60 else 8
    mine = torch.isin(i // batch % ctas, torch.tensor([w % ctas for w in which], device=dev()))
    x = torch.randn((B, V), device=dev(), generator=gen(B)) * 2
    x = torch.where(mine, i // batch * 0.5 + i % batch / batch * 0.5, x + i % 97 / 8)
    for top in (1, 7, 32):
        check_logprobs(x.to(TYPES[kind]), [j * 17 % V for j in range(B)], top)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_random_sizes(kind):
    r = torch.Generator().manual_seed(3 if kind == "bf16" else 4)
    pick = lambda *c: c[int(torch.randint(0, len(c), (1,), generator=r))]
    for k in range(150):
        B, top = pick(1, 2, 3, 20, 50), pick(1, 2, 5, 20, 32)
        V = int(torch.randint(32, 80000, (1,), generator=r))
        x = torch.randn((B, V), device=dev(), generator=gen(k)) * pick(0.1, 3.0, 20.0)
        check_logprobs(x.to(TYPES[kind]), [(j * 7919 + k) % (V + 1) - 1 for j in range(B)], top)
