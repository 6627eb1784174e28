"""The decode step over a paged cache at the edges of its inputs: masked rows of logits, bit patterns of NaN, weights far
below the largest, values near the type's largest, several host threads and streams,
outputs that overlap inputs, calls made again.

References and tolerances are those of test_gpu_paged.py.
"""
import math
import threading

import pytest
import torch

import gated_delta_rule_16_gb300 as gdn
from test_gpu_paged import ROW_TOL, TYPES, check_attend, check_sample, dev, i32, make, ref_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_delta_rule_16_gb300 import build
    build.build()
    gdn.load()


# ---- sampling: rows masked with the type's lowest value --------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 512, 1000, 2000, 100003])
def test_sample_top_k_of_rows_masked_with_the_lowest_value(kind, V):
    # log-probabilities of a few allowed tokens; the others finfo.min, -inf, or both: fewer allowed tokens than top_k asks for,
    # slices of the row without one, and threads that meet none that is finite
    lowest = float(torch.finfo(TYPES[kind]).min)
    g = torch.Generator(device=dev()).manual_seed(V)
    allowed = torch.tensor([-0.5, -0.75, -1.0, -1.5, -2.0], device=dev())
    x = torch.full((8, V), lowest, device=dev())
    at = torch.randperm(V, device=dev(), generator=g)
    x[1, ::2] = -math.inf
    x[2] = -math.inf
    x[3, V // 2:] = -math.inf
    x[4, : V // 3] = -math.inf
    x[5, torch.arange(V, device=dev()) % 1024 >= 28] = -math.inf   # whole threads without a finite token
    for r in range(6):
        x[r, at[:5]] = allowed
    x[5, :20] = -1.25
    x[6, 1::2] = -math.inf                           # nothing but the lowest value
    x[7, at[: V // 2]] = -3e38                       # a large negative level above the lowest
    x = x.to(TYPES[kind])
    drawn = set()
    for seed in range(6):
        u = torch.rand((8, V), device=dev(), generator=g)
        for k in (4, 10, 50, 600):
            tok, _ = check_sample(x, u, k=[k] * 8)
            drawn.add(int(tok[0]))
            check_sample(x, u, t=[0.7] * 8, k=[k] * 8, p=[0.8] * 8)
            check_sample(x, u, k=[k] * 8, m=[0.3] * 8)
    assert len(drawn) > 1                            # drawn, not the largest each time


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_sample_top_k_where_one_slice_of_the_row_has_few_tokens(kind):
    # 100003 tokens are shared by several CTAs; the k-th token lies in the slice with fewer than its share of the k
    V, k = 100003, 50
    x = torch.full((1, V), float(torch.finfo(TYPES[kind]).min), device=dev())
    x[0, :12000][torch.arange(12000, device=dev()) % 2048 >= 56] = -math.inf
    for s in range(1, 8):
        x[0, 12600 * s: 12600 * s + 7 * 300: 300] = -1.0 - 0.0625 * s
    x[0, 5] = -5.0
    x = x.to(TYPES[kind])
    u = torch.full((1, V), 0.25, device=dev())
    u[0, 5] = 1.0
    tok, _ = check_sample(x, u, k=[k])
    assert int(tok[0]) == 5


# ---- attention: NaN whatever its bits ---------------------------------------------------------------------
NAN_BITS = {"f32": [0x7FC00000, 0x7FFFFFFF, 0xFFFFFFFF, 0xFFC00000, 0x7F800001, 0xFFFFF000],
            "bf16": [0x7FC0, 0x7FFF, 0xFFFF, 0x7F81], "e4m3": [0x7F, 0xFF]}
WORDS = {1: torch.uint8, 2: torch.int16, 4: torch.int32}


def put(t, where, bits):
    size = t.element_size()
    bits -= 1 << 8 * size if size > 1 and bits >> (8 * size - 1) else 0
    t.view(WORDS[size])[where] = bits


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("d,group", [(64, 4), (128, 9), (256, 1)])
def test_attend_nan_of_any_bits_reaches_its_row_alone(kind, d, group):
    lens, page, heads = [40, 90, 2000, 17], 16, 2
    for bits in NAN_BITS[kind]:
        for token, b in ((0, 0), (89, 1), (1111, 2)):
            cell = lambda s: (int(s["block_table"][b, token // page]), token % page, 1, d - 3)
            mine = slice(group, 2 * group)
            for where in ("q", "k_cache", "v_cache"):
                s = make(kind, lens, heads, group, d, page, seed=d + group)
                if where == "q":
                    wide = bits if s["q"].element_size() == s["k_cache"].element_size() else 0x7FFF
                    put(s["q"], (b, group, 5), wide)
                else:
                    put(s[where], cell(s), bits)
                o, lse = gdn.gdn_paged_decode(**s)
                bad_o, bad_lse = torch.isnan(o), torch.isnan(lse)
                want_o, want_lse = torch.zeros_like(bad_o), torch.zeros_like(bad_lse)
                if where == "q":
                    want_o[b, group], want_lse[b, group] = True, True
                elif where == "k_cache":
                    want_o[b, mine], want_lse[b, mine] = True, True
                else:
                    want_o[b, mine, d - 3] = True
                assert torch.equal(bad_o, want_o) and torch.equal(bad_lse, want_lse), (hex(bits), token, where)
                assert torch.isfinite(o[~want_o]).all() and torch.isfinite(lse[~want_lse]).all()


# ---- several host threads -----------------------------------------------------------------------------------
def test_attend_from_two_threads_on_one_stream():
    # rows cut between CTAs, joined by a second launch: another thread's calls come in between
    cases = [make("bf16", [9000, 300, 4000], 2, 4, 128, 16, seed=21), make("e4m3", [20000, 1, 77, 5000, 12000], 4, 9, 128, 64, seed=22)]
    want = [gdn.gdn_paged_decode(**s) for s in cases]
    torch.cuda.synchronize()
    got, errors = [[], []], []
    meet = threading.Barrier(2)

    def run(i):
        try:
            meet.wait(30)
            for _ in range(200):
                got[i].append(gdn.gdn_paged_decode(**cases[i]))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in (0, 1):
        assert len(got[i]) == 200 and all(torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]) for o, lse in got[i])


# ---- attention: weights far below the largest ---------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("octaves", [10.0, 14.5, 20.3, 24.5, 25.0, 26.0, 30.0])
@pytest.mark.parametrize("tokens,rows", [(300, 1), (1 << 17, 1), (1 << 17, 700)])
def test_attend_a_long_tail_below_one_token(kind, octaves, tokens, rows):
    # One token's weight is 1, every other's 2^-octaves: what the tail holds together must not be lost.  With many rows each is
    # one CTA's, and a quarter of its tail one warp's.
    d, page, group = 64, 64, 4
    g = torch.Generator(device=dev()).manual_seed(3)
    q = torch.zeros((rows, group, d), device=dev())
    q[..., 0] = 1.0
    k, v = (torch.zeros((2, page, 1, d), device=dev()) for _ in range(2))
    k[0, 5, 0, 0] = 64.0                             # exact in every type
    v[0] = 0.25 * torch.randn((page, 1, d), device=dev(), generator=g)
    v[0, 5] = 0.5
    v[1] = 300.0
    table = torch.ones((1, tokens // page + 1), dtype=torch.int32, device=dev())
    table[0, 0] = 0                                  # the token's page once, the other one again and again
    scales = dict(zip(("k_scale", "v_scale"), torch.ones((2, 1), device=dev()) if kind == "e4m3" else (None, None)))
    scale = octaves * math.log(2.0) / 64.0
    # a warp adds tokens / 64 slices one after the other in fp32
    steps = tokens / 64 * 2.0 ** -23
    for order, n in ((table, tokens), (table.flip(1), table.shape[1] * page)):   # the token first, or in the row's last page
        s = dict(q=q.to(torch.float32 if kind == "f32" else torch.bfloat16), k_cache=k.to(TYPES[kind]), v_cache=v.to(TYPES[kind]),
                 block_table=order.contiguous().expand(rows, -1), seq_lens=i32([n] * rows), **scales)
        o, lse = gdn.gdn_paged_decode(**s, scale=scale)
        want_o, want_lse, off = ref_attend({**s, "q": s["q"][:1], "block_table": s["block_table"][:1], "seq_lens": s["seq_lens"][:1]}, scale=scale)
        err = (o.double() - want_o).norm(dim=-1) / want_o.norm(dim=-1)
        assert (err <= ROW_TOL[kind] + steps).all(), err.max().item()
        assert ((lse.double() - want_lse).abs() <= off + steps + 2.0 ** -20 * (1 + want_lse.abs())).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_attend_huge_values_of_tokens_without_weight(kind):
    # 3e38 at a weight of 2^-400 (0 in fp32) adds nothing
    s = make(kind, [100, 5000], 2, 4, 128, 16, seed=12)
    s["q"][...] = 0
    s["q"][..., 0] = 8.0
    s["k_cache"][..., 0] = 8.0
    huge = torch.finfo(TYPES[kind]).min / 2
    for b, token in ((0, 0), (0, 33), (0, 99), (1, 4000), (1, 3)):
        page, cell = int(s["block_table"][b, token // 16]), token % 16
        s["k_cache"][page, cell, :, 0] = -28.0
        s["v_cache"][page, cell, :, ::3] = huge
    check_attend(kind, s, scale=1.0)


def test_outputs_on_another_stream_are_not_what_pending_work_still_writes():
    s = make("bf16", [9000, 300, 4000], 2, 4, 128, 16, seed=23)
    x, u = (torch.rand((4, 50000), device=dev(), generator=torch.Generator(device=dev()).manual_seed(24)) for _ in range(2))
    top_k, new, free, table = i32([40] * 4), i32([5, 40]), i32(list(range(9))), torch.full((2, 4), -1, dtype=torch.int32, device=dev())
    calls = [lambda **kw: gdn.gdn_paged_decode(**s, **kw), lambda **kw: gdn.gdn_sample(x, u, top_k=top_k, **kw),
             lambda **kw: gdn.gdn_page_tables(new, free, table, page=16, n_slots=50, **kw)]
    side = torch.cuda.Stream()
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        # memory of every output's and the workspace's size that the current stream still writes after its owner is gone
        old = [torch.empty_like(t) for t in want for _ in range(3)] + [torch.empty(1 << 25, dtype=torch.uint8, device=dev())]
        torch.cuda._sleep(200_000_000)
        for t in old:
            t.fill_(3)
        del old, t
        got = call(stream=side)
        side.synchronize()
        first = [t.cpu() for t in got]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b.cpu()) and torch.equal(a, w.cpu()) for a, b, w in zip(first, got, want))


# ---- block tables -------------------------------------------------------------------------------------------
def test_tables_refuse_outputs_over_inputs():
    # all CTAs read the lengths and one writes the results: in place one would read what another has written
    lens, new, free = i32([5, 40, 3, 17]), i32([1, 1, 1, 1]), i32(list(range(12)))
    table = torch.full((4, 4), -1, dtype=torch.int32, device=dev())
    both = torch.zeros(9, dtype=torch.int32, device=dev())
    call = lambda **kw: gdn.gdn_page_tables(**{**dict(new_lens=new, free_pages=free, block_table=table, page=16, cached_lens=lens, n_slots=4), **kw})
    for kw in (dict(seq_lens=lens), dict(seq_lens=new), dict(cached_lens=both[:4], cu_new=both[3:8]), dict(positions=free[8:]),
               dict(counts=lens), dict(free_pages=table.view(-1))):
        with pytest.raises(gdn.GdnError):
            call(**kw)
    torch.cuda.synchronize()
    assert lens.tolist() == [5, 40, 3, 17] and (table == -1).all()
    got = call(cached_lens=both[:4], cu_new=both[4:])         # side by side
    assert got[0].tolist() == [0, 16, 32, 48] and both[4:].tolist() == [0, 1, 2, 3, 4]


# ---- sampling: what repeats ---------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_sample_repeats_bit_for_bit_and_across_batches_to_rounding(kind):
    g = torch.Generator(device=dev()).manual_seed(31)
    B, V = 40, 50001
    x = (torch.linspace(0.2, 6.0, B, device=dev())[:, None] * torch.randn((B, V), device=dev(), generator=g)).to(TYPES[kind])
    u = torch.rand((B, V), device=dev(), generator=g)
    f = lambda *v: torch.tensor([v[b % len(v)] for b in range(B)], device=dev())
    kw = dict(temperature=f(0.7, 1.0, 1.3), top_k=i32([[0, 40, 3000, 700][b % 4] for b in range(B)]), top_p=f(1.0, 0.5, 0.9, 0.95, 0.3),
              min_p=f(0.0, 0.02))
    want = gdn.gdn_sample(x, u, **kw)
    for _ in range(20):
        got = gdn.gdn_sample(x, u, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    big = gdn.gdn_sample(x.repeat(20, 1), u.repeat(20, 1), **{n: t.repeat(20) for n, t in kw.items()})   # fewer CTAs to a row
    assert torch.equal(big[0], want[0].repeat(20))       # no token of these rows is at an edge
    assert ((big[1] - want[1].repeat(20)).abs() <= 2.0 ** -20 * (1 + want[1].repeat(20).abs())).all()
