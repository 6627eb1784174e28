"""The prompt chunk's operators at their edges: concurrent calls, layouts that TMA cannot describe, long lists of requests, rows
that are masked almost everywhere.  References and tolerances are those of test_gpu_prompt.py."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import gated_delta_rule_16_gb300 as gdn
from test_gpu_prompt import INF, KINDS, NAN, TYPES, Case, _built, check_logprobs, check_rope, dev, gen, i32, same  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
def test_attend_calls_at_the_same_time(kind):
    cases = [Case([(900, 70), (0, 300)], kind=kind, d=d, seed=d, heads=4, kv_heads=2) for d in (64, 128, 256)]
    ws, streams = [gdn.Workspace() for _ in cases], [torch.cuda.Stream() for _ in cases]
    want = [c.call() for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [c.call(workspace=w, stream=s) for c, w, s in zip(cases, ws, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attend_beside_a_delta_prefill():
    # both take tensor memory of the same SMs
    c = Case([(2000, 300)], heads=8, kv_heads=2)
    want, want_lse = c.call()
    g = gen(0)
    q, k = (torch.nn.functional.normalize(torch.randn((1, 2048, 4, 128), device=dev(), generator=g), dim=-1).bfloat16() for _ in range(2))
    v = torch.randn((1, 2048, 8, 128), device=dev(), generator=g).bfloat16()
    beta, gate = torch.rand((1, 2048, 8), device=dev(), generator=g), -torch.rand((1, 2048, 8), device=dev(), generator=g).view(1, 32, 64, 8).cumsum(2).view(1, 2048, 8) / 64
    o0, _ = gdn.gdn_prefill_dense(q, k, v, beta, gate)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(10):
        got, got_lse = c.call(stream=s)
        o, _ = gdn.gdn_prefill_dense(q, k, v, beta, gate)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse) and torch.equal(o, o0)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_cache_of_one_head_for_all(kind):
    # stride 0 between KV heads, which a TMA map does not take
    c = Case([(300, 50), (17, 1)], kind=kind, heads=4, kv_heads=1, page=16)
    heads = Case([(300, 50), (17, 1)], kind=kind, heads=8, kv_heads=2, page=16)
    heads.k, heads.v = c.k.expand(-1, -1, 2, -1), c.v.expand(-1, -1, 2, -1)
    heads.table, heads.lens = c.table, c.lens
    if heads.scales:
        heads.scales = {n: t.expand(2).contiguous() for n, t in c.scales.items()}
    heads.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 4, 8, 40])
def test_attend_page_sizes_on_both_sides_of_a_tma_box(kind, page):
    Case([(250, 90), (64, 64), (0, 1), (63, 2)], kind=kind, page=page, d=128).check()
    Case([(250, 90), (64, 64), (0, 1), (63, 2)], kind=kind, page=page, d=256, window=100).check()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_one_tile_requests_in_a_row(kind):
    # a CTA goes through many units of one tile, each with its own queries
    for d in (64, 128, 256):
        Case([(i % 50, 1 + i % 7) for i in range(3000)], kind=kind, d=d, page=64 if d < 256 else 16, heads=2, kv_heads=2).check()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_units_of_one_and_two_row_tiles_in_a_row(kind):
    Case([(200, 1 if i % 2 else 130) for i in range(60)], kind=kind, heads=4, kv_heads=2, page=32).check()
    Case([(40 * i, 33 + i) for i in range(40)], kind=kind, heads=16, kv_heads=4, d=64, page=32).check()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_non_finite_everywhere_but_where_it_is_read(kind):
    # stale cells of live pages hold NaN and infinity of every sign; requests end inside tiles and pages
    c = Case([(100, 29), (0, 65), (191, 2), (0, 130)], kind=kind, page=64, heads=4, kv_heads=2)
    want, want_lse, far, lse_far = c.ref()
    for x in (c.k, c.v):
        raw = x.view(torch.uint8)
        stale = (raw == 0xFF).all(-1)
        for n, bits in enumerate(([0x7F, 0xFF] if kind == "e4m3" else [INF, -INF, NAN])):
            pick = stale & (torch.rand(stale.shape, device=dev(), generator=gen(n)) < 0.4)
            if kind == "e4m3":
                raw[pick] = bits
            else:
                x[pick] = bits
    o, lse = c.call()
    same(o.double(), want, far)
    same(lse.double(), want_lse, lse_far)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 256])
def test_attend_all_values_non_finite(kind, d):
    # every tile with a mask has what a masked weight must not meet: all of them take the slow way, and rows still end where they should
    c = Case([(0, 200)], kind=kind, d=d, heads=2, kv_heads=1, page=16)
    v = c.v.view(torch.uint8) if kind == "e4m3" else c.v
    for j in range(1, 200):
        v[int(c.table[0, j // 16]), j % 16, 0, j % d] = 0x7F if kind == "e4m3" else NAN
    o, lse = c.call()
    t, col = torch.arange(200, device=dev())[:, None], torch.arange(d, device=dev())
    hit = (t >= col) & (col > 0)  # column c is NaN from key c on
    if d == 64:
        hit = hit | (t >= 64)      # key 64 brings column 0 too
        hit[:, 0] = torch.arange(200, device=dev()) >= 64
    assert torch.equal(o.isnan(), hit[:, None].expand_as(o)) and lse.isfinite().all()


def test_attend_fp32_at_the_end_of_its_range():
    c = Case([(0, 100)], kind="f32", heads=2, kv_heads=1, d=64)
    want, _, far, _ = c.ref()
    for j, x in ((60, 3.4028e38), (61, -3.4028e38), (70, 3.40199e38), (71, 3.0e38)):
        c.v[int(c.table[0, j // 16]), j % 16, 0, 5] = x
    o, _ = c.call()
    assert ((o.double() - want).abs() <= far)[:60].all()
    rest = [i for i in range(64) if i != 5]
    assert ((o.double() - want).abs() <= far)[..., rest].all()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_lists_of_requests_that_are_not_in_order_stay_in_bounds(kind):
    # cu_new that goes back and forth: rows hold some request's attention, nothing else is written
    c = Case([(50, 20), (30, 40), (0, 30)], kind=kind, heads=4, kv_heads=2, behind=10)
    o, lse = torch.full_like(c.q, 7.0), torch.full(c.q.shape[:2], 7.0, device=dev())
    c.cu.copy_(i32([60, 10, 2 ** 31 - 1, 5]))
    c.call(o=o, lse=lse)
    c.cu.copy_(i32([-7, 1000, 0, 95]))
    c.call(o=o, lse=lse)
    torch.cuda.synchronize()
    assert o.shape == c.q.shape


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,V", [(1, 150000), (3, 150000), (700, 9001)])
@pytest.mark.parametrize("live", [0, 1, 5, 40])
def test_logprobs_of_rows_masked_almost_everywhere(kind, B, V, live):
    for mask in (-INF, torch.finfo(TYPES[kind]).min):
        x = torch.full((B, V), mask, device=dev(), dtype=TYPES[kind])
        if live:
            at = torch.randint(0, V, (B, live), device=dev(), generator=gen(live))
            x.scatter_(1, at, torch.randn((B, live), device=dev(), generator=gen(V)).to(x.dtype))
        check_logprobs(x, [i % V for i in range(B)], 20)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_logprobs_nan_almost_everywhere(kind):
    x = torch.full((3, 60000), NAN, device=dev(), dtype=TYPES[kind])
    x[0, 100:110], x[1, 59990:], x[2, 7] = 1.0, -INF, 3.0
    got, entropy, top_tokens, top_logprobs = gdn.gdn_logprobs(x, i32([0, 1, 2]), top=16)
    assert got.isnan().all() and entropy.isnan().all() and top_logprobs.isnan().all()
    assert top_tokens[0].tolist() == [*range(100, 110), *range(6)]
    assert top_tokens[1].tolist() == [*range(59990, 60000), *range(6)]
    assert top_tokens[2].tolist() == [7, *range(7), *range(8, 16)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_logprobs_far_from_zero(kind):
    # the distribution is that of the differences
    x = (torch.randn((6, 30001), device=dev(), generator=gen(0)) * 3).to(TYPES[kind])
    x[1] = (x[1].float() + 30000).to(x.dtype)
    x[2] = (x[2].float() - 30000).to(x.dtype)
    x[3] = (x[3].float() * 1e30).to(x.dtype)
    x[4] = (x[4].float() * 1e-30).to(x.dtype)
    x[5, ::3] = torch.finfo(x.dtype).max
    check_logprobs(x, [5, 6, 7, 8, 9, 3], 32)


def test_logprobs_of_overlapping_rows():
    x = torch.randn(20000, device=dev(), generator=gen(1))
    check_logprobs(x.as_strided((50, 10007), (1, 1)), list(range(50)), 9)
    check_logprobs(x[:10007].expand(5, -1), list(range(5)), 9)


def test_rope_of_more_heads_than_a_cta_takes():
    check_rope(n=3, heads=(96, 8))
    check_rope(n=1, heads=(300, 1), kind="f32", d=256)
    check_rope(n=2, heads=(40, 40), d=64, pairs=16)


def test_prompt_calls_captured_in_one_graph_and_replayed():
    c = Case([(70, 20), (0, 13)], heads=4, kv_heads=2, d=64, page=16)
    n = c.q.shape[0]
    freqs = 1e4 ** (-torch.arange(32, dtype=torch.float64, device=dev()) / 32)
    pos, tok = i32([*range(70, 90), *range(13)]), i32([0] * n)
    ws, head = gdn.Workspace(), torch.randn((256, 777), device=dev(), generator=gen(2)).bfloat16()
    bufs = dict(o=torch.zeros_like(c.q), lse=torch.zeros(c.q.shape[:2], device=dev()))

    def step():
        q, k = gdn.gdn_qk_rope(c.q, c.q[:, :2], pos, freqs)
        o, _ = gdn.gdn_paged_prefill(q, c.k, c.v, c.table, c.lens, c.cu, workspace=ws, **bufs)
        return [k, o, *gdn.gdn_logprobs(o.reshape(n, -1) @ head, tok, top=4)]
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gdn.gdn_paged_prefill_status(ws) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_attend_more_units_than_the_plan_holds_in_shared_memory(kind):
    r = torch.Generator().manual_seed(5)
    Case([(int(c), int(n)) for c, n in torch.randint(0, 5, (2600, 2), generator=r)] + [(40, 2)], kind=kind, d=64, page=8, heads=2, kv_heads=2).check()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_queries_past_32_bits(kind):
    c = Case([(70, 20), (0, 13)], kind=kind, heads=4, kv_heads=2)
    want = c.check()
    far = torch.empty(34 * 2 ** 27, dtype=c.q.dtype, device=dev()).as_strided(c.q.shape, (2 ** 27, 2 ** 25, 1))  # of 33 rows of 2^27
    far.copy_(c.q)
    c.q = far
    assert all(torch.equal(x, y) for x, y in zip(c.call(), want))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rope_and_logprobs_past_32_bits(kind):
    store = torch.empty(34 * 2 ** 27, dtype=TYPES[kind], device=dev())
    far = store.as_strided((33, 4, 128), (2 ** 27, 2 ** 25, 1))
    x = torch.randn((33, 4, 128), device=dev(), generator=gen(4)).to(TYPES[kind])
    pos, freqs = i32(list(range(33))), torch.linspace(0, 1, 64, dtype=torch.float64, device=dev())
    far.copy_(x)
    want = gdn.gdn_qk_rope(x, x[:, :1], pos, freqs)[0]
    assert torch.equal(gdn.gdn_qk_rope(far, x[:, :1], pos, freqs)[0], want)
    assert torch.equal(gdn.gdn_qk_rope(far, x[:, :1], pos, freqs, q_out=far)[0], want)
    rows = store.as_strided((33, 5003), (2 ** 27, 1))
    rows.copy_(torch.randn((33, 5003), device=dev(), generator=gen(5)))
    check_logprobs(rows, list(range(33)), 7)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_threads_of_one_stream(kind):
    # each thread's calls have a workspace of their own, whatever comes between their launches
    cases = [Case([(900, 70 + 10 * i), (0, 300), (33, 1)], kind=kind, seed=i, heads=4, kv_heads=2) for i in range(4)]
    want = [c.call() for c in cases]
    torch.cuda.synchronize()
    with ThreadPoolExecutor(len(cases)) as pool:
        got = list(pool.map(lambda c: [c.call() for _ in range(20)], cases))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x in a:
            assert torch.equal(x[0], b[0]) and torch.equal(x[1], b[1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,page", [(64, 64), (128, 64), (128, 16), (128, 1), (256, 64)])
def test_attend_copies_that_come_in_any_order(kind, d, page):
    # units of one row tile and of two take turns over contexts that no cache holds: a stage of keys or values may come after later ones
    sizes = [(13000, 100), (25000, 1), (9500, 1), (17000, 1), (6800, 1), (28000, 1), (5300, 70), (0, 60), (8800, 1), (30000, 130), (0, 1), (12800, 1), (64, 33), (2, 1), (22600, 1)]
    scale = 8 if kind == "f32" or d == 256 else 1
    c = Case([(a // scale, b) for a, b in sizes], kind=kind, heads=16, kv_heads=4, d=d, page=page)
    ws = gdn.Workspace()
    want = c.check(workspace=ws)
    for _ in range(30):
        got = c.call(workspace=ws)
        assert gdn.gdn_paged_prefill_status(ws) == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_units_of_one_tile_over_cold_keys(kind, d):
    # a tile of keys and one of values to each unit, thousands in a row
    c = Case([(0, 1 + i % 40) for i in range(3000)], kind=kind, heads=8, kv_heads=4, d=d, page=64)
    ws = gdn.Workspace()
    want = c.call(workspace=ws)
    for _ in range(20):
        got = c.call(workspace=ws)
        assert gdn.gdn_paged_prefill_status(ws) == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
