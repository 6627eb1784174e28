"""The decode step over a paged key-value cache against plain implementations in 64 bits.

Tolerances, from the arithmetic: scores are fp32 sums of d products, off by at most
d 2^-24 sum |q_i k_i| scale; so is lse (plus 2^-20 for exp and log), and a weight is off by
that much relatively.  Outputs in fp32: 1e-5 of a row's norm, the library's limit for fp32
storage.  Outputs in bf16: 2^-9 from rounding the output, and less than that from weights
held to 2^-12 of their size, so 2^-8 of a row's norm.  Slots, tables and tokens are exact.
"""
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_16_gb300 as gdn

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
ROW_TOL = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -8, "f32": 1e-5}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_delta_rule_16_gb300 import build
    build.build()
    gdn.load()


def dev():
    return torch.device("cuda:0")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


# ---- block tables and slot maps ---------------------------------------------------------------
def ref_tables(cached, new, free, table, page, n_slots):
    table = table.copy()
    B, wide = table.shape
    cached, new = [max(c, 0) for c in cached], [max(n, 0) for n in new]
    slots, pos, cu, status = [], [], [0], 0
    taken = 0
    for b in range(B):
        old, need = -(-cached[b] // page), -(-(cached[b] + new[b]) // page)
        if need > wide:
            status |= 2
        for j in range(old, wide):
            if j < min(need, wide):
                table[b, j] = free[taken] if taken < len(free) else -1
                taken += 1
            else:
                table[b, j] = -1
        for p in range(cached[b], cached[b] + new[b]):
            c = p // page
            ok = c < wide and table[b, c] >= 0
            slots.append(int(table[b, c]) * page + p % page if ok else -1)
            pos.append(p)
        cu.append(len(slots))
    if taken > len(free):
        status |= 1
    if len(slots) > n_slots:
        status |= 4
    total = len(slots)
    slots = (slots + [-1] * n_slots)[:n_slots]
    pos = (pos + [0] * n_slots)[:n_slots]
    lens = [c + n for c, n in zip(cached, new)]
    return table, slots, pos, lens, cu, [total, min(taken, len(free)), status, max(lens, default=0)]


def check_tables(cached, new, page, wide, n_free, n_slots, seed=0):
    r = np.random.default_rng(seed)
    B = len(new)
    have = [-(-max(c, 0) // page) for c in (cached or [0] * B)]
    ids = r.permutation(sum(have) + n_free).astype(np.int32)
    table = r.integers(-1, 5, (B, wide)).astype(np.int32)  # stale entries behind the pages held
    at = 0
    for b in range(B):
        for j in range(min(have[b], wide)):
            table[b, j] = ids[at]
            at += 1
    free = ids[len(ids) - n_free:]
    want = ref_tables(cached or [0] * B, new, free, table, page, n_slots)
    t = torch.from_numpy(table).to(dev())
    for _ in range(2):  # the second call writes the same values
        slots, pos, lens, cu, counts = gdn.gdn_page_tables(i32(new), i32(free.tolist()), t, page=page,
                                                           cached_lens=None if cached is None else i32(cached), n_slots=n_slots)
        got = [t.cpu().numpy(), slots.cpu().tolist(), pos.cpu().tolist(), lens.cpu().tolist(), cu.cpu().tolist(), counts.cpu().tolist()]
        assert np.array_equal(got[0], want[0])
        assert got[1:] == [*want[1:]]
        assert gdn.gdn_page_tables_status(counts) == (9 if want[5][2] else 0)


@pytest.mark.parametrize("B", [1, 2, 33, 511, 512, 513, 1300])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_tables_ragged(B, page):
    r = np.random.default_rng(B * 100 + page)
    cached = r.integers(0, 90, B).tolist()
    new = np.where(r.random(B) < 0.3, 0, r.integers(0, 40, B)).tolist()
    wide = -(-130 // page)
    check_tables(cached, new, page, wide, sum(new) // page + 2 * B, sum(new) + 7, B)


def test_tables_one_token_each_and_none_cached():
    check_tables([15, 16, 17, 0, 31], [1, 1, 1, 1, 1], 16, 4, 8, 5)
    check_tables(None, [5, 0, 33, 16], 16, 4, 8, 60)
    check_tables(None, [70000], 64, 1100, 1100, 70000)          # one long prompt, many CTAs
    check_tables([3, 4], [0, 0], 16, 2, 0, 0)                   # nothing to add, no slots, no free page


def test_tables_limits_are_latched_and_nothing_passes_them():
    check_tables([0, 10, 20], [40, 40, 40], 16, 8, 4, 120)      # free list too short: 1
    check_tables([0, 10, 20], [40, 90, 40], 16, 3, 40, 200)     # a row too short: 2
    check_tables([0, 10, 20], [40, 40, 40], 16, 8, 40, 50)      # slot map too short: 4
    check_tables([-3, 10], [5, -7], 16, 2, 4, 8)                # negative lengths count as 0
    check_tables([100, 0], [5, 5], 16, 2, 4, 12)                # more cached than the row holds


def test_tables_no_request():
    slots, pos, lens, cu, counts = gdn.gdn_page_tables(i32([]), i32([1, 2]), torch.empty((0, 4), dtype=torch.int32, device=dev()), page=16,
                                                       n_slots=3)
    assert slots.tolist() == [-1] * 3 and pos.tolist() == [0] * 3 and cu.tolist() == [0] and counts.tolist() == [0, 0, 0, 0]


# ---- cache writes -------------------------------------------------------------------------------
def e4m3_codes():
    """(values of the codes 0..126 in ascending order, in 64 bits)."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


def ref_e4m3(x32):
    """Codes of the nearest e4m3 values to fp32 numbers, ties to the even code, saturated."""
    v = e4m3_codes()
    x = x32.astype(np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(v, a), 1, 126)
    lo = hi - 1
    dl, dh = a - v[lo], v[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 0x7F, code) | (np.signbit(x32).astype(np.int64) << 7)
    return code.astype(np.uint8)


def new_cache(kind, pages, page, heads, d, head_major, fill=0.0):
    shape = (pages, heads, page, d) if head_major else (pages, page, heads, d)
    k, v = (torch.full(shape, fill, device=dev(), dtype=torch.float32).to(TYPES[kind]) for _ in range(2))
    return (k.transpose(1, 2), v.transpose(1, 2)) if head_major else (k, v)


@pytest.mark.parametrize("kind,src", [("bf16", "bf16"), ("f32", "f32"), ("e4m3", "bf16"), ("e4m3", "f32")])
@pytest.mark.parametrize("n,heads,d,page,head_major", [(1, 1, 64, 1, False), (37, 3, 128, 24, True), (300, 8, 256, 16, False),
                                                       (1025, 2, 64, 64, True)])
def test_append(kind, src, n, heads, d, page, head_major):
    g = torch.Generator(device=dev()).manual_seed(n * 7 + d)
    pages = -(-n // page) + 3
    k_cache, v_cache = new_cache(kind, pages, page, heads, d, head_major, 1.5)
    kv = torch.randn((n, 2 * heads, d), device=dev(), generator=g) * 3
    kv.view(-1)[::97] *= 1e4                       # past the 8-bit range
    kv.view(-1)[1::89] *= 1e-4                     # its subnormals and zero
    kv = kv.to(TYPES[src])
    kv[0, 0, 0], kv[0, heads, 1], kv[0, heads, 2] = float("nan"), float("inf"), float("-inf")
    k, v = kv[:, :heads], kv[:, heads:]            # slices of one tensor: strided rows
    perm = torch.randperm(pages * page, device=dev(), generator=g)
    slots = perm[:n].clone()
    if n > 3:
        slots[1], slots[2], slots[n - 1] = -1, pages * page, -(2 ** 40)   # skipped
    scales = [None, None]
    if kind == "e4m3":
        scales = [torch.rand(heads, device=dev(), generator=g) * 0.05 + 0.01 for _ in range(2)]
    before = [c.clone() for c in (k_cache, v_cache)]
    gdn.gdn_kv_append(k, v, slots, k_cache, v_cache, k_scale=scales[0], v_scale=scales[1])
    s = slots.cpu().numpy()
    real = (s >= 0) & (s < pages * page)
    for got, was, x, scale in zip((k_cache, v_cache), before, (k, v), scales):
        word = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[got.element_size()]
        bits, want = got.contiguous().view(word).cpu().numpy(), was.contiguous().view(word).cpu().numpy()
        if kind == "e4m3":
            x32 = (x.float() / scale[:, None]).cpu().numpy()
            rows = ref_e4m3(x32)
            nan = np.isnan(x32)
        else:
            rows, nan = x.contiguous().view(word).cpu().numpy(), None
        want[s[real] // page, s[real] % page] = rows[real]
        if nan is not None:  # any NaN code will do
            w = np.zeros(want.shape, bool)
            w[s[real] // page, s[real] % page] = nan[real]
            assert ((bits[w] & 0x7F) == 0x7F).all()
            bits[w] = want[w]
        assert np.array_equal(bits, want)


def test_append_nothing():
    k_cache, v_cache = new_cache("bf16", 2, 16, 2, 64, False)
    x = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=dev())
    gdn.gdn_kv_append(x, x, torch.zeros(0, dtype=torch.int64, device=dev()), k_cache, v_cache)
    assert not k_cache.any()


# ---- attention of one token over the cache --------------------------------------------------------
def make(kind, lens, heads, group, d, page, head_major=False, seed=0, spread=2.0, table_pad=2):
    g = torch.Generator(device=dev()).manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    shape = (pages, heads, page, d) if head_major else (pages, page, heads, d)
    x = torch.randn((2, *shape), device=dev(), generator=g)
    scales = (None, None)
    if kind == "e4m3":
        scales = tuple(0.01 + 0.01 * torch.rand(heads, device=dev(), generator=g) for _ in range(2))
        x = (x * 80.0).clamp(-448.0, 448.0)  # torch's cast does not saturate
    x = x.to(TYPES[kind])
    k, v = (t.transpose(1, 2) if head_major else t for t in (x[0], x[1]))
    ids = torch.randperm(pages, device=dev(), generator=g).tolist()
    table = torch.full((len(lens), max(need, default=0) + table_pad), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(ids[at:at + m], dtype=torch.int32)
        at += m
    q = (spread * torch.randn((len(lens), heads * group, d), device=dev(), generator=g)).to(TYPES["f32" if kind == "f32" else "bf16"])
    return dict(q=q, k_cache=k, v_cache=v, block_table=table.to(dev()), seq_lens=i32(lens), k_scale=scales[0], v_scale=scales[1])


def poison(s):
    """NaN in every cell that no request's tokens use."""
    pages, page = s["k_cache"].shape[:2]
    used = torch.zeros((pages, page), dtype=torch.bool, device=dev())
    for b, n in enumerate(s["seq_lens"].tolist()):
        j = torch.arange(n, device=dev())
        ids = s["block_table"][b].long()[j // page]
        ok = (ids >= 0) & (ids < pages)
        used[ids[ok], (j % page)[ok]] = True
    for c in (s["k_cache"], s["v_cache"]):
        if c.dtype == torch.float8_e4m3fn:
            c.view(torch.uint8)[~used] = 0x7F
        else:
            c[~used] = float("nan")


def ref_attend(s, window=0, scale=None):
    """(o, lse, bound on the scores' error) in 64 bits, request by request."""
    q = s["q"].double()
    B, Hq, d = q.shape
    pages, page, heads, _ = s["k_cache"].shape
    scale = d ** -0.5 if scale is None else scale
    o, lse, off = torch.zeros_like(q), torch.full((B, Hq), -math.inf, dtype=torch.float64, device=dev()), torch.zeros(B, Hq, device=dev()).double()
    for b, n in enumerate(s["seq_lens"].tolist()):
        n = min(max(n, 0), s["block_table"].shape[1] * page)
        j = torch.arange(max(0, n - window) if window else 0, n, device=dev())
        ids = s["block_table"][b].long()[j // page]
        ok = (ids >= 0) & (ids < pages)
        j, ids = j[ok], ids[ok]
        if len(j) == 0:
            continue
        for h in range(heads):
            kv = []
            for c, f in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
                x = c.view(torch.uint8)[ids, j % page, h].view(c.dtype) if f is not None else c[ids, j % page, h]
                kv.append(x.double() * (1.0 if f is None else f[h].double()))
            hs = slice(h * (Hq // heads), (h + 1) * (Hq // heads))
            z = q[b, hs] @ kv[0].T * scale
            o[b, hs] = torch.softmax(z, 1) @ kv[1]
            lse[b, hs] = torch.logsumexp(z, 1)
            off[b, hs] = (q[b, hs].abs() @ kv[0].T.abs()).amax(1) * scale * d * 2.0 ** -24
    return o, lse, off


def check_attend(kind, s, window=0, **kw):
    o, lse = gdn.gdn_paged_decode(**s, window=window, **kw)
    want_o, want_lse, off = ref_attend(s, window, kw.get("scale"))
    assert o.dtype == s["q"].dtype and torch.isfinite(o).all()
    err = (o.double() - want_o).norm(dim=-1)
    assert (err <= ROW_TOL[kind] * want_o.norm(dim=-1)).all(), (err / want_o.norm(dim=-1)).nan_to_num().max().item()
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (o[empty] == 0).all()
    d = (lse.double() - want_lse).abs()[~empty]
    assert (d <= off[~empty] + 2.0 ** -20 * (1 + want_lse[~empty].abs())).all(), d.max().item()
    again = gdn.gdn_paged_decode(**s, window=window, **kw)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])  # the same call, the same bits
    return o, lse


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 9, 16])
def test_attend_types_and_heads(kind, d, group):
    s = make(kind, [1, 0, 63, 64, 65, 200, 17, 1029], 2, group, d, 16, head_major=group % 2 == 0, seed=d + group)
    poison(s)
    check_attend(kind, s)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("group", [17, 32, 40])
def test_attend_many_query_heads_per_kv_head(kind, group):
    check_attend(kind, make(kind, [5, 333], 2, group, 128, 32, seed=group))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 100, 4096])
def test_attend_pages(kind, page):
    s = make(kind, [1, 16, 100, 101, 515, 0, 2050], 3, 4, 64, page, head_major=page % 2 == 0, seed=page)
    poison(s)
    check_attend(kind, s)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 5000])
def test_attend_window(kind, window):
    check_attend(kind, make(kind, [1, 7, 64, 300, 1000, 0, 129], 2, 4, 128, 24, seed=window), window)


@pytest.mark.parametrize("lens", [[1], [2], [40000], [0], [0, 0, 0], [30000, 1, 1, 1], list(range(0, 700, 7)), [3] * 1100, [100] * 400])
def test_attend_lengths(lens):
    s = make("bf16", lens, 1, 8, 128, 16, seed=len(lens))
    poison(s)
    check_attend("bf16", s)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_attend_ids_outside_the_pool_are_masked(kind):
    s = make(kind, [100, 64, 700, 33], 2, 4, 128, 16, seed=5)
    t = s["block_table"]
    t[0, 2], t[1, :], t[2, 3], t[2, 10] = -1, -1, 1 << 30, -(2 ** 31)
    poison(s)
    check_attend(kind, s)


def test_attend_length_is_cut_at_the_table():
    s = make("bf16", [100, 64], 2, 4, 128, 16, seed=6, table_pad=0)
    s["seq_lens"] = i32([1 << 30, -5])
    check_attend("bf16", s)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_attend_sharp_and_extreme_scores(kind):
    # one token takes nearly everything; scores of thousands; queries of tiny and huge size
    s = make(kind, [50, 500, 3000], 2, 4, 128, 16, seed=8, spread=60.0)
    check_attend(kind, s)
    s["q"] = s["q"] * 0
    o, lse = check_attend(kind, s)  # uniform weights
    assert torch.allclose(lse[2], torch.tensor(math.log(3000.0), device=dev()), atol=1e-5)
    s = make(kind, [50, 500], 2, 4, 128, 16, seed=9)
    s["q"] = s["q"] * 1e30
    check_attend(kind, s, scale=2.0 ** -104)
    s["q"] = s["q"] * 1e-36 * 1e-30
    check_attend(kind, s, scale=2.0 ** 100)


def test_attend_nan_and_inf_stay_in_their_row():
    s = make("bf16", [40, 90, 200], 2, 4, 128, 16, seed=10)
    page, cell = int(s["block_table"][1, 2]), 5
    s["k_cache"][page, cell, 0, 3] = float("nan")
    s["v_cache"][int(s["block_table"][2, 0]), 0, 1, 7] = float("inf")
    o, lse = gdn.gdn_paged_decode(**s)
    assert torch.isnan(o[1, :4]).all() and torch.isnan(lse[1, :4]).all()
    assert torch.isinf(o[2, 4:, 7]).all() and torch.isfinite(lse[2]).all()
    o[1, :4], o[2, 4:, 7] = 0, 0
    assert torch.isfinite(o).all()


def test_attend_strides_streams_and_given_outputs():
    s = make("bf16", [100, 257, 31], 2, 4, 128, 16, seed=11)
    want = gdn.gdn_paged_decode(**s)
    # queries inside a wider projection, a table that is a slice of a wider one
    wide = torch.randn((3, 20, 128), device=dev()).to(torch.bfloat16)
    wide[:, 4:12] = s["q"]
    table = torch.full((3, 50), 7, dtype=torch.int32, device=dev())
    n = s["block_table"].shape[1]
    table[:, 20:20 + n] = s["block_table"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = torch.full_like(want[0], 9), torch.full_like(want[1], 9)
    got = gdn.gdn_paged_decode(**{**s, "q": wide[:, 4:12], "block_table": table[:, 20:20 + n]}, o=o, lse=lse, stream=side, workspace=gdn.Workspace())
    side.synchronize()
    assert got[0] is o and got[1] is lse and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    with torch.cuda.stream(side):
        got = gdn.gdn_paged_decode(**s)
    side.synchronize()
    assert torch.equal(got[0], want[0])


def test_attend_a_chunk_of_rows_over_one_table_row():
    s = make("bf16", [300], 2, 4, 128, 16, seed=12)
    rows = 20
    q = torch.randn((rows, 8, 128), device=dev()).to(torch.bfloat16)
    lens = i32(list(range(281, 301)))
    o, lse = gdn.gdn_paged_decode(q, s["k_cache"], s["v_cache"], s["block_table"].expand(rows, -1), lens)
    for r in (0, 7, 19):
        one = {**s, "q": q[r:r + 1], "seq_lens": lens[r:r + 1]}
        want = ref_attend(one)
        assert (o[r].double() - want[0][0]).norm(dim=-1).le(2.0 ** -8 * want[0][0].norm(dim=-1)).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_attend_offsets_past_32_bits(kind):
    # the pool holds more than 2^32 elements; the pages in use lie at its end
    page, heads, d = 64, 8, 128
    pages = (1 << 32) // (page * heads * d) + 40
    s = make(kind, [700, 90], heads, 2, d, page, seed=13)
    small = s["k_cache"].shape[0]
    for name in ("k_cache", "v_cache"):
        big = torch.empty((pages, page, heads, d), dtype=TYPES[kind], device=dev())
        big[pages - small:] = s[name]
        s[name] = big
    s["block_table"] = torch.where(s["block_table"] >= 0, s["block_table"] + pages - small, -1)
    check_attend(kind, s)
    k = torch.randn((3, heads, d), device=dev()).to(torch.float32 if kind == "f32" else torch.bfloat16)
    slots = torch.tensor([pages * page - 1, -1, pages * page - page * 2 - 3], device=dev())
    gdn.gdn_kv_append(k, k, slots, s["k_cache"], s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    for r in (0, 2):
        got = s["v_cache"][int(slots[r]) // page, int(slots[r]) % page].float()
        want = k[r].float() if kind != "e4m3" else (k[r].float() / s["v_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float()
        assert torch.equal(got, want)


def test_attend_under_graph_replay_with_growing_lengths():
    s = make("bf16", [100, 1000, 40], 2, 8, 128, 16, seed=14)
    ws = gdn.Workspace()
    o, lse = gdn.gdn_paged_decode(**s, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_paged_decode(**s, workspace=ws, o=o, lse=lse)
    for lens in ([1, 1000, 0], [100, 3, 40], [64, 999, 17]):
        s["seq_lens"].copy_(i32(lens))
        g.replay()
        torch.cuda.synchronize()
        want = gdn.gdn_paged_decode(**s)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_attend_no_request_no_page():
    s = make("bf16", [5], 2, 4, 64, 16, seed=15)
    o, lse = gdn.gdn_paged_decode(s["q"][:0], s["k_cache"], s["v_cache"], s["block_table"][:0], s["seq_lens"][:0])
    assert o.shape == (0, 8, 64) and lse.shape == (0, 8)
    o, lse = gdn.gdn_paged_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"][:, :0], s["seq_lens"])
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = gdn.gdn_paged_decode(s["q"], s["k_cache"][:0], s["v_cache"][:0], s["block_table"], s["seq_lens"])
    assert (o == 0).all() and torch.isneginf(lse).all()


# ---- sampling -------------------------------------------------------------------------------------
def ref_sample(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, logprob) of one row in 64 bits, over a sorted list."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x.astype(np.float64), 3.402823466e38))
    if not (x > -np.inf).any():
        return -1, -math.inf
    if not t > 0:
        return int(np.argmax(x)), 0.0
    with np.errstate(all="ignore"):
        y = (x - x.max()) / t
        w = np.exp(y)
    order = np.lexsort((np.arange(len(x)), -x))
    if 0 < k < len(x):
        order = order[:k]
    if p < 1:
        mass = np.cumsum(w[order])
        order = order[:1 + int(np.searchsorted(mass, max(p, 0.0) * mass[-1], side="left"))]
    keep = [i for i in order if w[i] > 0 and w[i] >= m] or [int(np.argmax(x))]
    uu = np.clip(u.astype(np.float64), 2.0 ** -32, 1 - 2.0 ** -24)
    best = max(keep, key=lambda i: (y[i] - math.log(-math.log(uu[i])), -i))
    return int(best), float(y[best] - math.log(w.sum()))


def check_sample(x, u, t=None, k=None, p=None, m=None):
    f = lambda v: None if v is None else torch.tensor(v, dtype=torch.float32, device=dev())
    tok, lp = gdn.gdn_sample(x, u, temperature=f(t), top_k=None if k is None else i32(k), top_p=f(p), min_p=f(m))
    xs, us = x.float().cpu().numpy(), u.cpu().numpy()
    f32 = lambda v: float(np.float32(v))
    for b in range(x.shape[0]):
        want = ref_sample(xs[b], us[b], f32(t[b]) if t else 1.0, k[b] if k else 0, f32(p[b]) if p else 1.0, f32(m[b]) if m else 0.0)
        assert int(tok[b]) == want[0], (b, int(tok[b]), want)
        if math.isinf(want[1]):
            assert float(lp[b]) == want[1]
        else:
            # y is off by 2^-23 of its size, the sum of weights by 2^-22 relatively, the result by its own rounding
            assert abs(float(lp[b]) - want[1]) <= 2.0 ** -21 * (1 + abs(want[1])) + 2.0 ** -22 * abs(want[1])
    return tok, lp


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (5, 31), (4, 1000), (2, 4097), (7, 32768), (3, 100003), (1, 300000)])
def test_sample_filters(kind, B, V):
    g = torch.Generator(device=dev()).manual_seed(V)
    x = (3 * torch.randn((B, V), device=dev(), generator=g)).to(TYPES[kind])
    u = torch.rand((B, V), device=dev(), generator=g)
    r = np.random.default_rng(V)
    pick = lambda *c: [c[i] for i in r.integers(0, len(c), B)]
    check_sample(x, u)
    check_sample(x, u, t=pick(0.5, 1.0, 1.7))
    check_sample(x, u, t=pick(0.7, 1.0), k=pick(1, 2, 20, V, V + 5, -1))
    check_sample(x, u, p=pick(0.0, 0.3, 0.9, 0.999, 1.0))
    check_sample(x, u, m=pick(0.0, 0.01, 0.5, 1.0, 2.0))
    for _ in range(3):
        check_sample(x, u, t=pick(0.0, 0.3, 1.0), k=pick(0, 5, 50, 3000), p=pick(0.5, 0.9, 1.0), m=pick(0.0, 0.05))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_sample_ties_go_to_the_lowest_index(kind):
    V = 5000
    x = torch.zeros((4, V), device=dev(), dtype=TYPES[kind])
    x[1, ::2] = -0.0                                # equal to 0
    x[2, 100:200] = 1.0
    x[3] = float(torch.finfo(TYPES[kind]).min)      # a row of the type's lowest value: uniform
    u = torch.rand((4, V), device=dev(), generator=torch.Generator(device=dev()).manual_seed(1))
    check_sample(x, u, k=[1, 1, 1, 1])
    check_sample(x, u, k=[7, 300, 150, 50])
    check_sample(x, u, p=[0.25, 0.5, 0.01, 0.75])
    check_sample(x, u, k=[1000, 1000, 150, 64], p=[0.1, 0.9, 0.7, 0.5])
    check_sample(x, torch.full_like(u, 0.5))        # equal noise as well: the first of the largest
    tok, _ = check_sample(x, u, t=[0.0] * 4)
    assert tok.tolist() == [0, 0, 100, 0]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_sample_infinities_nan_and_masked_rows(kind):
    V, ninf = 3001, -math.inf
    g = torch.Generator(device=dev()).manual_seed(3)
    x = torch.randn((8, V), device=dev(), generator=g).to(TYPES[kind])
    x[0] = ninf                                     # nothing left
    x[1] = float("nan")
    x[2] = ninf
    x[2, 2999] = -5.0                               # one token left
    x[3, 17] = math.inf
    x[4, ::2] = ninf
    x[4, 1::4] = float("nan")
    x[5, 5:] = float(torch.finfo(TYPES[kind]).min)
    x[6] = ninf
    x[6, [10, 20]] = math.inf                       # two largest
    u = torch.rand((8, V), device=dev(), generator=g)
    u[7, :1500] = 0.0                               # clamped at both ends
    u[7, 1500:] = 1.0
    for t in (0.0, 0.6):
        for k in (0, 1, 40):
            for p in (0.3, 1.0):
                tok, lp = check_sample(x, u, t=[t] * 8, k=[k] * 8, p=[p] * 8, m=[0.02] * 8)
                assert tok[:3].tolist() == [-1, -1, 2999] and int(tok[3]) == 17


def test_sample_row_strides_and_stream():
    g = torch.Generator(device=dev()).manual_seed(4)
    big = torch.randn((6, 1009), device=dev(), generator=g).to(torch.bfloat16)
    noise = torch.rand((6, 1501), device=dev(), generator=g)
    x, u = big[:, 3:1004], noise[:, 1:1002]         # rows at odd addresses
    check_sample(x, u, t=[0.9] * 6, k=[30] * 6, p=[0.8] * 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = gdn.gdn_sample(x, u)
    got = gdn.gdn_sample(x, u, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_sample_draws_follow_the_weights():
    # 20000 draws of a 6-token row: each count within 5 standard deviations of its expectation
    n, V = 20000, 6
    x = torch.tensor([1.0, 0.0, 2.0, -1.0, 0.5, -math.inf], device=dev()).expand(n, V).contiguous()
    u = torch.rand((n, V), device=dev(), generator=torch.Generator(device=dev()).manual_seed(5))
    tok, _ = gdn.gdn_sample(x, u)
    w = torch.softmax(x[0].double(), 0).cpu().numpy()
    c = torch.bincount(tok.long(), minlength=V).cpu().numpy()
    assert (np.abs(c - n * w) <= 5 * np.sqrt(n * w * (1 - w)) + 1e-9).all(), c


def test_refusals():
    s = make("bf16", [40, 90], 2, 4, 128, 16, seed=20)
    call = lambda **kw: gdn.gdn_paged_decode(**{**s, **kw})
    for kw in (dict(q=s["q"].float()), dict(block_table=s["block_table"].long()), dict(seq_lens=s["seq_lens"].long()),
               dict(k_cache=s["k_cache"].half(), v_cache=s["v_cache"].half())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=s["q"][:, :, :64]), dict(seq_lens=s["seq_lens"][:1]), dict(block_table=s["block_table"][:1]),
               dict(v_cache=s["v_cache"][:2]), dict(k_scale=torch.ones(2, device=dev())), dict(seq_lens=s["seq_lens"].cpu()),
               dict(q=s["q"].transpose(1, 2).contiguous().transpose(1, 2)), dict(o=torch.empty(1, device=dev(), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=s["q"][:, :7]), dict(window=-1), dict(workspace=torch.empty(8, dtype=torch.uint8, device=dev()))):
        with pytest.raises(gdn.GdnError):
            call(**kw)
    e = make("e4m3", [40], 2, 4, 128, 16, seed=21)
    with pytest.raises(ValueError):
        gdn.gdn_paged_decode(e["q"], e["k_cache"], e["v_cache"], e["block_table"], e["seq_lens"])
    x = torch.randn((2, 50), device=dev())
    with pytest.raises(ValueError):
        gdn.gdn_sample(x, x[:1])
    with pytest.raises(TypeError):
        gdn.gdn_sample(x.half(), x)
    with pytest.raises(TypeError):
        gdn.gdn_sample(x, x, top_k=torch.ones(2, device=dev()))
    with pytest.raises(ValueError):
        gdn.gdn_sample(x.T, x.T)
    with pytest.raises(ValueError):
        gdn.gdn_page_tables(i32([1]), i32([1]), i32([[1]]), page=16)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_page_tables(i32([1]), i32([1]), i32([[1]]), page=0, n_slots=1)
    k = torch.zeros((3, 2, 128), dtype=torch.float32, device=dev())
    with pytest.raises(gdn.GdnError):
        gdn.gdn_kv_append(k, k, torch.zeros(3, dtype=torch.int64, device=dev()), s["k_cache"], s["v_cache"])
    with pytest.raises(ValueError):
        gdn.gdn_kv_append(k[:2], k[:2], torch.zeros(3, dtype=torch.int64, device=dev()), s["k_cache"], s["v_cache"])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_sample_noise_in_the_logits_order(kind):
    # the race's best are outside the kept prefix again and again, in rows too flat for their prefix to be gathered
    V = 60000
    x = torch.linspace(0.0, -2.0, V, device=dev()).to(TYPES[kind]).repeat(4, 1)
    u = torch.linspace(0.0, 1.0, V, device=dev()).repeat(4, 1)
    check_sample(x, u, t=[1.0, 1.0, 0.5, 2.0], p=[0.5, 0.9, 0.3, 0.01])
    check_sample(x, u, k=[30000, 0, 50000, 5000], p=[0.5, 0.2, 0.7, 0.9])
    check_sample(x.flip(1).contiguous(), u, k=[30000, 0, 50000, 5000], p=[0.5, 0.2, 0.7, 0.9])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("spread", [0.05, 1.0, 8.0])
def test_sample_flat_and_sharp_rows_with_large_k(kind, spread):
    g = torch.Generator(device=dev()).manual_seed(int(spread * 100))
    B, V = 12, 70001
    x = (spread * torch.randn((B, V), device=dev(), generator=g)).to(TYPES[kind])
    x[3, 1000:] = -math.inf
    x[4, ::3] = float(x[4].float().max())            # a third of the row in one tie
    u = torch.rand((B, V), device=dev(), generator=g)
    for k in ([600, 5000, 20000, 900, 30000, 69000, 2048, 2049, 4096, 513, 257, 70000],):
        check_sample(x, u, k=k)
        check_sample(x, u, k=k, p=[0.9, 0.5, 0.99, 0.7, 0.3, 0.05, 0.8, 0.9, 0.95, 0.6, 0.4, 0.2])
        check_sample(x, u, t=[1.5] * B, k=k, p=[0.7] * B, m=[0.0, 0.01, 0.1] * 4)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [900, 70001])
def test_sample_prefix_of_the_largest_token_alone(kind, V):
    # top_p below, at and above the share of the largest token; of equal largest ones the first is the prefix
    g = torch.Generator(device=dev()).manual_seed(V)
    x = (0.5 * torch.randn((8, V), device=dev(), generator=g)).to(TYPES[kind])
    x[0, V // 3] = 16.0                               # nearly all of the mass
    x[1, V // 2] = 9.0
    x[2, [V // 5, V // 2]] = 14.0                     # half of it each
    x[3, [V // 5, V // 2]] = 14.0
    x[4:6] = 0.0                                      # as many shares as tokens
    u = torch.rand((8, V), device=dev(), generator=g)
    for k in (None, [3, 0, 1, 2, 0, 700, 0, 5]):
        tok, _ = check_sample(x, u, k=k, p=[0.9, 0.1, 0.4, 0.6, 0.5 / V, 0.0, 0.0, 1e-7], m=[0.0, 0.0, 0.5, 0.0, 0.0, 0.0, 0.9, 0.0])
        assert tok[2] == V // 5 and tok[4] == 0 and tok[5] == 0


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("e4m3", 128), ("f32", 64), ("bf16", 256)])
@pytest.mark.parametrize("lens", [
    [9000, 1, 0, 17, 12000, 128, 64, 129, 1, 1, 9001, 15000, 3, 63, 65, 14000, 0, 5000],
    [1] * 60 + [20000] + [64, 128, 0, 1] * 12 + [700] * 30 + [19999] + [2] * 40 + [4096, 3],
])
def test_attend_long_and_short_rows_together(kind, d, lens):
    # enough tokens that a row's ends count in the shares of the CTAs, which may then begin or end between two rows
    s = make(kind, lens, 8, 4, d, 16, seed=len(lens) + d)
    poison(s)
    check_attend(kind, s)
    check_attend(kind, s, window=8000)
