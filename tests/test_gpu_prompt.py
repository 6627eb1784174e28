"""A prompt chunk's operators against plain implementations in 64 bits.

Tolerances, from the arithmetic (half a step of rounding: bf16 2^-8, fp16 2^-11, fp32 2^-24 of the value):
  attention  scores are fp32 sums of d products, each addition off by at most 2^-23 (a sum may be cut) of the terms' absolute sum:
             delta = d 2^-23 scale sum |q_i k_i|, and a weight by 2 delta + 2^-20 (exp) relatively.  Weights enter the product
             with V in 8 (bf16), 11 (e4m3) or 22 bits: w = 2^-8, 2^-11, 2^-22 of each, and 2^-32 of the largest at least.  Sums over L
             tokens are off by L 2^-23 at most.  So |o - o*| <= r |o*| + (w + 2 delta + 2^-20 + L 2^-23) sum p |v|, with r = 2^-8 for
             a bf16 output and 2^-24 for fp32; |lse - lse*| <= delta + 2^-20 (1 + |lse*|) + L 2^-23.
  rotary     cos and sin to 2^-22, an angle at position p to (1 + 2^-53 p) 2^-22, norm and products to 2^-21: 2^-19 of |a| + |b|
             besides the output's rounding.
  log probs  exponentials to 2^-20 of each, sums of n to (log2 n + 64) 2^-24: 2^-17 (1 + |x - m|).
"""
import math

import pytest
import torch

import gated_delta_rule_16_gb300 as gdn

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
NAN, INF = float("nan"), float("inf")


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


def gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


# ---- norm and rotary positions -------------------------------------------------------------------
def ref_rope(x, positions, freqs, weight, eps, interleaved, mscale):
    """(values, |a| + |b| of each value's pair) in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    r = freqs.numel()
    angle = positions.double()[:, None] * freqs
    cos, sin = (mscale * torch.cos(angle))[:, None], (mscale * torch.sin(angle))[:, None]
    out, size = x.clone(), x.abs()
    a, b = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else (slice(0, r), slice(r, 2 * r))
    out[..., a], out[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., a] * sin + x[..., b] * cos
    size[..., a] = size[..., b] = abs(mscale) * (x[..., a].abs() + x[..., b].abs())
    return out, size


def check_rope(n=5, heads=(4, 2), d=128, pairs=64, kind="bf16", interleaved=False, norm=True, mscale=1.0, positions=None, inplace=False, seed=0, base=1e4):
    g = gen(seed)
    qkv = (torch.randn((n, heads[0] + 2 * heads[1], d), device=dev(), generator=g) * 3).to(TYPES[kind])
    q, k = qkv[:, :heads[0]], qkv[:, heads[0]:heads[0] + heads[1]]
    freqs = base ** (-torch.arange(pairs, dtype=torch.float64, device=dev()) / max(pairs, 1))
    pos = torch.randint(0, 100000, (n,), device=dev(), generator=g, dtype=torch.int32) if positions is None else i32(positions)
    w = [0.5 + torch.rand(d, device=dev(), generator=g) if norm else None for _ in range(2)]
    want = [ref_rope(x, pos, freqs, y, 1e-6, interleaved, mscale) for x, y in zip((q, k), w)]
    rest = qkv[:, sum(heads):].clone()
    out = dict(q_out=q, k_out=k) if inplace else {}
    got = gdn.gdn_qk_rope(q, k, pos, freqs, q_weight=w[0], k_weight=w[1], interleaved=interleaved, mscale=mscale, **out)
    for x, (y, size) in zip(got, want):
        assert x.dtype is TYPES[kind] and x.shape == y.shape
        far = (x.double() - y).abs() - HALF[x.dtype] * y.abs() - 2.0 ** -19 * size
        assert far.max() <= 0 if n else True
    assert torch.equal(qkv[:, sum(heads):], rest)
    return got


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("pairs", [0, 1, 3, 8, 16, 27, 32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_layouts(kind, d, pairs, interleaved):
    check_rope(d=d, pairs=pairs, kind=kind, interleaved=interleaved, norm=pairs % 2 == 0)
    check_rope(d=d, pairs=d // 2 - pairs // 2, kind=kind, interleaved=interleaved, norm=pairs % 2 == 1, mscale=1.3)


@pytest.mark.parametrize("n,heads", [(0, (2, 1)), (1, (1, 1)), (1, (7, 3)), (2, (64, 8)), (33, (5, 5)), (700, (3, 1)), (3000, (8, 1))])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("inplace", [False, True])
def test_rope_sizes(n, heads, kind, inplace):
    check_rope(n=n, heads=heads, kind=kind, inplace=inplace)
    check_rope(n=n, heads=heads, kind=kind, d=256, pairs=13, norm=False, inplace=inplace)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_far_and_negative_positions(interleaved):
    check_rope(n=9, kind="f32", norm=False, interleaved=interleaved, base=1e6,
               positions=[0, 1, -1, 1000003, -1000003, 2 ** 24 + 1, 2 ** 30 + 1, 2 ** 31 - 1, -2 ** 31])


def test_rope_other_values_pass_and_stay_in_their_rows():
    x = torch.randn((3, 2, 64), device=dev()).to(torch.bfloat16)
    x[0, 0, 60], x[1, 1, 5], x[2, 0, 63] = INF, NAN, -INF
    freqs = 0.1 ** torch.arange(16, dtype=torch.float64, device=dev())
    q, k = gdn.gdn_qk_rope(x, x[:, :1], i32([3, 4, 5]), freqs)
    assert torch.equal(q[..., 32:].nan_to_num(7.0), x[..., 32:].nan_to_num(7.0)) and torch.equal(k.nan_to_num(7.0), q[:, :1].nan_to_num(7.0))
    bad = torch.zeros((3, 2, 64), dtype=torch.bool, device=dev())
    bad[1, 1, 5] = bad[1, 1, 21] = True
    assert torch.equal(q.isnan(), bad)


def test_rope_output_strides_and_no_heads():
    x = torch.randn((6, 4, 128), device=dev()).to(torch.bfloat16)
    freqs = 0.5 ** torch.arange(64, dtype=torch.float64, device=dev())
    pos = i32(list(range(6)))
    out = torch.zeros((4, 6, 136), device=dev(), dtype=torch.bfloat16)
    q, k = gdn.gdn_qk_rope(x, x[:, :0], pos, freqs, q_out=out[..., :128].transpose(0, 1))
    assert k.shape == (6, 0, 128) and not out[..., 128:].any()
    assert torch.equal(q, gdn.gdn_qk_rope(x[:, :0], x, pos, freqs)[1])


# ---- attention of new tokens -----------------------------------------------------------------------
class Case:
    """A cache with tables for requests of (cached, new) tokens; what no token of theirs uses is NaN."""

    def __init__(self, requests, heads=8, kv_heads=2, d=128, page=16, kind="bf16", head_major=False, window=0, behind=0, seed=0, q_scale=1.0, wide=0):
        g = gen(seed)
        self.requests, self.window, self.kind = requests, window, kind
        lengths = [c + n for c, n in requests]
        wide = max(max((-(-n // page) for n in lengths), default=0), wide, 1)
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + 3
        shape = (pages, kv_heads, page, d) if head_major else (pages, page, kv_heads, d)
        ids = torch.randperm(pages, device=dev(), generator=g).tolist()
        rows, at = [], 0
        live = torch.zeros((pages, page), dtype=torch.bool, device=dev())
        for n, m in zip(lengths, need):
            mine = ids[at:at + m]
            at += m
            rows.append(mine + [-1] * (wide - m))
            for i, p in enumerate(mine):
                live[p, :min(page, n - i * page)] = True
        self.table = i32(rows).view(len(requests), wide)

        def values():
            x = torch.randn(shape, device=dev(), generator=g)
            x = (x * 60).clamp(-448, 448).to(TYPES[kind]) if kind == "e4m3" else x.to(TYPES[kind])
            x = x.transpose(1, 2) if head_major else x
            x.view(torch.uint8).masked_fill_(~live[:, :, None, None], 0xFF if kind == "e4m3" else 0xFF)  # NaN in each type
            return x
        self.k, self.v = values(), values()
        self.scales = {}
        if kind == "e4m3":
            self.scales = {n: 0.01 + 0.01 * torch.rand(kv_heads, device=dev(), generator=g) for n in ("k_scale", "v_scale")}
        cu = [0]
        for _, n in requests:
            cu.append(cu[-1] + n)
        self.cu, self.lens = i32(cu), i32(lengths)
        self.qkind = torch.float32 if kind == "f32" else torch.bfloat16
        self.q = (q_scale * torch.randn((cu[-1] + behind, heads, d), device=dev(), generator=g)).to(self.qkind)

    def call(self, **kw):
        kw = {**dict(window=self.window, **self.scales), **kw}
        return gdn.gdn_paged_prefill(self.q, self.k, self.v, self.table, self.lens, self.cu, **kw)

    def ref(self, scale=None):
        """o, lse, and the bounds of both in 64 bits; rows of no request are NaN."""
        n, heads, d = self.q.shape
        kv_heads, page = self.k.shape[2], self.k.shape[1]
        group = heads // kv_heads
        scale = d ** -0.5 if scale is None else scale
        o = torch.full((n, heads, d), NAN, dtype=torch.float64, device=dev())
        lse, o_far, lse_far = torch.full((n, heads), NAN, dtype=torch.float64, device=dev()), o.clone(), torch.zeros((n, heads), dtype=torch.float64, device=dev())
        cu, lens, table = self.cu.tolist(), self.lens.tolist(), self.table.long()
        w = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11, "f32": 2.0 ** -22}[self.kind]
        for b in range(len(lens)):
            rows = range(cu[b], cu[b + 1])
            if not rows:
                continue
            room = table.shape[1] * page
            j = torch.arange(max(0, min(lens[b], room)), device=dev())
            at = table[b, j // page]
            ok = (at >= 0) & (at < self.k.shape[0])
            at, cell = torch.where(ok, at, 0), j % page
            x = self.q[cu[b]:cu[b + 1]].double()
            pos = torch.arange(cu[b], cu[b + 1], device=dev()) - cu[b + 1] + lens[b]
            seen = ok & (j <= pos[:, None])
            if self.window:
                seen &= j > pos[:, None] - self.window
            for h in range(kv_heads):
                mine = slice(h * group, (h + 1) * group)
                k, v = (c.view(torch.uint8)[at, cell, h].view(c.dtype).double() if self.kind == "e4m3" else c[at, cell, h].double() for c in (self.k, self.v))
                if self.scales:
                    k, v = k * self.scales["k_scale"][h].double(), v * self.scales["v_scale"][h].double()
                k, v = k.masked_fill(~ok[:, None], 0), v.masked_fill(~ok[:, None], 0)
                s = torch.einsum("ngd,ld->ngl", x[:, mine], k) * scale
                size = torch.einsum("ngd,ld->ngl", x[:, mine].abs(), k.abs()) * abs(scale)
                s = s.masked_fill(~seen[:, None], -INF)
                top = s.amax(-1, keepdim=True) if len(j) else torch.full(s.shape[:2] + (1,), -INF, dtype=torch.float64, device=dev())
                top = torch.where(top == -INF, 0.0, top)
                p = torch.exp(s - top)
                z = p.sum(-1, keepdim=True)
                # weights that are exactly 0 do not read
                read = seen[:, None].expand_as(p)
                pv = torch.where(read[..., None], p[..., None] * v, 0.0).sum(2) if not v.isfinite().all() else torch.einsum("ngl,ld->ngd", p, v)
                o[cu[b]:cu[b + 1], mine] = torch.where(z == 0, 0.0, pv / z)
                lse[cu[b]:cu[b + 1], mine] = (top + torch.log(z))[..., 0]
                size = torch.where(seen[:, None], size, 0.0).amax(-1) if len(j) else torch.zeros(s.shape[:2], dtype=torch.float64, device=dev())
                delta = d * 2.0 ** -23 * size
                pav = torch.einsum("ngl,ld->ngd", p / torch.where(z == 0, 1.0, z), v.abs().nan_to_num(0, 0))
                length = len(j)
                far = HALF[self.qkind] * o[cu[b]:cu[b + 1], mine].abs() + (w + 2 * delta[..., None] + 2.0 ** -20 + length * 2.0 ** -23) * pav
                o_far[cu[b]:cu[b + 1], mine] = far + 2.0 ** -32 * (v.abs().nan_to_num(0, 0).sum(0) if length else 0.0)
                lse_far[cu[b]:cu[b + 1], mine] = delta + 2.0 ** -20 * (1 + lse[cu[b]:cu[b + 1], mine].abs()) + length * 2.0 ** -23
        return o, lse, o_far, lse_far

    def check(self, scale=None, **kw):
        o, lse, o_far, lse_far = self.ref(scale)
        if scale is not None:
            kw["scale"] = scale
        got, got_lse = self.call(**kw)
        real = slice(0, int(self.cu[-1]))
        same(got[real].double(), o[real], o_far[real])
        same(got_lse[real].double(), lse[real], lse_far[real])
        return got, got_lse


def same(x, y, far):
    fine = y.isfinite()
    assert (x.isfinite() == fine).all()
    assert torch.equal(x.isneginf() | x.isposinf() | x.isnan(), ~fine)
    inf = y.isinf() & (y < 0)
    assert (x[inf] == y[inf]).all()
    off = (x - y).abs()[fine] - far[fine]
    assert off.numel() == 0 or off.max() <= 0, f"off by {(x - y).abs()[fine].max()}"


KINDS = ["bf16", "e4m3", "f32"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("requests", [[(0, 1)], [(0, 37)], [(5, 300)], [(127, 1)], [(128, 1), (0, 129), (640, 17), (3, 0), (255, 257)]])
def test_attend_sizes(kind, d, requests):
    Case(requests, kind=kind, d=d).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (4, 2), (10, 2), (12, 1), (16, 1), (48, 2), (33, 1)])
def test_attend_groups(kind, heads, kv_heads):
    Case([(70, 61), (0, 9)], heads=heads, kv_heads=kv_heads, kind=kind, d=64).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page,head_major", [(1, False), (1, True), (7, False), (16, True), (24, False), (48, True), (64, False), (100, False), (128, True), (512, False)])
def test_attend_pages(kind, page, head_major):
    Case([(190, 75), (33, 1)], page=page, head_major=head_major, kind=kind).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 1000])
def test_attend_windows(kind, window):
    Case([(300, 140), (0, 200), (500, 1)], window=window, kind=kind, heads=6).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_rows_cut_over_long_contexts(kind, d):
    # few rows, so that their keys are shared by many CTAs
    Case([(20000, 3)], heads=4, kv_heads=1, kind=kind, d=d, page=64).check()
    Case([(5000, 100), (30, 20), (0, 700), (9000, 1)], heads=8, kv_heads=2, kind=kind, d=d, page=32).check()
    Case([(7000, 40)], heads=8, kv_heads=4, kind=kind, d=d, window=3000).check()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_many_requests(kind):
    r = torch.Generator().manual_seed(3)
    sizes = torch.randint(0, 40, (1500, 2), generator=r).tolist()
    Case([(c, n if i % 3 else 1) for i, (c, n) in enumerate(sizes)], kind=kind, d=64, page=8, heads=4, kv_heads=1).check()
    Case([(c, 1) for c, _ in sizes[:300]], kind=kind, d=128, page=8, heads=4, kv_heads=2).check()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_whole_prompt(kind):
    Case([(0, 2500)], kind=kind, heads=4, kv_heads=2, page=64).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_scale", [0.0, 8.0, 60.0])
def test_attend_scores_from_flat_to_steep(kind, q_scale):
    Case([(900, 50)], kind=kind, q_scale=q_scale, d=64).check()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_scores_that_rise_along_the_row(kind):
    # every tile has a new maximum, far above the last one's
    c = Case([(1500, 40)], kind=kind, d=64, heads=2, kv_heads=1, page=1)
    order = c.table[0, :1540].long()
    ramp = torch.linspace(0.01, 1, 1540, device=dev())[:, None, None]
    x = torch.ones((1, 1, 64), device=dev()) * ramp * (400 if kind == "e4m3" else 6)
    c.k.view(torch.uint8 if kind == "e4m3" else c.k.dtype)[order] = x.expand(1540, 1, 64)[:, None].to(c.k.dtype).view(torch.uint8 if kind == "e4m3" else c.k.dtype)
    c.q.fill_(4.0)
    c.check()
    c.q.fill_(-4.0)
    c.check()


def test_attend_other_scale_and_no_lse_of_empty_rows():
    Case([(100, 30)]).check(scale=0.5)
    Case([(100, 30)]).check(scale=-0.25)
    Case([(100, 30)]).check(scale=0.0)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_rows_behind_the_last_request_stay(kind):
    c = Case([(40, 20), (0, 0), (7, 1)], kind=kind, behind=13)
    o = torch.full_like(c.q, 5.0)
    lse = torch.full(c.q.shape[:2], 6.0, device=dev())
    got, got_lse = c.check(o=o, lse=lse)
    assert got is o and got_lse is lse
    assert (o[21:] == 5).all() and (lse[21:] == 6).all()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_rows_before_the_first_request_stay(kind):
    c = Case([(40, 20), (3, 4)], kind=kind, behind=10)
    c.cu += 5  # rows 0 to 4 are nobody's
    o, lse = torch.full_like(c.q, 5.0), torch.full(c.q.shape[:2], 6.0, device=dev())
    want, want_lse, o_far, lse_far = c.ref()
    c.call(o=o, lse=lse)
    same(o[5:29].double(), want[5:29], o_far[5:29])
    assert (o[:5] == 5).all() and (o[29:] == 5).all() and (lse[:5] == 6).all() and (lse[29:] == 6).all()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_tables_with_holes(kind):
    c = Case([(300, 150), (40, 30)], kind=kind)
    c.table[0, 3] = -1
    c.table[0, 10:20] = 2 ** 31 - 1
    c.table[1, 0] = c.k.shape[0]
    c.table[0, 27] = -2 ** 31
    c.check()
    c.table.fill_(-1)
    o, lse = c.check()
    assert not o.any() and (lse == -INF).all()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_lengths_that_do_not_fit(kind):
    c = Case([(300, 150), (40, 30), (0, 20)], kind=kind)
    c.lens[1] = 10   # fewer tokens than rows: the first 20 rows have no position
    c.lens[2] = -5
    c.check()
    c.lens[0] = 10 ** 6  # the table ends before
    c.table[0, -1] = -1
    n, page = c.table.shape[1], 16
    o, lse = c.call()
    short = Case([(300, 150), (40, 30), (0, 20)], kind=kind)
    short.table, short.lens, short.k, short.v, short.q = c.table, c.lens.clone(), c.k, c.v, c.q
    want, want_lse, o_far, lse_far = short.ref()
    same(o.double(), want, o_far)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_without_cache_or_rows(kind):
    c = Case([(30, 20)], kind=kind)
    o, lse = gdn.gdn_paged_prefill(c.q, c.k[:0], c.v[:0], c.table, c.lens, c.cu, **c.scales)
    assert not o.any() and (lse == -INF).all()
    o, lse = gdn.gdn_paged_prefill(c.q, c.k, c.v, c.table[:, :0], c.lens, c.cu, **c.scales)
    assert not o.any() and (lse == -INF).all()
    o, lse = gdn.gdn_paged_prefill(c.q[:0], c.k, c.v, c.table, c.lens, c.cu, **c.scales)
    assert o.shape[0] == 0
    o, lse = gdn.gdn_paged_prefill(c.q[:0], c.k, c.v, c.table[:0], c.lens[:0], c.cu[:1], **c.scales)
    assert o.shape[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("which", ["k", "v"])
def test_attend_non_finite_values_reach_later_rows_only(kind, d, bad, which):
    if kind == "e4m3" and bad != bad:
        pass
    elif kind == "e4m3":
        pytest.skip("the format has no infinity")
    c = Case([(0, 700), (60, 50)], kind=kind, d=d, heads=4, kv_heads=2, page=16)
    t = {"k": c.k, "v": c.v}[which]
    want, _, far, _ = c.ref()
    j, dim = 413, 17
    cell = t[int(c.table[0, j // 16]), j % 16, 1]
    if kind == "e4m3":
        cell.view(torch.uint8)[dim] = 0x7F
    else:
        cell[dim] = bad
    o, lse = c.call()
    before = torch.ones(750, dtype=torch.bool, device=dev())
    before[413:700] = False
    # a tile with such a value sums its products in another order, as any order inside the bounds
    fine = (o.double() - want).abs() <= far
    assert fine[before].all() and fine[:, :2].all()
    hit = ~o[413:700, 2:].isfinite()
    if which == "v":
        assert hit[..., dim].all() and hit.sum() == hit[..., dim].numel()
        assert lse.isfinite().all()
    elif bad != bad or kind == "e4m3":
        assert hit.all() and lse[413:700, 2:].isnan().all()
    else:
        assert (hit.all(-1) | ~hit.any(-1)).all() and hit.any()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_non_finite_values_in_a_window(kind):
    c = Case([(200, 400)], kind=kind, heads=4, kv_heads=1, window=150, page=16, d=64)
    want, _, far, _ = c.ref()
    for j in (50, 255, 256, 400):
        c.v[int(c.table[0, j // 16]), j % 16, 0].view(torch.uint8 if kind == "e4m3" else c.v.dtype)[9] = 0x7F if kind == "e4m3" else NAN
    o, _ = c.call()
    pos = torch.arange(200, 600, device=dev())
    hit = torch.zeros(400, dtype=torch.bool, device=dev())
    for j in (50, 255, 256, 400):
        hit |= (pos >= j) & (pos < j + 150)
    assert (o[..., 9].isnan().all(1) == hit).all()
    fine = (o.double() - want).abs() <= far
    rest = [i for i in range(64) if i != 9]
    assert fine[~hit].all() and fine[..., rest].all()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_non_finite_queries_stay_in_their_rows(kind):
    c = Case([(500, 100)], kind=kind, heads=4, kv_heads=1, d=64)
    clean, clean_lse = c.call()
    c.q[40, 2, 3], c.q[77, 0, 0] = NAN, INF
    o, lse = c.call()
    hit = torch.zeros((100, 4), dtype=torch.bool, device=dev())
    hit[40, 2] = hit[77, 0] = True
    assert (o[~hit] == clean[~hit]).all() and (lse[~hit] == clean_lse[~hit]).all()
    assert not o[hit].isfinite().any() and not lse[hit].isfinite().any()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_strides(kind):
    c = Case([(100, 60), (9, 5)], kind=kind, d=64, heads=4, kv_heads=2)
    want, want_lse = c.check()
    n = c.q.shape[0]
    big = torch.zeros((n, 9, 64), dtype=c.qkind, device=dev())
    big[:, 2:6] = c.q
    c.q = big[:, 2:6]
    wide = torch.full((2, c.table.shape[1] + 5), -1, dtype=torch.int32, device=dev())
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide[:, :c.table.shape[1]]
    pages = c.k.shape[0]

    def apart(x):
        far = torch.zeros((2, pages + 1, 20, 192), dtype=x.dtype, device=dev())
        y = far[:, :pages, :16, 64:128].permute(1, 2, 0, 3)
        y.view(torch.uint8).copy_(x.view(torch.uint8)) if kind == "e4m3" else y.copy_(x)
        return y
    c.k, c.v = apart(c.k), apart(c.v)
    got, got_lse = c.call()
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


def test_attend_shared_table_row():
    c = Case([(64, 32)], heads=4, kv_heads=2)
    want, want_lse, o_far, lse_far = c.ref()
    # the chunk as two requests of one sequence
    o, lse = gdn.gdn_paged_prefill(c.q, c.k, c.v, c.table.expand(2, -1), i32([80, 96]), i32([0, 16, 32]))
    same(o.double(), want, o_far)
    same(lse.double(), lse.double(), lse_far)


def test_attend_offsets_past_32_bits():
    # pages far apart: element offsets beyond 2^32
    d, page, pages = 128, 16, 6
    far = torch.empty((pages, 2 ** 30), dtype=torch.bfloat16, device=dev())
    k, v = (far.as_strided((pages, page, 1, d), (2 ** 30, d, d, 1), s) for s in (0, 2 ** 29))
    c = Case([(60, 30)], heads=4, kv_heads=1, page=page)
    c.table = i32([[5, 4, 3, 2, 1, 0]])
    for x in (k, v):
        x.copy_(torch.randn((pages, page, 1, d), device=dev()))
    c.k, c.v = k, v
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_same_bits_again(kind):
    c = Case([(3000, 200), (100, 1), (5, 90)], kind=kind, heads=8, kv_heads=2)
    o, lse = c.call()
    for _ in range(3):
        again, again_lse = c.call()
        assert torch.equal(o, again) and torch.equal(lse, again_lse)


def test_attend_status_and_workspace():
    c = Case([(100, 30)])
    ws = gdn.Workspace()
    c.check(workspace=ws)
    assert gdn.gdn_paged_prefill_status(ws) == 0
    need = gdn.load().gdn_paged_prefill_workspace_bytes(gdn.prompt._cache(c.k, c.v, None, None, 0), 1, 30, 8)
    with pytest.raises(gdn.GdnError) as e:
        c.call(workspace=ws.buf[:need // 512 * 256])
    assert e.value.status == 5
    ws.buf.fill_(0xFF)  # what a workspace holds before does not matter
    c.check(workspace=ws)
    assert gdn.gdn_paged_prefill_status(ws) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_attend_captured_and_replayed_with_other_lengths(kind):
    c = Case([(500, 64), (30, 64), (900, 1)], kind=kind, heads=8, kv_heads=2)
    ws = [gdn.Workspace() for _ in range(2)]
    o, lse = torch.zeros_like(c.q), torch.zeros(c.q.shape[:2], device=dev())
    o2, lse2 = o.clone(), lse.clone()
    for w in ws:
        c.call(workspace=w)
    torch.cuda.synchronize()
    graphs = []
    for w, x, y in ((ws[0], o, lse), (ws[1], o2, lse2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(o=x, lse=y, workspace=w)
        graphs.append(g)
    for lens, cu in (([564, 94, 901], [0, 64, 128, 129]), ([70, 40, 555], [0, 1, 41, 129]), ([9, 0, 0], [0, 9, 9, 9])):
        c.lens.copy_(i32(lens))
        c.cu.copy_(i32(cu))
        streams = [torch.cuda.Stream() for _ in graphs]
        o.fill_(3), o2.fill_(3)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):  # both at once, each in its workspace
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        want, want_lse, o_far, lse_far = c.ref()
        real = slice(0, cu[-1])
        same(o[real].double(), want[real], o_far[real])
        same(lse[real].double(), want_lse[real], lse_far[real])
        assert torch.equal(o, o2) and (o[cu[-1]:] == 3).all()


def test_calls_on_another_stream():
    s = torch.cuda.Stream()
    c = Case([(500, 64)])
    x = torch.randn((8, 5000), device=dev())
    tok, pos, freqs = i32(list(range(8))), i32(list(range(64))), torch.ones(64, dtype=torch.float64, device=dev())
    want = [*c.call(), *gdn.gdn_logprobs(x, tok, top=3), *gdn.gdn_qk_rope(c.q, c.q, pos, freqs)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [*c.call(stream=s), *gdn.gdn_logprobs(x, tok, top=3, stream=s), *gdn.gdn_qk_rope(c.q, c.q, pos, freqs, stream=s)]
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- log probabilities ---------------------------------------------------------------------------
def check_logprobs(x, tokens, top):
    B, V = x.shape
    got, entropy, top_tokens, top_logprobs = gdn.gdn_logprobs(x, i32(tokens), top=top)
    y = x.double()
    m = y.amax(1, keepdim=True)
    none = m[:, 0] == -INF
    y = torch.where(none[:, None], 0.0, y - m)
    logp = y - torch.log(torch.exp(y).sum(1, keepdim=True))
    logp[none] = -INF
    p = torch.exp(logp)
    want_entropy = torch.where(none, 0.0, -torch.where(p == 0, 0.0, p * logp).sum(1))
    tok = torch.tensor(tokens, device=dev())
    inside = (tok >= 0) & (tok < V)
    want = torch.where(inside, logp[torch.arange(B, device=dev()), tok.clamp(0, V - 1)], 0.0)
    near(got, want)
    near(entropy, want_entropy, 8.0)
    order = torch.sort(x.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(top_tokens.long(), order)
    near(top_logprobs, torch.gather(logp, 1, order))


def near(x, y, more=0.0):
    x = x.double()
    inf = y == -INF
    assert torch.equal(x == -INF, inf)
    assert ((x - y).abs()[~inf] <= 2.0 ** -17 * (1 + more + y.abs()[~inf])).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 33, 1000, 4096, 8191, 100003])
@pytest.mark.parametrize("B", [1, 3, 37])
def test_logprobs_sizes(kind, V, B):
    x = (torch.randn((B, V), device=dev(), generator=gen(V + B)) * 3).to(TYPES[kind])
    tokens = [(i * 7919) % (V + 2) - 1 for i in range(B)]
    for top in {0, 1, min(5, V), min(32, V)}:
        check_logprobs(x, tokens, top)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_logprobs_many_rows(kind):
    x = (torch.randn((1500, 5003), device=dev(), generator=gen(1)) * 4).to(TYPES[kind])
    check_logprobs(x, [i % 5003 for i in range(1500)], 20)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1, 3, 5])
def test_logprobs_rows_of_any_alignment(kind, offset):
    x = (torch.randn((5, 9001), device=dev(), generator=gen(offset)) * 3).to(TYPES[kind])
    check_logprobs(x[:, offset:offset + 8000], [0, 1, 7999, 8000, -1], 7)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 20000, 140001])
@pytest.mark.parametrize("shape", ["equal", "two", "rising", "falling", "zeros", "late"])
def test_logprobs_ties_and_orders(kind, V, shape):
    i = torch.arange(V, device=dev())
    x = {"equal": torch.full((V,), 1.5, device=dev()), "two": (i % 3 == 1).float(), "rising": i / V * 30, "falling": -i / V * 30,
         "zeros": torch.where(i % 2 == 0, -0.0, 0.0), "late": torch.where(i > V - 60, 5.0, -i / V)}[shape]
    check_logprobs(x.to(TYPES[kind]).expand(3, V).contiguous(), [0, V - 1, V // 2], 32)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 70001])
def test_logprobs_masked_rows(kind, V):
    x = (torch.randn((4, V), device=dev(), generator=gen(V)) * 3).to(TYPES[kind])
    x[0, 5:] = -INF
    x[1] = -INF
    x[2, ::2] = torch.finfo(x.dtype).min
    x[3, 1:] = -INF
    check_logprobs(x, [3, 3, 4, 0], 10)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 70001])
def test_logprobs_non_finite_rows(kind, V):
    x = torch.randn((4, V), device=dev(), generator=gen(V)).to(TYPES[kind])
    x[1, 7], x[2, V - 3] = NAN, INF
    x[2, 4] = INF
    got, entropy, top_tokens, top_logprobs = gdn.gdn_logprobs(x, i32([1, 1, 1, -1]), top=4)
    bad = torch.tensor([False, True, True, False], device=dev())
    assert torch.equal(got.isnan(), bad) and torch.equal(entropy.isnan(), bad) and torch.equal(top_logprobs.isnan().all(1), bad)
    assert got[3] == 0 and top_tokens[2, :2].tolist() == [4, V - 3]
    order = torch.sort(torch.where(x.isnan(), -INF, x.float()), dim=1, descending=True, stable=True).indices[:, :4]
    assert torch.equal(top_tokens.long(), order)
    y = torch.full((1, 6), NAN, device=dev(), dtype=x.dtype)
    y[0, 3], y[0, 4] = -INF, 1.0
    assert gdn.gdn_logprobs(y, i32([0]), top=6)[2].tolist() == [[4, 3, 0, 1, 2, 5]]


def test_logprobs_same_bits_and_graph():
    x = torch.randn((9, 50021), device=dev(), generator=gen(5)) * 3
    tok = i32(list(range(9)))
    want = gdn.gdn_logprobs(x, tok, top=9)
    out = dict(logprobs=want[0].clone(), entropy=want[1].clone(), top_tokens=want[2].clone(), top_logprobs=want[3].clone())
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        gdn.gdn_logprobs(x, tok, top=9, **out)
    for t in out.values():
        t.zero_()
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(out.values(), want))


# ---- the operators in a row -----------------------------------------------------------------------
@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_a_prompt_in_chunks_is_the_prompt_at_once(cache):
    """Rotate, append, attend, score: in chunks of any size the last layer's log probabilities are those of one chunk."""
    kind, B, heads, kv_heads, d, page, V = TYPES[cache], 3, 4, 2, 64, 16, 500
    g = gen(11)
    lens = [150, 33, 97]
    x = [torch.randn((n, heads + 2 * kv_heads, d), device=dev(), generator=g).to(kind) for n in lens]
    head = (torch.randn((heads * d, V), device=dev(), generator=g) / 8).to(kind)
    freqs = 1e4 ** (-torch.arange(d // 2, dtype=torch.float64, device=dev()) / (d // 2))
    w = 0.5 + torch.rand(d, device=dev(), generator=g)
    tokens = [torch.randint(0, V, (n,), device=dev(), generator=g, dtype=torch.int32) for n in lens]

    def go(chunk):
        pages = sum(-(-n // page) for n in lens)
        k_cache, v_cache = (torch.full((pages, page, kv_heads, d), NAN, dtype=kind, device=dev()) for _ in range(2))
        table, free = torch.full((B, 10), -1, dtype=torch.int32, device=dev()), torch.arange(pages, dtype=torch.int32, device=dev())
        done, taken, got = [0] * B, 0, [[] for _ in range(B)]
        while any(a < n for a, n in zip(done, lens)):
            add = [min(chunk, n - a) for a, n in zip(done, lens)]
            qkv = torch.cat([y[a:a + m] for y, a, m in zip(x, done, add)])
            slots, pos, seq, cu, counts = gdn.gdn_page_tables(i32(add), free[taken:], table, page=page, cached_lens=i32(done), n_slots=sum(add))
            taken += int(counts[1])
            q, k = gdn.gdn_qk_rope(qkv[:, :heads], qkv[:, heads:heads + kv_heads], pos, freqs, q_weight=w, k_weight=w)
            gdn.gdn_kv_append(k, qkv[:, heads + kv_heads:], slots, k_cache, v_cache)
            o, _ = gdn.gdn_paged_prefill(q, k_cache, v_cache, table, seq, cu)
            logits = o.reshape(len(o), -1) @ head
            lp = gdn.gdn_logprobs(logits, torch.cat([t[a:a + m] for t, a, m in zip(tokens, done, add)]))[0]
            for b, part in enumerate(lp.split(add)):
                got[b].append(part)
            done = [a + m for a, m in zip(done, add)]
        return torch.cat([torch.cat(y) for y in got])
    whole = go(1000)
    # attention's outputs differ by their rounding at most twice; a logit sums 256 products with weights of 1/8
    tol = {"bf16": 0.1, "f32": 1e-4}[cache]
    for chunk in (1, 16, 41):
        assert (go(chunk) - whole).abs().max() <= tol
