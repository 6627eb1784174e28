"""What a program meets around the prompt chunk's calls: the status of calls without rows, outputs that share memory, the end of
fp32's range, lists of requests in any order, waits that run out.  References and tolerances are those of test_gpu_prompt.py."""
import copy
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import gated_delta_rule_16_gb300 as gdn
from test_gpu_prompt import INF, KINDS, Case, _built, dev, i32, same  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("used", [False, True])
def test_status_after_a_call_without_rows(kind, used):
    c = Case([(30, 20)], kind=kind)
    ws = gdn.Workspace()
    if used:
        c.call(workspace=ws)
    else:
        ws.buf = torch.empty(1 << 26, dtype=torch.uint8, device=c.q.device)
    for q, table, lens, cu in ((c.q[:0], c.table, c.lens, i32([0, 0])), (c.q[:0], c.table[:0], c.lens[:0], i32([0])),
                               (c.q, c.table[:0], c.lens[:0], i32([0]))):
        ws.buf.fill_(0xFF)  # what memory held before, or an earlier call's status
        gdn.gdn_paged_prefill(q, c.k, c.v, table, lens, cu, workspace=ws, **c.scales)
        assert gdn.gdn_paged_prefill_status(ws) == 0
        assert (ws.buf[4:] == 0xFF).all()
    c.check(workspace=ws)
    assert gdn.gdn_paged_prefill_status(ws) == 0


# ---- outputs that share memory -------------------------------------------------------------------
def refused(fn, *tensors):
    """The call is GDN_ERR_UNSUPPORTED and writes nothing."""
    before = [t.clone() for t in tensors]
    with pytest.raises(gdn.GdnError) as e:
        fn()
    assert e.value.status == 6
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(tensors, before))


def test_rope_outputs_that_share_memory():
    n, d = 40, 128
    buf = torch.randn((n + 2, 16, d), device=dev()).bfloat16()
    q, k = buf[:n, :8], buf[:n, 8:10]
    pos, freqs = i32(list(range(n))), 0.5 ** torch.arange(64, dtype=torch.float64, device=dev())
    go = lambda q_out=None, k_out=None, q=q, k=k: gdn.gdn_qk_rope(q, k, pos, freqs, q_out=q_out, k_out=k_out)
    want = go()
    refused(lambda: go(buf[1:n + 1, :8]), buf)            # q, a token on
    refused(lambda: go(buf[:n, 1:9]), buf)                # a head on
    refused(lambda: go(buf[:n, 3:11]), buf)               # over some of q and of k
    refused(lambda: go(buf[:n, 9:].as_strided((n, 8, d), (16 * d, d - 64, 1))), buf)  # heads over one another, and k
    refused(lambda: go(k_out=buf[:n, 7:9]), buf)
    refused(lambda: go(buf[:n, :8], q=buf[:n, :8], k=buf[:n, 4:6]), buf)   # in place over what k is
    refused(lambda: go(buf[:n, :2], buf[:n, 8:10], q=k, k=q[:, :2]), buf)  # each over the other
    refused(lambda: go(buf[:n, 10:11].expand(n, 8, d)), buf)  # every head to one place
    refused(lambda: go(buf[:1, 10:].as_strided((n, 6, d), (0, d, 1)), q=q[:, :6]), buf)
    out = torch.zeros((n, 9, d), dtype=torch.bfloat16, device=dev())
    refused(lambda: go(out[:, :8], out[:, 7:9]), out)
    # what shares no byte: slices of the projection itself, and one buffer for both outputs
    got = go(buf[:n, 10:16], q=q[:, :6])
    assert torch.equal(got[0], want[0][:, :6]) and torch.equal(got[1], want[1])
    wide = torch.zeros((n, 10, d), dtype=torch.bfloat16, device=dev())
    got = go(wide[:, :8], wide[:, 8:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    major = torch.zeros((10, n, d), dtype=torch.bfloat16, device=dev()).transpose(0, 1)
    got = go(major[:, :8], major[:, 8:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = go(q, k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("kind", KINDS)
def test_attend_outputs_that_share_memory(kind):
    c = Case([(300, 50), (9, 30)], kind=kind, heads=8, kv_heads=2)
    n, heads, d = c.q.shape
    want, want_lse = c.check()
    buf = torch.zeros((n + 3, heads, d), dtype=c.qkind, device=dev())
    buf[:n] = c.q
    at = lambda x, shape: x.reshape(-1)[:shape.numel()].view(shape)
    q, c.q = c.q, buf[:n]
    refused(lambda: c.call(o=buf[1:n + 1]), buf)
    refused(lambda: c.call(lse=at(buf.view(torch.float32), want_lse.shape)), buf)
    if kind == "bf16":
        refused(lambda: c.call(o=at(c.k, q.shape)), c.k)
        refused(lambda: c.call(o=at(c.v, q.shape)), c.v)
    o = torch.zeros(2 * q.numel(), dtype=c.qkind, device=dev())
    refused(lambda: c.call(o=at(o, q.shape), lse=at(o.view(torch.float32)[8:], want_lse.shape)), o)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=dev())
    refused(lambda: c.call(o=at(ws.view(c.qkind), q.shape), workspace=ws), ws)
    wide = torch.zeros((n, heads + 3, d), dtype=c.qkind, device=dev())
    wide[:, :heads] = q
    c.q = wide[:, :heads]
    refused(lambda: c.call(o=wide.view(-1)[:q.numel()].view(q.shape)), wide)
    # in place, where the layouts are one; rows that are cut and joined too
    c.q = buf[:n]
    got, got_lse = c.call(o=buf[:n])
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse) and not buf[n:].any()
    long = Case([(9000, 3), (0, 700)], kind=kind, heads=4, kv_heads=1, page=64)
    want, want_lse = long.call()
    got, got_lse = long.call(o=long.q)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


# ---- the end of fp32's range ---------------------------------------------------------------------
@pytest.mark.parametrize("call", ["decode", "prefill"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sign", [1, -1])
def test_fp32_magnitudes_count_as_infinite_from_the_documented_one_on(call, d, sign):
    # 2^128 - 2^116 is what rounds to infinity in the 11 bits of a high tf32 term; the number before it does not
    border = torch.tensor(0x7f7ff000, dtype=torch.int32).view(torch.float32).double().item()
    assert border == 2.0 ** 128 - 2.0 ** 116
    for bits, finite in ((0x7f7fefff, True), (0x7f7ff000, False), (0x7f7ff7ff, False), (0x7f7fffff, False)):
        c = Case([(0, 1)], kind="f32", heads=2, kv_heads=1, d=d)
        x = sign * torch.tensor(bits, dtype=torch.int32).view(torch.float32).item()
        at = int(c.table[0, 0]), 0, 0
        c.v[at][5] = x
        go = lambda: gdn.gdn_paged_decode(c.q, c.k, c.v, c.table, c.lens) if call == "decode" else c.call()
        o, lse = go()
        assert bool(o[..., 5].isfinite().all()) == finite and lse.isfinite().all()
        if finite:
            # one token has a weight of 1: two terms of 11 bits each, and one rounding
            assert ((o[0, :, 5].double() / x - 1).abs() <= 2.0 ** -22 + 2.0 ** -24).all()
        c.v[at][5] = 1.0
        c.k[at][3], c.q[..., 3] = x, 2.0 ** -120
        o, lse = go()
        assert bool(lse.isfinite().all()) == finite


# ---- lists of requests ---------------------------------------------------------------------------
class Guarded:
    """o and lse inside larger buffers of 7."""

    def __init__(self, c, rows=40):
        n, heads, d = c.q.shape
        self.rows, self.all_o = rows, torch.full((n + 2 * rows, heads, d), 7.0, dtype=c.qkind, device=dev())
        self.all_lse = torch.full((n + 2 * rows, heads), 7.0, device=dev())
        self.o, self.lse = self.all_o[rows:rows + n], self.all_lse[rows:rows + n]

    def untouched(self):
        return all((x[:self.rows] == 7).all() and (x[-self.rows:] == 7).all() for x in (self.all_o, self.all_lse))


def alone(c, b, lo, hi):
    """(o, lse and their bounds) of the rows [lo, hi) that request b names, as if it were the only one."""
    x = copy.copy(c)
    x.table, x.cu = c.table[b:b + 1], i32([lo, hi])
    x.lens = i32([max(0, int(c.lens[b])) - int(c.cu[b + 1]) + hi])
    return x.ref()


LISTS = [[0, 20, 15, 50], [60, 10, 2 ** 31 - 1, 5], [-7, 1000, 0, 95], [0, 100, 100, 100], [100, 0, 100, 0], [30, 30, 30, 30], [90, 100, 0, 20],
         [5, 5, -2 ** 31, 2 ** 31 - 1]]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cu", LISTS)
@pytest.mark.parametrize("repeat", [1, 5])
def test_attend_lists_of_requests_in_no_order(kind, cu, repeat):
    c = Case([(50, 20), (30, 40), (0, 30)], kind=kind, heads=4, kv_heads=2, behind=10)
    n = c.q.shape[0]
    cu = cu + (cu[1:] if cu[0] == 0 else cu) * (repeat - 1)
    B = len(cu) - 1
    c.table, c.lens = c.table.repeat(-(-B // 3), 1)[:B].contiguous(), c.lens.repeat(-(-B // 3))[:B].contiguous()
    c.cu = i32(cu)
    ws, out = gdn.Workspace(), Guarded(c)
    c.call(o=out.o, lse=out.lse, workspace=ws)
    assert gdn.gdn_paged_prefill_status(ws) == 0 and out.untouched()
    owners, fine_o, fine_lse = torch.zeros(n, dtype=torch.int64, device=dev()), (out.o == 7).clone(), (out.lse == 7).clone()
    stayed = fine_o.flatten(1).all(1) & fine_lse.all(1)
    close = lambda x, y, far: (x == y) | ((x - y).abs() <= far)
    for b in range(B):
        lo, hi = min(max(cu[b], 0), n), min(cu[b + 1], n)
        if hi <= lo:
            continue
        o, lse, o_far, lse_far = (x[lo:hi] for x in alone(c, b, lo, hi))
        owners[lo:hi] += 1
        fine_o[lo:hi] |= close(out.o[lo:hi].double(), o, o_far)
        fine_lse[lo:hi] |= close(out.lse[lo:hi].double(), lse, lse_far)
    assert stayed[owners == 0].all()                     # rows of no request
    assert fine_o.all() and fine_lse.all()               # every piece is that of a request that names the row
    if int(owners.sum()) <= n:
        assert not stayed[owners > 0].any()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_lse_of_requests_that_share_a_table_row(kind):
    c = Case([(64, 32)], heads=4, kv_heads=2, kind=kind)
    want, want_lse, o_far, lse_far = c.ref()
    o, lse = gdn.gdn_paged_prefill(c.q, c.k, c.v, c.table.expand(2, -1), i32([80, 96]), i32([0, 16, 32]), **c.scales)
    same(o.double(), want, o_far)
    same(lse.double(), want_lse, lse_far)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_lse_of_a_sequence_longer_than_its_table(kind):
    c = Case([(300, 150), (40, 30), (0, 20)], kind=kind)
    c.lens.copy_(i32([10 ** 6, 10, -5]))
    c.table[0, -1] = -1
    o, lse = c.check()
    assert (lse[150:170] == -INF).all() and (lse[180:] == -INF).all() and lse[:150].isfinite().all()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_lse_of_rows_behind_others_that_stay(kind):
    c = Case([(40, 20), (3, 4)], kind=kind, behind=10)
    c.cu += 5  # rows 0 to 4 are nobody's
    out = Guarded(c)
    want, want_lse, o_far, lse_far = c.ref()
    c.call(o=out.o, lse=out.lse)
    same(out.o[5:29].double(), want[5:29], o_far[5:29])
    same(out.lse[5:29].double(), want_lse[5:29], lse_far[5:29])
    assert out.untouched() and all((x[:5] == 7).all() and (x[29:] == 7).all() for x in (out.o, out.lse))


# ---- waits that run out --------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [64, 1])  # keys and values by TMA, and 16 bytes at a time
def test_attend_waits_that_run_out_are_reported(kind, d, page):
    c = Case([(500, 130), (0, 300), (40, 1), (40000, 20)], kind=kind, heads=8, kv_heads=2, d=d, page=page)
    ws, out = gdn.Workspace(), Guarded(c)
    want = c.call()
    assert gdn.gdn_paged_prefill_status() == 0
    for _ in range(3):
        gdn.gdn_selftest_paged_prefill_wait(5)
        try:
            c.call(o=out.o, lse=out.lse, workspace=ws)
            assert gdn.gdn_paged_prefill_status(ws) == 10
            c.call(o=out.o, lse=out.lse)
            assert gdn.gdn_paged_prefill_status() == 10
        finally:
            gdn.gdn_selftest_paged_prefill_wait()
        assert out.untouched()
        # the next call is as any other, in the same workspace
        got = c.check(workspace=ws)
        assert gdn.gdn_paged_prefill_status(ws) == 0 and all(torch.equal(x, y) for x, y in zip(got, want))
        got = c.check()
        assert gdn.gdn_paged_prefill_status() == 0 and all(torch.equal(x, y) for x, y in zip(got, want))


def test_attend_wait_limits_belong_to_a_thread():
    c = Case([(500, 130)])
    ws = gdn.Workspace()
    c.call(workspace=ws)
    with ThreadPoolExecutor(1) as pool:
        pool.submit(gdn.gdn_selftest_paged_prefill_wait, 5).result()
        c.check(workspace=ws)
        assert gdn.gdn_paged_prefill_status(ws) == 0
    f = Case([(500, 130)], kind="f32")  # whose kernel waits for no barrier in memory
    gdn.gdn_selftest_paged_prefill_wait(5)
    try:
        f.check(workspace=ws)
        assert gdn.gdn_paged_prefill_status(ws) == 0
    finally:
        gdn.gdn_selftest_paged_prefill_wait(0)
    short = Case([(0, 100)])  # whose keys come before copies stop
    gdn.gdn_selftest_paged_prefill_wait(2000)
    try:
        short.check(workspace=ws)
        assert gdn.gdn_paged_prefill_status(ws) == 0
    finally:
        gdn.gdn_selftest_paged_prefill_wait(0)
    for bad in (-1, 2001):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_selftest_paged_prefill_wait(bad)
