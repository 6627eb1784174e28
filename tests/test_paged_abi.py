"""The decode-step entry points over a paged cache: refusals of the C ABI and of the
binding.  No GPU: every call fails validation, so no pointer is dereferenced."""
import ctypes

import pytest
import torch

import gated_delta_rule_16_gb300 as gdn
from gated_delta_rule_16_gb300 import _binding as bnd

FAKE = 1 << 20
F = ctypes.c_void_p(FAKE)
OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED, DEVICE = 0, 1, 2, 3, 4, 5, 6, 8


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_16_gb300 import build
    build.build()
    return gdn.load()


def cache(dtype=bnd.GDN_BF16, **kw):
    x = dict(k=FAKE, v=FAKE, stride_page=16 * 8 * 128, stride_token=8 * 128, stride_head=128, k_scale=None, v_scale=None,
             pages=100, page=16, Hkv=8, d=128)
    if dtype == bnd.GDN_E4M3:
        x.update(k_scale=FAKE, v_scale=FAKE)
    x.update(kw)
    return bnd.GdnKvCache(x["k"], x["v"], x["stride_page"], x["stride_token"], x["stride_head"], x["k_scale"], x["v_scale"],
                          x["pages"], x["page"], x["Hkv"], x["d"], dtype)


BAD_CACHES = [
    (dict(d=96), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(Hkv=0), SHAPE), (dict(page=0), SHAPE), (dict(page=-4), SHAPE),
    (dict(pages=-1), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 2), ALIGN),
    (dict(stride_token=1023), ALIGN), (dict(stride_page=4), ALIGN), (dict(stride_head=-128), ALIGN), (dict(dtype=5), DTYPE),
    (dict(k_scale=FAKE), UNSUPPORTED), (dict(dtype=bnd.GDN_E4M3, v_scale=None), NULL),
    (dict(dtype=bnd.GDN_E4M3, k_scale=FAKE + 2), ALIGN), (dict(dtype=bnd.GDN_E4M3, stride_token=8), ALIGN),
]


def append(lib, c=None, n=4, dtype=0, k=FAKE, ks=(1024, 128), v=FAKE, vs=(1024, 128), slots=FAKE):
    return lib.gdn_kv_append(c or cache(), n, dtype, k, *ks, v, *vs, slots, None)


def decode(lib, c=None, B=2, Hq=16, dtype=0, q=FAKE, qs=(2048, 128), table=FAKE, ts=10, pages=10, lens=FAKE, window=0, o=FAKE, lse=FAKE,
           ws=FAKE, nbytes=1 << 40):
    return lib.gdn_paged_decode(c or cache(), B, Hq, dtype, q, *qs, table, ts, pages, lens, window, 0.1, o, lse, ws, nbytes, None)


def sample(lib, B=2, V=100, dtype=1, x=FAKE, xs=100, u=FAKE, us=100, t=None, k=None, p=None, m=None, tok=FAKE, lp=FAKE):
    return lib.gdn_sample(B, V, dtype, x, xs, u, us, t, k, p, m, tok, lp, None)


def tables(lib, B=2, page=16, wide=10, cached=None, new=FAKE, free=FAKE, n_free=5, table=FAKE, lens=FAKE, cu=FAKE, slots=FAKE, pos=FAKE, n=4,
           counts=FAKE):
    return lib.gdn_page_tables(B, page, wide, cached, new, free, n_free, table, lens, cu, slots, pos, n, counts, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_refusals(lib, kw, want):
    dtype = kw.get("dtype", bnd.GDN_BF16)
    c = cache(**kw)
    assert append(lib, c) == want
    assert decode(lib, c) == want


def test_append_refusals(lib):
    assert append(lib) == DEVICE                       # all arguments pass: stops at the device check here
    assert append(lib, n=-1) == SHAPE
    assert append(lib, n=0, k=None, v=None, slots=None) == OK
    assert append(lib, cache(pages=0, k=None, v=None)) == OK
    assert append(lib, dtype=1) == DTYPE               # fp32 rows into a bf16 cache
    assert append(lib, cache(bnd.GDN_E4M3), dtype=1) == DEVICE
    assert append(lib, cache(bnd.GDN_E4M3), dtype=2) == DTYPE
    assert append(lib, k=None) == NULL and append(lib, slots=None) == NULL
    assert append(lib, v=FAKE + 8) == ALIGN and append(lib, slots=FAKE + 4) == ALIGN
    assert append(lib, ks=(1024, 4)) == ALIGN and append(lib, vs=(1001, 128)) == ALIGN


def test_decode_refusals(lib):
    assert decode(lib) == DEVICE
    assert decode(lib, B=0, q=None, lens=None, o=None, ws=None) == OK
    assert decode(lib, lse=None) == DEVICE             # lse is optional
    assert decode(lib, ts=0) == DEVICE                 # all requests share one table row
    assert decode(lib, cache(pages=0, k=None, v=None), table=None) == DEVICE
    assert decode(lib, pages=0, table=None) == DEVICE
    for kw in (dict(B=-1), dict(Hq=0), dict(Hq=12), dict(pages=-1), dict(window=-1), dict(ts=-1), dict(B=1 << 30, Hq=1024)):
        assert decode(lib, **kw) == SHAPE, kw
    assert decode(lib, dtype=1) == DTYPE and decode(lib, cache(bnd.GDN_E4M3), dtype=2) == DTYPE
    for name in ("q", "table", "lens", "o", "ws"):
        assert decode(lib, **{name: None}) == NULL, name
    for kw in (dict(q=FAKE + 8), dict(o=FAKE + 4), dict(qs=(2047, 128)), dict(table=FAKE + 2), dict(lens=FAKE + 1), dict(lse=FAKE + 2),
               dict(ws=FAKE + 64)):
        assert decode(lib, **kw) == ALIGN, kw
    assert decode(lib, pages=1 << 27) == UNSUPPORTED   # 2^31 token positions
    c = cache()
    need = lib.gdn_paged_decode_workspace_bytes(c, 16)
    assert need > 0 and decode(lib, nbytes=need - 1) == WORKSPACE and decode(lib, nbytes=need) == DEVICE
    assert lib.gdn_paged_decode_workspace_bytes(c, 12) == 0 and lib.gdn_paged_decode_workspace_bytes(cache(d=32), 16) == 0


def test_sample_refusals(lib):
    assert sample(lib) == DEVICE and sample(lib, lp=None) == DEVICE
    assert sample(lib, B=0, x=None, u=None, tok=None) == OK
    assert sample(lib, V=0) == SHAPE and sample(lib, B=-1) == SHAPE and sample(lib, xs=-1) == SHAPE
    assert sample(lib, V=(1 << 22) + 1) == UNSUPPORTED
    assert sample(lib, dtype=2) == DTYPE
    for name in ("x", "u", "tok"):
        assert sample(lib, **{name: None}) == NULL, name
    for kw in (dict(x=FAKE + 2), dict(u=FAKE + 2), dict(t=FAKE + 1), dict(k=FAKE + 2), dict(tok=FAKE + 2)):
        assert sample(lib, **kw) == ALIGN, kw
    assert sample(lib, dtype=0, x=FAKE + 2) == DEVICE  # bf16 rows need no more than their own alignment


def test_tables_refusals(lib):
    assert tables(lib) == DEVICE
    assert tables(lib, B=0, new=None, lens=None, table=None) == DEVICE   # counts and cu_new are still written
    assert tables(lib, n=0, slots=None, pos=None) == DEVICE and tables(lib, n_free=0, free=None) == DEVICE
    for kw in (dict(B=-1), dict(page=0), dict(wide=-1), dict(n_free=-1), dict(n=-1)):
        assert tables(lib, **kw) == SHAPE, kw
    for name in ("new", "free", "table", "lens", "cu", "slots", "pos", "counts"):
        assert tables(lib, **{name: None}) == NULL, name
    for kw in (dict(slots=FAKE + 4), dict(cached=FAKE + 2), dict(counts=FAKE + 1)):
        assert tables(lib, **kw) == ALIGN, kw
    assert lib.gdn_page_tables_status(None, None) == NULL


def test_binding_refuses_host_tensors():
    z = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_paged_decode(torch.zeros(2, 4, 64, dtype=torch.bfloat16), z, z, i, i[:, 0])
    with pytest.raises(ValueError):
        gdn.gdn_kv_append(z[:, 0], z[:, 0], torch.zeros(4, dtype=torch.int64), z, z)
    with pytest.raises(ValueError):
        gdn.gdn_page_tables(i[:, 0], i[0], i, page=16, n_slots=4)
    with pytest.raises(ValueError):
        gdn.gdn_sample(torch.zeros(2, 8), torch.zeros(2, 8))
