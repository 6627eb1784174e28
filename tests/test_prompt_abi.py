"""The prompt chunks' entry points: refusals of the C ABI and of the binding.  No GPU: every call fails validation, so no
pointer is dereferenced."""
import pytest
import torch

import gated_delta_rule_16_gb300 as gdn
from gated_delta_rule_16_gb300 import _binding as bnd
from test_paged_abi import ALIGN, BAD_CACHES, DEVICE, DTYPE, FAKE, NULL, OK, SHAPE, UNSUPPORTED, WORKSPACE, cache


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_16_gb300 import build
    build.build()
    return gdn.load()


def rope(lib, n=4, Hq=8, Hkv=2, d=128, dtype=0, q=FAKE, qs=(1024, 128), k=FAKE, ks=(256, 128), pos=FAKE, freqs=FAKE, pairs=64, inter=0,
         qw=None, kw=None, qo=FAKE + 16, qos=(1024, 128), ko=FAKE + 16, kos=(256, 128)):
    return lib.gdn_qk_rope(n, Hq, Hkv, d, dtype, q, *qs, k, *ks, pos, freqs, pairs, inter, 1.0, qw, kw, 1e-6, qo, *qos, ko, *kos, None)


def prefill(lib, c=None, B=2, n=40, Hq=16, dtype=0, q=FAKE, qs=(2048, 128), table=FAKE, ts=10, pages=10, lens=FAKE, cu=FAKE, window=0, o=FAKE,
            lse=FAKE, ws=FAKE, nbytes=1 << 40):
    return lib.gdn_paged_prefill(c or cache(), B, n, Hq, dtype, q, *qs, table, ts, pages, lens, cu, window, 0.1, o, lse, ws, nbytes, None)


def logprobs(lib, B=2, V=100, dtype=1, x=FAKE, xs=100, tok=FAKE, top=5, lp=FAKE, ent=FAKE, tt=FAKE, tl=FAKE):
    return lib.gdn_logprobs(B, V, dtype, x, xs, tok, top, lp, ent, tt, tl, None)


def test_rope_refusals(lib):
    assert rope(lib) == DEVICE  # all arguments pass: stops at the device check here
    assert rope(lib, qo=FAKE, ko=FAKE) == DEVICE
    assert rope(lib, dtype=2) == DTYPE
    assert rope(lib, n=-1) == SHAPE and rope(lib, Hq=-1) == SHAPE and rope(lib, pairs=-1) == SHAPE and rope(lib, pairs=65) == SHAPE
    assert rope(lib, Hq=65000, Hkv=600) == SHAPE
    assert rope(lib, d=96) == UNSUPPORTED
    assert rope(lib, n=0, q=None, k=None, pos=None) == OK and rope(lib, Hq=0, Hkv=0, q=None, k=None) == OK
    assert rope(lib, Hkv=0, k=None, ko=None) == DEVICE and rope(lib, Hq=0, q=None, qo=None) == DEVICE
    assert rope(lib, q=None) == NULL and rope(lib, ko=None) == NULL and rope(lib, pos=None) == NULL and rope(lib, freqs=None) == NULL
    assert rope(lib, freqs=None, pairs=0) == DEVICE
    assert rope(lib, q=FAKE + 8) == ALIGN and rope(lib, ks=(256, 4)) == ALIGN and rope(lib, qos=(1028, 128)) == ALIGN
    assert rope(lib, pos=FAKE + 2) == ALIGN and rope(lib, freqs=FAKE + 4) == ALIGN and rope(lib, qw=FAKE + 2) == ALIGN
    assert rope(lib, qo=FAKE, qos=(2048, 128)) == UNSUPPORTED and rope(lib, ko=FAKE, kos=(256, 64)) == UNSUPPORTED
    assert rope(lib, qs=(-1024, 128)) == ALIGN


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_refusals(lib, kw, want):
    assert prefill(lib, cache(**kw), dtype=0) == want


def test_prefill_refusals(lib):
    assert prefill(lib) == DEVICE and prefill(lib, lse=None) == DEVICE
    assert prefill(lib, B=-1) == SHAPE and prefill(lib, n=-1) == SHAPE and prefill(lib, Hq=12) == SHAPE and prefill(lib, Hq=0) == SHAPE
    assert prefill(lib, window=-1) == SHAPE and prefill(lib, pages=-1) == SHAPE and prefill(lib, ts=-1) == SHAPE
    assert prefill(lib, n=2 ** 28) == SHAPE
    assert prefill(lib, dtype=1) == DTYPE and prefill(lib, cache(bnd.GDN_E4M3), dtype=1) == DTYPE
    assert prefill(lib, cache(bnd.GDN_E4M3)) == DEVICE and prefill(lib, cache(bnd.GDN_F32), dtype=1) == DEVICE
    assert prefill(lib, pages=2 ** 27) == UNSUPPORTED
    assert prefill(lib, B=0, q=None, cu=None) == OK and prefill(lib, n=0, q=None, o=None) == OK
    for name in ("q", "table", "lens", "cu", "o", "ws"):
        assert prefill(lib, **{name: None}) == NULL, name
    assert prefill(lib, pages=0, table=None) == DEVICE and prefill(lib, cache(pages=0, k=None, v=None)) == DEVICE
    for name in ("q", "o"):
        assert prefill(lib, **{name: FAKE + 8}) == ALIGN, name
    for name in ("table", "lens", "cu", "lse"):
        assert prefill(lib, **{name: FAKE + 2}) == ALIGN, name
    assert prefill(lib, ws=FAKE + 64) == ALIGN and prefill(lib, qs=(2048, 4)) == ALIGN
    need = lib.gdn_paged_prefill_workspace_bytes(cache(), 2, 40, 16)
    assert need > 0 and prefill(lib, nbytes=need) == DEVICE and prefill(lib, nbytes=need - 1) == WORKSPACE
    assert lib.gdn_paged_prefill_workspace_bytes(cache(d=96), 2, 40, 16) == 0
    assert lib.gdn_paged_prefill_workspace_bytes(cache(), 2, 40, 12) == 0
    assert lib.gdn_paged_prefill_workspace_bytes(cache(), -1, 40, 16) == 0 and lib.gdn_paged_prefill_workspace_bytes(cache(), 2, -1, 16) == 0
    assert lib.gdn_paged_prefill_status(None, None) == NULL and lib.gdn_paged_prefill_status(FAKE + 4, None) == ALIGN


def test_logprobs_refusals(lib):
    assert logprobs(lib) == DEVICE and logprobs(lib, ent=None) == DEVICE
    assert logprobs(lib, dtype=2) == DTYPE
    assert logprobs(lib, B=-1) == SHAPE and logprobs(lib, V=0) == SHAPE and logprobs(lib, xs=-1) == SHAPE
    assert logprobs(lib, top=-1) == SHAPE and logprobs(lib, V=4) == SHAPE
    assert logprobs(lib, top=33) == UNSUPPORTED and logprobs(lib, V=2 ** 30 + 1) == UNSUPPORTED
    assert logprobs(lib, B=0, x=None) == OK
    assert logprobs(lib, x=None) == NULL and logprobs(lib, tok=None) == NULL and logprobs(lib, lp=None) == NULL
    assert logprobs(lib, tt=None) == NULL and logprobs(lib, tl=None) == NULL and logprobs(lib, top=0, tt=None, tl=None) == DEVICE
    assert logprobs(lib, x=FAKE + 2) == ALIGN and logprobs(lib, dtype=0, x=FAKE + 2) == DEVICE and logprobs(lib, dtype=0, x=FAKE + 1) == ALIGN
    assert logprobs(lib, tok=FAKE + 2) == ALIGN and logprobs(lib, lp=FAKE + 1) == ALIGN


def test_binding_refusals():
    x, pos = torch.zeros((2, 4, 64)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gdn.gdn_qk_rope(x, x, pos, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        gdn.gdn_paged_prefill(x, x, x, pos, pos, pos)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gdn.gdn_logprobs(x[0], pos)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gdn.gdn_paged_prefill_status(torch.zeros(256, dtype=torch.uint8))
