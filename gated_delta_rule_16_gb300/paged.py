"""Decode step over a paged key-value cache: ctypes binding of the entry points of the same names.

A cache is a pair of tensors indexed [page, cell, kv_head, dim] whose last
dimension is contiguous; head-major storage [pages, kv_heads, page, dim] is
passed as its ``transpose(1, 2)`` view.  An 8-bit cache is a pair of
``torch.float8_e4m3fn`` tensors with one fp32 scale per KV head.

These calls run once per layer and token, so the marshalling is kept short:
each check reads a tensor's attributes once, and the default workspace belongs
to one host thread, device and stream.  A workspace of the caller's is for one
call at a time: calls of several threads need one each.  Every call is enqueued
on `stream` (default: the current stream of the tensors' device) and returns
without waiting; what it allocates is free in that stream's order.  Inputs have
to be ready in it and to live (or be recorded on it) until the call has run, as
for any torch operation.  For a call inside a CUDA graph pass the outputs and a
workspace that outlive the graph.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import _binding
from ._binding import GDN_BF16, GDN_E4M3, GDN_F32, GdnKvCache, Workspace, _check, load

_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
_CACHE_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32, torch.float8_e4m3fn: GDN_E4M3}
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


class _Local(threading.local):
    """A thread's default workspaces, by device and stream.  Attention is two launches, between which another thread's
    calls on the same stream may come.  Attention of new tokens has its own, whose status stays what its last call left."""

    def __init__(self):
        self.ws, self.prefill = {}, {}


_local = _Local()
_ws_bytes = {}  # answers of gdn_paged_decode_workspace_bytes
# not in a torch built without CUDA, in which no call gets as far as these
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_empty = torch.empty


def _want(t, name, dtype, shape, dev):
    """A contiguous tensor of this type, shape and CUDA device number; returns its address."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, is on {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _cuda(t, name):
    """The number of a tensor's CUDA device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _handle(dev, stream):
    """The call's stream as an address."""
    return _current_stream(dev) if stream is None else stream.cuda_stream


def _elsewhere(dev, stream):
    """Whether the call's stream is not the current one."""
    return stream.cuda_stream != _current_stream(dev)


def _on(stream, dev, fn, given, *args, **kw):
    """fn on another stream than the current one.  It becomes the current one for the call, so that the memory of outputs
    and workspaces which the call makes is free in that stream's order; memory that work of the stream outside may still
    use is not handed out.  Tensors of either stream are recorded on the other: they are not reused while one of both uses them."""
    if stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    outside = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        got = fn(*args, **kw)
    for t in given:
        if isinstance(t, Workspace):
            t = t.buf
        if t is not None:
            t.record_stream(stream)
    for t in got:
        t.record_stream(outside)
    return got


def _workspace(ws, nbytes, dev, handle, own=None):
    """(address, bytes) of the caller's workspace, or of this thread, device and stream's own."""
    if ws is None:
        if own is None:
            own = _local.ws
        buf = own.get((dev, handle))
        if buf is None or buf.numel() < nbytes:
            buf = own[dev, handle] = _empty((nbytes,), dtype=torch.uint8, device=torch.device("cuda", dev))
        return buf.data_ptr(), buf.numel()
    if isinstance(ws, Workspace):
        ws = ws.get(nbytes, torch.device("cuda", dev))
    if ws.get_device() != dev:
        raise ValueError(f"workspace must be on cuda:{dev}, is on {ws.device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _call(name, dev, *args):
    fn = getattr(_binding._lib or load(), name)
    if _current_device() == dev:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc:
        _check(name, rc)


def _cache(k, v, k_scale, v_scale, dev):
    """The C description of a cache, checked."""
    shape, stride, kind = k.shape, k.stride(), k.dtype
    if len(shape) != 4:
        raise ValueError(f"k_cache must have 4 dimensions [pages, page, kv_heads, dim], got {len(shape)}")
    code = _CACHE_CODES.get(kind)
    if code is None:
        raise TypeError(f"k_cache must be bfloat16, float32 or float8_e4m3fn, got {kind}")
    if v.dtype is not kind or v.shape != shape or v.stride() != stride:
        raise ValueError("v_cache must have k_cache's dtype, shape and strides")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"the cache must be on cuda:{dev}")
    pages, page, heads, d = shape
    if stride[3] != 1:
        raise ValueError("the cache's last dimension must be contiguous")
    ks = vs = None
    if code == GDN_E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        ks, vs = _want(k_scale, "k_scale", _F32, (heads,), dev), _want(v_scale, "v_scale", _F32, (heads,), dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to an 8-bit cache")
    return GdnKvCache(k.data_ptr(), v.data_ptr(), stride[0], stride[1], stride[2], ks, vs, pages, page, heads, d, code)


def gdn_page_tables(new_lens, free_pages, block_table, *, page, cached_lens=None, n_slots=None, slots=None,
                    positions=None, seq_lens=None, cu_new=None, counts=None, stream=None):
    """Block tables and slot maps of one step, from the requests' lengths.

    new_lens [B] and cached_lens [B] (default 0) int32: tokens that each request adds and has;
    free_pages int32: ids of free pages, taken in order; block_table [B, max_pages] int32, updated
    in place (entries of pages held already are kept).  n_slots: length of the slot map (at least
    the number of new tokens; a captured step keeps it fixed), or pass `slots` and `positions`.
    Returns (slots int64, positions int32, seq_lens int32 [B], cu_new int32 [B+1], counts int32 [4] =
    {tokens, pages taken, status bits, longest sequence}); gdn_page_tables_status reads the status."""
    dev = _cuda(block_table, "block_table")
    if stream is not None and _elsewhere(dev, stream):
        return _on(stream, dev, gdn_page_tables, (slots, positions, seq_lens, cu_new, counts), new_lens, free_pages, block_table,
                   page=page, cached_lens=cached_lens, n_slots=n_slots, slots=slots, positions=positions, seq_lens=seq_lens,
                   cu_new=cu_new, counts=counts)
    B, max_pages = block_table.shape
    if n_slots is None:
        if slots is None:
            raise ValueError("gdn_page_tables needs n_slots or slots")
        n_slots = slots.numel()
    device = block_table.device
    if slots is None:
        slots = _empty((n_slots,), dtype=_I64, device=device)
    if positions is None:
        positions = _empty((n_slots,), dtype=_I32, device=device)
    if seq_lens is None:
        seq_lens = _empty((B,), dtype=_I32, device=device)
    if cu_new is None:
        cu_new = _empty((B + 1,), dtype=_I32, device=device)
    if counts is None:
        counts = _empty((4,), dtype=_I32, device=device)
    n_free = free_pages.numel()
    _call("gdn_page_tables", dev, B, page, max_pages, None if cached_lens is None else _want(cached_lens, "cached_lens", _I32, (B,), dev),
          _want(new_lens, "new_lens", _I32, (B,), dev), _want(free_pages, "free_pages", _I32, (n_free,), dev), n_free,
          _want(block_table, "block_table", _I32, (B, max_pages), dev), _want(seq_lens, "seq_lens", _I32, (B,), dev),
          _want(cu_new, "cu_new", _I32, (B + 1,), dev), _want(slots, "slots", _I64, (n_slots,), dev),
          _want(positions, "positions", _I32, (n_slots,), dev), n_slots, _want(counts, "counts", _I32, (4,), dev),
          _current_stream(dev))
    return slots, positions, seq_lens, cu_new, counts


def gdn_page_tables_status(counts, stream=None) -> int:
    """Status of a gdn_page_tables call from its counts (synchronises the stream): 0, or
    9 (GDN_ERR_CAPACITY) if the free list, the table or the slot map was too short."""
    dev = _cuda(counts, "counts")
    with torch.cuda.device(dev):
        return int(load().gdn_page_tables_status(_want(counts, "counts", _I32, (4,), dev), _handle(dev, stream)))


def gdn_kv_append(k, v, slots, k_cache, v_cache, *, k_scale=None, v_scale=None, stream=None):
    """Write new tokens' keys and values, k and v [n, kv_heads, dim], to slots [n] (int64; -1 is skipped)
    of a cache in place.  k and v have the cache's dtype, or bfloat16 / float32 with an 8-bit cache."""
    dev = _cuda(k_cache, "k_cache")
    c = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    code = _CODES.get(k.dtype)
    if code is None or v.dtype is not k.dtype:
        raise TypeError(f"k and v must both be bfloat16 or float32, got {k.dtype} and {v.dtype}")
    n = slots.numel()
    if k.shape != (n, c.Hkv, c.d) or v.shape != k.shape:
        raise ValueError(f"k and v must be [{n}, {c.Hkv}, {c.d}], got {tuple(k.shape)} and {tuple(v.shape)}")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"k and v must be on cuda:{dev}")
    ks, vs = k.stride(), v.stride()
    if ks[2] != 1 or vs[2] != 1:
        raise ValueError("the last dimension of k and v must be contiguous")
    _call("gdn_kv_append", dev, c, n, code, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
          _want(slots, "slots", _I64, (n,), dev), _handle(dev, stream))


def gdn_paged_decode(q, k_cache, v_cache, block_table, seq_lens, *, k_scale=None, v_scale=None, scale=None, window=0,
                     o=None, lse=None, workspace=None, stream=None):
    """Softmax attention of one new token per request, q [B, heads, dim], over its cached tokens.

    block_table [B, max_pages] int32 (its row stride may be 0: all requests share one row); seq_lens
    [B] int32, the new token included; window: only the last `window` tokens (0: all); scale:
    default dim ** -0.5.  Returns (o [B, heads, dim] in q's dtype, lse [B, heads] fp32)."""
    dev = _cuda(q, "q")
    if stream is not None and _elsewhere(dev, stream):
        return _on(stream, dev, gdn_paged_decode, (o, lse, workspace), q, k_cache, v_cache, block_table, seq_lens, k_scale=k_scale,
                   v_scale=v_scale, scale=scale, window=window, o=o, lse=lse, workspace=workspace)
    c = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    code = _CODES.get(q.dtype)
    if code is None or (c.dtype != GDN_E4M3 and c.dtype != code):
        raise TypeError(f"q must have the cache's dtype (bfloat16 with an 8-bit cache), got {q.dtype}")
    B, heads, d = q.shape
    if d != c.d:
        raise ValueError(f"q has dim {d}, the cache {c.d}")
    qs, ts = q.stride(), block_table.stride()
    if qs[2] != 1:
        raise ValueError("the last dimension of q must be contiguous")
    if block_table.dtype is not _I32:
        raise TypeError(f"block_table must be int32, got {block_table.dtype}")
    if block_table.get_device() != dev:
        raise ValueError(f"block_table must be on cuda:{dev}, is on {block_table.device}")
    rows, max_pages = block_table.shape
    if rows != B or (ts[1] != 1 and max_pages > 1):
        raise ValueError(f"block_table must be [{B}, max_pages] with contiguous rows, got {tuple(block_table.shape)}")
    if o is None:
        o = _empty((B, heads, d), dtype=q.dtype, device=q.device)
        o_at = o.data_ptr()
    else:
        o_at = _want(o, "o", q.dtype, (B, heads, d), dev)
    if lse is None:
        lse = _empty((B, heads), dtype=_F32, device=q.device)
        lse_at = lse.data_ptr()
    else:
        lse_at = _want(lse, "lse", _F32, (B, heads), dev)
    handle = _current_stream(dev)
    key = (c.dtype, d, heads, c.Hkv)
    nbytes = _ws_bytes.get(key)
    if nbytes is None:
        nbytes = _ws_bytes[key] = load().gdn_paged_decode_workspace_bytes(c, heads)
    ws, ws_bytes = _workspace(workspace, nbytes, dev, handle)
    _call("gdn_paged_decode", dev, c, B, heads, code, q.data_ptr(), qs[0], qs[1], block_table.data_ptr(), ts[0], max_pages,
          _want(seq_lens, "seq_lens", _I32, (B,), dev), window, d ** -0.5 if scale is None else scale, o_at, lse_at,
          ws, ws_bytes, handle)
    return o, lse


def gdn_sample(logits, noise, *, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, logprobs=None,
               stream=None):
    """The next token of every row of logits [B, V] (bfloat16 or float32), from uniform random numbers
    noise [B, V] (fp32).  temperature, top_p, min_p [B] fp32 and top_k [B] int32: include/gdn.h has the
    order of the filters; None leaves one out.  Returns (tokens int32 [B], logprobs fp32 [B])."""
    dev = _cuda(logits, "logits")
    if stream is not None and _elsewhere(dev, stream):
        return _on(stream, dev, gdn_sample, (tokens, logprobs), logits, noise, temperature=temperature, top_k=top_k, top_p=top_p,
                   min_p=min_p, tokens=tokens, logprobs=logprobs)
    code = _CODES.get(logits.dtype)
    if code is None:
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    B, V = logits.shape
    if noise.dtype is not _F32 or noise.shape != logits.shape or noise.get_device() != dev:
        raise ValueError(f"noise must be float32 {tuple(logits.shape)} on cuda:{dev}")
    ls, ns = logits.stride(), noise.stride()
    if V > 1 and (ls[1] != 1 or ns[1] != 1):
        raise ValueError("the rows of logits and noise must be contiguous")
    rows = (B,)
    if tokens is None:
        tokens = _empty(rows, dtype=_I32, device=logits.device)
    if logprobs is None:
        logprobs = _empty(rows, dtype=_F32, device=logits.device)
    _call("gdn_sample", dev, B, V, code, logits.data_ptr(), ls[0], noise.data_ptr(), ns[0],
          None if temperature is None else _want(temperature, "temperature", _F32, rows, dev),
          None if top_k is None else _want(top_k, "top_k", _I32, rows, dev),
          None if top_p is None else _want(top_p, "top_p", _F32, rows, dev),
          None if min_p is None else _want(min_p, "min_p", _F32, rows, dev),
          _want(tokens, "tokens", _I32, rows, dev), _want(logprobs, "logprobs", _F32, rows, dev),
          _current_stream(dev))
    return tokens, logprobs
