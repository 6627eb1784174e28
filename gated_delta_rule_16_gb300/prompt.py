"""Prompt chunks through softmax-attention layers: ctypes binding of the entry points of the same names.

New tokens' queries and keys are normalised per head and rotated (gdn_qk_rope), the keys and values written to the paged cache
(gdn_kv_append), the queries attended over it (gdn_paged_prefill), and a scored prompt's logits become log probabilities
(gdn_logprobs).  Caches, streams and workspaces are as in the decode step's calls (paged.py).
"""
from __future__ import annotations

import torch

from . import paged
from ._binding import GDN_E4M3, Workspace, _check, load
from .paged import _CODES, _F32, _I32, _cache, _call, _cuda, _elsewhere, _handle, _on, _want, _workspace

_F64 = torch.float64
_ws_bytes = {}  # answers of gdn_paged_prefill_workspace_bytes


def _rows(t, name, dtype, shape, dev):
    """Strides of a tensor [n, heads, dim] on this CUDA device whose last dimension is contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, is on {t.device}")
    s = t.stride()
    if s[2] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return s


def gdn_qk_rope(q, k, positions, freqs, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, mscale=1.0,
                q_out=None, k_out=None, stream=None):
    """Per-head norm (where weights [dim] fp32 are given) and rotary positions of q [n, heads, dim] and k [n, kv_heads, dim].

    positions [n] int32; freqs [pairs] float64: radians per token of the first 2 * pairs dims' pairs, (i, i + pairs) or,
    interleaved, (2 i, 2 i + 1); the rotated dims are scaled by mscale.  q and k may be slices of one projection, and q_out and
    k_out may be q and k.  Returns (q_out, k_out)."""
    dev = _cuda(q, "q")
    if stream is not None and _elsewhere(dev, stream):
        return _on(stream, dev, gdn_qk_rope, (q_out, k_out), q, k, positions, freqs, q_weight=q_weight, k_weight=k_weight, eps=eps,
                   interleaved=interleaved, mscale=mscale, q_out=q_out, k_out=k_out)
    code = _CODES.get(q.dtype)
    if code is None:
        raise TypeError(f"q must be bfloat16 or float32, got {q.dtype}")
    n, heads, d = q.shape
    kv_heads = k.shape[1]
    qs, ks = _rows(q, "q", q.dtype, (n, heads, d), dev), _rows(k, "k", q.dtype, (n, kv_heads, d), dev)
    if q_out is None:
        q_out, qo = paged._empty((n, heads, d), dtype=q.dtype, device=q.device), (heads * d, d)
    else:
        qo = _rows(q_out, "q_out", q.dtype, (n, heads, d), dev)
    if k_out is None:
        k_out, ko = paged._empty((n, kv_heads, d), dtype=q.dtype, device=q.device), (kv_heads * d, d)
    else:
        ko = _rows(k_out, "k_out", q.dtype, (n, kv_heads, d), dev)
    pairs = freqs.numel()
    _call("gdn_qk_rope", dev, n, heads, kv_heads, d, code, q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1],
          _want(positions, "positions", _I32, (n,), dev), _want(freqs, "freqs", _F64, (pairs,), dev), pairs, int(interleaved), mscale,
          None if q_weight is None else _want(q_weight, "q_weight", _F32, (d,), dev),
          None if k_weight is None else _want(k_weight, "k_weight", _F32, (d,), dev), eps,
          q_out.data_ptr(), qo[0], qo[1], k_out.data_ptr(), ko[0], ko[1], paged._current_stream(dev))
    return q_out, k_out


def gdn_paged_prefill(q, k_cache, v_cache, block_table, seq_lens, cu_new, *, k_scale=None, v_scale=None, scale=None, window=0,
                      o=None, lse=None, workspace=None, stream=None):
    """Softmax attention of the new tokens q [n, heads, dim] over the cache, which holds them already.

    Request b's tokens are rows cu_new[b] to cu_new[b + 1] (cu_new [B+1] int32) and the last of its seq_lens[b] tokens; each attends
    to those up to itself, or to the last `window` of them.  block_table [B, max_pages] int32 (its row stride may be 0); scale:
    default dim ** -0.5.  Rows behind cu_new[B] are left as they are.  o may be q where q is contiguous.  Returns (o [n, heads, dim] in q's
    dtype, lse [n, heads] fp32).  A `workspace` belongs to one call at a time (default: this thread's for the device and stream); gdn_paged_prefill_status
    asks whether the call ran through."""
    dev = _cuda(q, "q")
    if stream is not None and _elsewhere(dev, stream):
        return _on(stream, dev, gdn_paged_prefill, (o, lse, workspace), q, k_cache, v_cache, block_table, seq_lens, cu_new,
                   k_scale=k_scale, v_scale=v_scale, scale=scale, window=window, o=o, lse=lse, workspace=workspace)
    c = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    code = _CODES.get(q.dtype)
    if code is None or (c.dtype != GDN_E4M3 and c.dtype != code):
        raise TypeError(f"q must have the cache's dtype (bfloat16 with an 8-bit cache), got {q.dtype}")
    n, heads, d = q.shape
    if d != c.d:
        raise ValueError(f"q has dim {d}, the cache {c.d}")
    qs, ts = q.stride(), block_table.stride()
    if qs[2] != 1:
        raise ValueError("the last dimension of q must be contiguous")
    if block_table.dtype is not _I32:
        raise TypeError(f"block_table must be int32, got {block_table.dtype}")
    if block_table.get_device() != dev:
        raise ValueError(f"block_table must be on cuda:{dev}, is on {block_table.device}")
    B, max_pages = block_table.shape
    if ts[1] != 1 and max_pages > 1:
        raise ValueError("the rows of block_table must be contiguous")
    if o is None:
        o = paged._empty((n, heads, d), dtype=q.dtype, device=q.device)
        o_at = o.data_ptr()
    else:
        o_at = _want(o, "o", q.dtype, (n, heads, d), dev)
    if lse is None:
        lse = paged._empty((n, heads), dtype=_F32, device=q.device)
        lse_at = lse.data_ptr()
    else:
        lse_at = _want(lse, "lse", _F32, (n, heads), dev)
    handle = paged._current_stream(dev)
    key = (c.dtype, d, heads, c.Hkv, B, n)
    nbytes = _ws_bytes.get(key)
    if nbytes is None:
        if len(_ws_bytes) > 4096:  # prompts of ever other lengths
            _ws_bytes.clear()
        nbytes = _ws_bytes[key] = load().gdn_paged_prefill_workspace_bytes(c, B, n, heads)
    ws, ws_bytes = _workspace(workspace, nbytes, dev, handle, paged._local.prefill)
    _call("gdn_paged_prefill", dev, c, B, n, heads, code, q.data_ptr(), qs[0], qs[1], block_table.data_ptr(), ts[0], max_pages,
          _want(seq_lens, "seq_lens", _I32, (B,), dev), _want(cu_new, "cu_new", _I32, (B + 1,), dev), window,
          d ** -0.5 if scale is None else scale, o_at, lse_at, ws, ws_bytes, handle)
    return o, lse


def gdn_paged_prefill_status(workspace=None, stream=None) -> int:
    """Status of the gdn_paged_prefill call that used a workspace last (synchronises the stream): 0, or 10 (GDN_ERR_TIMEOUT)
    if a wait inside a kernel ran out, with the outputs not valid.  Without a workspace: of this thread's last call without one on
    the stream (default: the current one of the current device)."""
    if workspace is None:
        dev = torch.cuda.current_device() if stream is None else stream.device_index
        buf = paged._local.prefill.get((dev, _handle(dev, stream)))
    else:
        buf = workspace.buf if isinstance(workspace, Workspace) else workspace
    if buf is None:
        raise ValueError("no call has used the workspace")
    dev = _cuda(buf, "workspace")
    with torch.cuda.device(dev):
        return int(load().gdn_paged_prefill_status(buf.data_ptr(), _handle(dev, stream)))


def gdn_selftest_paged_prefill_wait(limit_ms: int = 0) -> None:
    """In this thread's following gdn_paged_prefill calls a CTA's copies wait after its first 128 keys for what never comes; the wait
    runs out after limit_ms (1 to 2000), and the status is 10.  0: as normally."""
    _check("gdn_selftest_paged_prefill_wait", load().gdn_selftest_paged_prefill_wait(limit_ms))


def gdn_logprobs(logits, tokens, *, top=0, logprobs=None, entropy=None, top_tokens=None, top_logprobs=None, stream=None):
    """Log probabilities of tokens [B] (int32; one outside the vocabulary gets 0) under logits [B, V] (bfloat16 or float32).

    Returns (logprobs [B], entropy [B], top_tokens int32 [B, top], top_logprobs [B, top]): the `top` (at most 32) likeliest tokens in
    descending order, ties by the lowest index."""
    dev = _cuda(logits, "logits")
    if stream is not None and _elsewhere(dev, stream):
        return _on(stream, dev, gdn_logprobs, (logprobs, entropy, top_tokens, top_logprobs), logits, tokens, top=top, logprobs=logprobs,
                   entropy=entropy, top_tokens=top_tokens, top_logprobs=top_logprobs)
    code = _CODES.get(logits.dtype)
    if code is None:
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    B, V = logits.shape
    stride = logits.stride()
    if V > 1 and stride[1] != 1:
        raise ValueError("the rows of logits must be contiguous")
    device = logits.device
    if logprobs is None:
        logprobs = paged._empty((B,), dtype=_F32, device=device)
    if entropy is None:
        entropy = paged._empty((B,), dtype=_F32, device=device)
    if top_tokens is None:
        top_tokens = paged._empty((B, max(top, 0)), dtype=_I32, device=device)
    if top_logprobs is None:
        top_logprobs = paged._empty((B, max(top, 0)), dtype=_F32, device=device)
    _call("gdn_logprobs", dev, B, V, code, logits.data_ptr(), stride[0], _want(tokens, "tokens", _I32, (B,), dev), top,
          _want(logprobs, "logprobs", _F32, (B,), dev), _want(entropy, "entropy", _F32, (B,), dev),
          _want(top_tokens, "top_tokens", _I32, (B, max(top, 0)), dev), _want(top_logprobs, "top_logprobs", _F32, (B, max(top, 0)), dev),
          paged._current_stream(dev))
    return logprobs, entropy, top_tokens, top_logprobs
