"""PyTorch front end of the operators on a paged cache (include/kda_cache.h):
argument marshalling only, as in ``ops``.  The common case is marshalled by a
CPython module (csrc/py_cache.cpp): the checks here take longer than a small call.

A cache is [pages, page_size, heads, d], in any order in memory that keeps a
head's d channels contiguous and places apart: [pages, heads, page_size, d]
transposed, or halves of [pages, 2, page_size, heads, d].  Calls run on the
current stream of the tensors' own device, whichever device is current.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._lib import cache_calls, check, lib
from .layer import _MOST, _call, _dtype, _expect, _fits, _rows, _sizes_fit, _workspace
from .ops import _DTYPES, _ptr


_INT32, _FLOAT32 = torch.int32, torch.float32
_stream = torch._C._cuda_getCurrentRawStream


def _on_current_device(t) -> bool:
    """Whether a call on ``t`` may go through csrc/py_cache.cpp, which does not
    change the device (it returns None where an argument needs a word said)."""
    return isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == torch.cuda.current_device()


def _row_stride(t, name, dtype, T, H, d, device) -> int:
    """``_rows`` of a [T, H, d] tensor with the common cases first."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (T, H, d) and t.device == device:
        row, head, one = t.stride()
        if one == 1 and head == d and row >= H * d and T > 1 and H > 0:
            return row
    return _rows(t, name, dtype, torch.Size((T, H, d)), device, 1)


def _ints(t, name, shape, device):
    """Check a dense int32 tensor."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _INT32 and t.shape == shape
            and t.device == device and t.is_contiguous()):
        if t is None:
            raise TypeError(f"{name} must be a tensor")
        _expect(t, name, _INT32, shape, device)


def _cache(t, name, dtype, device, heads, d):
    """Check a cache; returns (pages, page size, distances between pages, tokens, heads)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != 4 or t.shape[2:] != (heads, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected (pages, page_size, {heads}, {d})")
    n, page = t.shape[:2]
    s = t.stride()
    if s[3] != 1 and d != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    if n > _MOST or not 1 <= page <= _MOST:
        _sizes_fit(name, n, page)
        raise ValueError(f"{name}: a page holds at least one token")
    return (n, page, s[0] if n > 1 else 0, s[1] if page > 1 else 0, s[2] if heads > 1 else 0)


def _caches(k_cache, v_cache, dtype, device, heads, d):
    k = _cache(k_cache, "k_cache", dtype, device, heads, d)
    if v_cache is not None:
        if (isinstance(v_cache, torch.Tensor) and v_cache.shape == k_cache.shape
                and v_cache.dtype is dtype and v_cache.stride() == k_cache.stride()
                and v_cache.device == device):
            return k
        if _cache(v_cache, "v_cache", dtype, device, heads, d) != k:
            raise ValueError("k_cache and v_cache must have one shape and one order in memory")
    return k


def _sessions(page_table, lens, cu_seqlens, tokens, device):
    """Check the sessions' table, lengths and offsets; returns (sessions, table width)."""
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a 2-D tensor")
    n, width = page_table.shape
    if n > _MOST or width > _MOST or tokens > _MOST:
        _sizes_fit("page_table", n, width, tokens)
    _ints(page_table, "page_table", (n, width), device)
    _ints(lens, "lens", (n,), device)
    if cu_seqlens is not None:
        _ints(cu_seqlens, "cu_seqlens", (n + 1,), device)
    elif tokens % n if n else tokens:
        raise ValueError(f"{tokens} tokens are not the same number for each of {n} sessions")
    return n, width


def cache_append(k: torch.Tensor, v: Optional[torch.Tensor], k_cache: torch.Tensor,
                 v_cache: Optional[torch.Tensor], page_table: torch.Tensor, lens: torch.Tensor,
                 cu_seqlens: Optional[torch.Tensor] = None, *, q: Optional[torch.Tensor] = None,
                 table: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 rotary_offset: int = 0, interleaved: bool = False,
                 out_q: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Keys and values of new tokens into a paged cache, the keys (and ``q``)
    rotated by position on the way (``kda_cache_append``); the caches are
    updated in place.

    k, v: [T, H, d] float32 or bfloat16 (may be slices of wider rows), d 64, 128
    or 576; v and v_cache None for a latent cache, whose values are channels of
    its keys.  k_cache, v_cache: [pages, page_size, H, d], in one order in
    memory.  page_table: [N, width] int32, the pages of each session's own
    tokens; lens: [N] int32, how many those are with the new ones; cu_seqlens:
    [N + 1] int32 for packed tokens, else T / N of each session.  ``table``
    [rows, rotary_dim] fp32 holds cos, then sin, and ``positions`` [T] int32 the
    row of each token, as for ``qk_norm``; channels rotary_offset .. rotary_offset +
    rotary_dim of each head are rotated in pairs (i, i + rotary_dim / 2), or
    (2 i, 2 i + 1) with ``interleaved``.  Returns the rotated q [T, Hq, d]
    (``out_q``, which may be ``q`` itself), or None without q.
    """
    if out_q is None and _on_current_device(k):
        done = cache_calls().append(_stream(k.get_device()), k, v, k_cache, v_cache, page_table, lens,
                                    cu_seqlens, q, table, positions, rotary_offset, interleaved)
        if done is not None:
            if done[0]:
                check(done[0], "kda_cache_append")
            return done[1]
    dt = _dtype_of_rows(k, "k")
    T, H, d = k.shape
    dev, dtype = k.device, k.dtype
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    ks = _row_stride(k, "k", dtype, T, H, d, dev)
    vs = 0 if v is None else _row_stride(v, "v", dtype, T, H, d, dev)
    pages, page, *strides = _caches(k_cache, v_cache, dtype, dev, H, d)
    n, width = _sessions(page_table, lens, cu_seqlens, T, dev)
    hq = qs = os = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [T, Hq, d]")
        hq = q.shape[1]
        _fits(q, "q")
        qs = _row_stride(q, "q", dtype, T, hq, d, dev)
        if out_q is None:
            out_q, os = torch.empty((T, hq, d), dtype=dtype, device=dev), hq * d
        else:
            os = _row_stride(out_q, "out_q", dtype, T, hq, d, dev)
    elif out_q is not None:
        raise ValueError("out_q needs q")
    rot = rows = 0
    if (table is None) != (positions is None):
        raise ValueError("a rotation needs both table and positions")
    if table is not None:
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table must be [rows, rotary_dim]")
        rows, rot = table.shape
        _fits(table, "table")
        _expect(table, "table", _FLOAT32, (rows, rot), dev)
        _ints(positions, "positions", (T,), dev)
    if not -_MOST <= rotary_offset <= _MOST:
        _sizes_fit("rotary_offset", abs(rotary_offset))
    _call("kda_cache_append", dev, _ptr(q), k.data_ptr(), _ptr(v), _ptr(table), _ptr(positions),
          page_table.data_ptr(), lens.data_ptr(), _ptr(cu_seqlens), _ptr(out_q), k_cache.data_ptr(),
          _ptr(v_cache), T, n, hq, H, d, rot, rotary_offset, rows, pages, page, width, qs, ks, vs, os,
          *strides, 1 if interleaved else 0, dt)
    return out_q


def _dtype_of_rows(t, name):
    dt = _dtype(t, name)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, d]")
    return dt


def prefix_attention_workspace_size(tokens: int, num_seqs: int, q_heads: int, kv_heads: int,
                                    head_dim: int, v_dim: int, page_size: int, table_width: int,
                                    prefix_width: int, dtype: torch.dtype) -> int:
    """Bytes of workspace ``prefix_attention`` needs (table_width, prefix_width:
    columns of page_table, entries of prefix_pages)."""
    sizes = (tokens, num_seqs, q_heads, kv_heads, head_dim, v_dim, page_size, table_width,
             prefix_width)
    _sizes_fit("prefix_attention", *sizes)
    n = lib().kda_prefix_attn_workspace_size(*sizes, _DTYPES[dtype])
    if n < 0:
        raise ValueError("invalid sizes")
    return int(n)


def prefix_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: Optional[torch.Tensor],
                     page_table: torch.Tensor, lens: torch.Tensor,
                     prefix_pages: Optional[torch.Tensor] = None,
                     prefix_len: Optional[torch.Tensor] = None,
                     cu_seqlens: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                     v_dim: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     output_lse: bool = False
                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Softmax attention of the new tokens of a batch of sessions over a prefix
    that they share (read once for every 128 of their rows) and each session's own
    tokens up to the new one itself (``kda_prefix_attn_fwd``).

    q: [T, Hq, d] (may be a slice of wider rows), Hq a multiple of the cache's
    heads, whose head j query heads Hq / H * j .. read; caches, page_table, lens
    and cu_seqlens as for ``cache_append``, which has put the new tokens' keys
    and values there.  prefix_pages: [P] int32 pages of the shared prefix and
    prefix_len: [1] int32 how many tokens of them count, or None.  d 64 or 128,
    or 576 with v_cache None and v_dim 512 (bfloat16): the values are then the
    first 512 channels of the keys.  ``scale`` is d ** -0.5 by default.  Returns
    (out [T, Hq, v_dim], lse [T, Hq] fp32, the log of each token's sum of
    exponentials, or None): 0 and -inf where a token sees nothing, be it that the
    lengths are zero or that no page it could see is there.
    """
    if (out is None and lse is None and workspace is None and _on_current_device(q) and q.dim() == 3
            and q.shape[-1]):
        d = q.shape[-1]
        done = cache_calls().attention(
            _stream(q.get_device()), q, k_cache, v_cache, page_table, lens, prefix_pages, prefix_len,
            cu_seqlens, d ** -0.5 if scale is None else scale,
            v_dim if v_dim is not None else (512 if v_cache is None and d == 576 else d), output_lse)
        if done is not None:
            if done[0]:
                check(done[0], "kda_prefix_attn_fwd")
            return done[1], done[2]
    dt = _dtype_of_rows(q, "q")
    T, hq, d = q.shape
    if not d:
        raise ValueError("q: a head has no channels")
    dev, dtype = q.device, q.dtype
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, heads, d]")
    H = k_cache.shape[2]
    if hq % H if H else hq:
        raise ValueError(f"{hq} query heads cannot share {H} heads of the cache")
    if H > _MOST:
        _sizes_fit("k_cache", H)
    pages, page, *strides = _caches(k_cache, v_cache, dtype, dev, H, d)
    dv = v_dim if v_dim is not None else (512 if v_cache is None and d == 576 else d)
    if not 0 <= dv <= _MOST:
        raise ValueError(f"v_dim is {dv}")
    qs = _row_stride(q, "q", dtype, T, hq, d, dev)
    n, width = _sessions(page_table, lens, cu_seqlens, T, dev)
    P = 0
    if (prefix_pages is None) != (prefix_len is None):
        raise ValueError("a prefix needs both prefix_pages and prefix_len")
    if prefix_pages is not None:
        if not isinstance(prefix_pages, torch.Tensor) or prefix_pages.dim() != 1:
            raise ValueError("prefix_pages must be a 1-D tensor")
        P = prefix_pages.shape[0]
        if P > _MOST:
            _sizes_fit("prefix_pages", P)
        _ints(prefix_pages, "prefix_pages", (P,), dev)
        _ints(prefix_len, "prefix_len", (1,), dev)
    if out is None:
        out, os = torch.empty((T, hq, dv), dtype=dtype, device=dev), hq * dv
    else:
        os = _row_stride(out, "out", dtype, T, hq, dv, dev)
    if lse is not None:
        _expect(lse, "lse", _FLOAT32, (T, hq), dev)
    elif output_lse:
        lse = torch.empty((T, hq), dtype=_FLOAT32, device=dev)
    need = lib().kda_prefix_attn_workspace_size(T, n, hq, H, d, dv, page, width, P, dt)
    ws, room = None, 0
    if need > 0 or workspace is not None:
        ws = _workspace(workspace, max(need, 0), dev)
        room = ws.numel()
    _call("kda_prefix_attn_fwd", dev, q.data_ptr(), k_cache.data_ptr(), _ptr(v_cache),
          page_table.data_ptr(), lens.data_ptr(), _ptr(prefix_pages), _ptr(prefix_len),
          _ptr(cu_seqlens), out.data_ptr(), _ptr(lse), T, n, hq, H, d, dv, pages, page, width, P, qs,
          os, *strides, d ** -0.5 if scale is None else scale, dt, _ptr(ws), room)
    return out, lse
