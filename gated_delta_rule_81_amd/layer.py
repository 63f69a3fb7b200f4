"""PyTorch front end of the operators around the recurrence
(include/kda_layer.h): argument marshalling only, as in ``ops``.

Tensors with one row per token ([B, T, ...] or [B, ...] for a single token) may
be slices of wider rows: everything behind the token axis has to be contiguous
and consecutive tokens a fixed distance apart.  Calls run on the current stream
of the tensors' own device, whichever device is current.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._lib import check, lib
from .ops import _DTYPES, _ptr
from .ops import _expect as _expect_dense

_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
_NORMS = {"l2": 0, "rms": 1}

_MOST = (1 << 31) - 1  # sizes go to the library in 32 bits, which ctypes would cut off


def _sizes_fit(name, *sizes):
    if max(sizes, default=0) > _MOST:
        raise ValueError(f"{name}: a size of {max(sizes)} does not fit 32 bits")


def _fits(t, name):
    if not 0 < t.numel() <= _MOST:  # else no size is larger
        _sizes_fit(name, *t.shape)


def _rows(t, name, dtype, shape, device, lead: int) -> int:
    """Check a tensor whose first ``lead`` axes count tokens; returns the
    distance in elements between consecutive tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    sizes = t.shape
    if sizes != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return sizes[lead:].numel()
    strides, width = t.stride(), 1
    for i in range(len(sizes) - 1, lead - 1, -1):
        if strides[i] != width and sizes[i] != 1:
            raise ValueError(f"{name}: the values of a token must be contiguous")
        width *= sizes[i]
    row, count = None, 1  # distance between tokens; tokens behind the axis looked at
    for i in range(lead - 1, -1, -1):
        if sizes[i] != 1:
            if row is None:
                row = strides[i]
            elif strides[i] != row * count:
                raise ValueError(f"{name}: tokens must be a fixed distance apart")
            count *= sizes[i]
    row = width if row is None or t.numel() == 0 else row
    if row < width:
        raise ValueError(f"{name}: the rows of two tokens overlap")
    return row


def _expect(t, name, dtype, shape, device):
    """``ops._expect`` with the common case first."""
    if t is None or (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                     and t.device == device and t.is_contiguous()):
        return
    _expect_dense(t, name, dtype, shape, device)


def _dtype(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    _fits(t, name)
    return _DTYPES[t.dtype]


def _num_seqs(cu_seqlens, batch, device):
    if cu_seqlens is None:
        return batch
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or not len(cu_seqlens):
        raise ValueError("cu_seqlens must be a 1-D tensor")
    _expect(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, device)
    if batch != 1:
        raise ValueError("packed sequences need a batch of 1")
    _fits(cu_seqlens, "cu_seqlens")
    return cu_seqlens.shape[0] - 1


def _call(name, device, *args):
    """Call a library function on ``device``'s current stream."""
    if device.type != "cuda":
        raise ValueError(f"{name} needs tensors on a GPU, got {device}")
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)  # no Stream object for a handle
    if torch.cuda.current_device() == index:
        rc = getattr(lib(), name)(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = getattr(lib(), name)(*args, stream)
    if rc:
        check(rc, name)


def _workspace(workspace, need, device):
    if need < 0:
        raise ValueError("invalid sizes")
    if workspace is None:
        return torch.empty(max(int(need), 1), dtype=torch.uint8, device=device)
    _expect(workspace, "workspace", torch.uint8, (workspace.numel(),), device)
    return workspace


def _out(t, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device) if t is None else t


def _out_rows(t, name, like, device, lead: int):
    """An output with ``like``'s dtype and shape, new if ``t`` is None, and the
    distance between its tokens."""
    if t is None:
        return (torch.empty_like(like, memory_format=torch.contiguous_format),
                like.shape[lead:].numel())
    return t, _rows(t, name, like.dtype, like.shape, device, lead)


# ---------------------------------------------------------------- short convolution
def _conv_common(x, weight, bias, activation):
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or 'none', got {activation!r}")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [C, width]")
    _fits(weight, "weight")
    C = x.shape[2]
    _expect(weight, "weight", torch.float32, (C, weight.shape[1]), x.device)
    _expect(bias, "bias", torch.float32, (C,), x.device)
    return _ACTIVATIONS[activation]


def short_conv(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               initial_state: Optional[torch.Tensor] = None,
               cu_seqlens: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
               out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
               output_final_state: bool = True
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Depthwise causal convolution over a few tokens (``kda_short_conv_fwd``),
    the stage before a recurrence's q, k and v (or x, B and C).

    x: [B, T, C] float32 or bfloat16 (may be a slice of wider rows); weight:
    [C, width] fp32, width 2 to 4, the last tap is the token itself; bias: [C]
    fp32 or None; initial_state: [N, width - 1, C] rows before each sequence's
    first token, dtype of x, or None (zeros); cu_seqlens as for ``chunk_fwd``;
    activation "silu" or "none".  Returns (out [B, T, C], final_state
    [N, width - 1, C] or None): the rows the next call continues from.
    """
    dt = _dtype(x, "x")
    act = _conv_common(x, weight, bias, activation)
    (B, T, C), W, dev = x.shape, weight.shape[1], x.device
    xs = _rows(x, "x", x.dtype, x.shape, dev, 2)
    N = _num_seqs(cu_seqlens, B, dev)
    state = (N, W - 1, C)
    _expect(initial_state, "initial_state", x.dtype, state, dev)
    out, os = _out_rows(out, "out", x, dev, 2)
    if final_state is None and output_final_state:
        final_state = torch.empty(state, dtype=x.dtype, device=dev)
    _expect(final_state, "final_state", x.dtype, state, dev)
    _call("kda_short_conv_fwd", dev, _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state),
          _ptr(cu_seqlens), _ptr(out), _ptr(final_state), B, T, C, W, xs, os,
          N if cu_seqlens is not None else 0, act, dt)
    return out, final_state


def short_conv_bwd_workspace_size(batch: int, seq_len: int, channels: int, width: int) -> int:
    """Bytes of workspace ``short_conv_bwd`` needs."""
    _sizes_fit("short_conv_bwd", batch, seq_len, channels, width)
    n = lib().kda_short_conv_bwd_workspace_size(batch, seq_len, channels, width)
    if n < 0:
        raise ValueError("invalid sizes")
    return int(n)


def short_conv_bwd(x: torch.Tensor, weight: torch.Tensor, d_out: torch.Tensor,
                   bias: Optional[torch.Tensor] = None,
                   d_final_state: Optional[torch.Tensor] = None,
                   initial_state: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, *,
                   activation: Optional[str] = "silu", workspace: Optional[torch.Tensor] = None,
                   grads: Optional[dict] = None,
                   output_initial_state_grad: bool = True) -> dict:
    """Gradients of ``short_conv`` (``kda_short_conv_bwd``): given dL/d out and
    dL/d final_state (None = zero), a dict with dx (dtype of x), dweight, dbias
    (fp32; dbias None without a bias) and d_initial_state (dtype of x, or None
    when ``output_initial_state_grad`` is False).  ``grads`` may hold
    preallocated outputs under the same names, ``workspace`` a uint8 tensor of
    ``short_conv_bwd_workspace_size`` bytes.
    """
    dt = _dtype(x, "x")
    act = _conv_common(x, weight, bias, activation)
    (B, T, C), W, dev = x.shape, weight.shape[1], x.device
    xs = _rows(x, "x", x.dtype, x.shape, dev, 2)
    gs = _rows(d_out, "d_out", x.dtype, x.shape, dev, 2)
    N = _num_seqs(cu_seqlens, B, dev)
    state = (N, W - 1, C)
    _expect(initial_state, "initial_state", x.dtype, state, dev)
    _expect(d_final_state, "d_final_state", x.dtype, state, dev)
    g = dict(grads or {})
    g["dx"], dxs = _out_rows(g.get("dx"), "dx", x, dev, 2)
    g["dweight"] = _out(g.get("dweight"), (C, W), torch.float32, dev)
    _expect(g["dweight"], "dweight", torch.float32, (C, W), dev)
    g["dbias"] = None if bias is None else _out(g.get("dbias"), (C,), torch.float32, dev)
    _expect(g["dbias"], "dbias", torch.float32, (C,), dev)
    g.setdefault("d_initial_state", None)
    if g["d_initial_state"] is None and output_initial_state_grad:
        g["d_initial_state"] = torch.empty(state, dtype=x.dtype, device=dev)
    _expect(g["d_initial_state"], "d_initial_state", x.dtype, state, dev)
    ws = _workspace(workspace, lib().kda_short_conv_bwd_workspace_size(B, T, C, W), dev)
    _call("kda_short_conv_bwd", dev, _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_state),
          _ptr(cu_seqlens), _ptr(d_out), _ptr(d_final_state), _ptr(g["dx"]), _ptr(g["dweight"]),
          _ptr(g["dbias"]), _ptr(g["d_initial_state"]), B, T, C, W, xs, gs, dxs,
          N if cu_seqlens is not None else 0, act, dt, _ptr(ws), ws.numel())
    return g


def short_conv_step(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``short_conv`` for one token per session (``kda_short_conv_step``): x
    [B, C], state [B, width - 1, C] moved on by one row in place.  Returns out
    [B, C]."""
    dt = _dtype(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [B, C]")
    act = _conv_common(x[None], weight, bias, activation)
    (B, C), W, dev = x.shape, weight.shape[1], x.device
    xs = _rows(x, "x", x.dtype, x.shape, dev, 1)
    if state is None:
        raise TypeError("state must be a tensor")
    _expect(state, "state", x.dtype, (B, W - 1, C), dev)
    out, os = _out_rows(out, "out", x, dev, 1)
    _call("kda_short_conv_step", dev, _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(out),
          B, C, W, xs, os, act, dt)
    return out


# ---------------------------------------------------------------- norm and rotation
def _qk_common(q, k, q_weight, k_weight, table, positions, kind):
    if kind not in _NORMS:
        raise ValueError(f"kind must be 'l2' or 'rms', got {kind!r}")
    if q.dim() < 2 or k.dim() != q.dim() or q.shape[:-2] != k.shape[:-2]:
        raise ValueError("q and k must be [..., heads, d] with the same leading axes")
    d, dev, lead = q.shape[-1], q.device, q.dim() - 2
    strides = (_rows(q, "q", q.dtype, q.shape, dev, lead),
               _rows(k, "k", q.dtype, (*k.shape[:-1], d), dev, lead))
    _expect(q_weight, "q_weight", torch.float32, (d,), dev)
    _expect(k_weight, "k_weight", torch.float32, (d,), dev)
    rot = rows = 0
    if (table is None) != (positions is None):
        raise ValueError("a rotation needs both table and positions")
    if table is not None:
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table must be [rows, rotary_dim]")
        rows, rot = table.shape
        _fits(table, "table")
        _expect(table, "table", torch.float32, (rows, rot), dev)
        _expect(positions, "positions", torch.int32, q.shape[:-2], dev)
    tokens = 1
    for n in q.shape[:-2]:
        tokens *= n
    _fits(k, "k")
    if tokens > _MOST:
        _sizes_fit("q and k", tokens)
    return tokens, q.shape[-2], k.shape[-2], d, rot, rows, strides, lead


def qk_norm(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
            k_weight: Optional[torch.Tensor] = None, table: Optional[torch.Tensor] = None,
            positions: Optional[torch.Tensor] = None, *, kind: str = "l2", eps: float = 1e-6,
            interleaved: bool = False, out_q: Optional[torch.Tensor] = None,
            out_k: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Every head of q and k over its norm, times a weight, its first channels
    rotated by position (``kda_qk_norm_fwd``): what ``chunk_fwd`` and
    ``decode_step`` expect of their q and k with ``kind="l2"`` alone.

    q: [..., Hq, d], k: [..., Hk, d], the same leading axes ([B, T] for a
    prompt, [B] for one token each), one dtype, d 64 or 128 (may be slices of
    wider rows); weights [d] fp32 or None; ``kind`` "l2" (root of the sum of
    squares) or "rms" (of their mean).  ``table`` [rows, rotary_dim] fp32 holds
    cos, then sin, of each position's angles and ``positions`` (int32, the
    leading axes' shape) the row of each token: any frequencies or scaling,
    rotary_dim a multiple of 16 up to d.  Pairs are (i, i + rotary_dim / 2), or
    (2 i, 2 i + 1) with ``interleaved``.  Returns (q', k').
    """
    dt = _dtype(q, "q")
    n, hq, hk, d, rot, rows, (qs, ks), lead = _qk_common(q, k, q_weight, k_weight, table,
                                                         positions, kind)
    out_q, oqs = _out_rows(out_q, "out_q", q, q.device, lead)
    out_k, oks = _out_rows(out_k, "out_k", k, q.device, lead)
    _call("kda_qk_norm_fwd", q.device, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
          _ptr(table), _ptr(positions), _ptr(out_q), _ptr(out_k), n, hq, hk, d, rot, rows, qs, ks,
          oqs, oks, eps, _NORMS[kind], int(bool(interleaved)), dt)
    return out_q, out_k


def qk_norm_bwd_workspace_size(tokens: int, q_heads: int, k_heads: int, head_dim: int) -> int:
    """Bytes of workspace ``qk_norm_bwd`` needs when it returns weights' gradients."""
    _sizes_fit("qk_norm_bwd", tokens, q_heads, k_heads, head_dim)
    n = lib().kda_qk_norm_bwd_workspace_size(tokens, q_heads, k_heads, head_dim)
    if n < 0:
        raise ValueError("invalid sizes")
    return int(n)


def qk_norm_bwd(q: torch.Tensor, k: torch.Tensor, d_out_q: torch.Tensor, d_out_k: torch.Tensor,
                q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                table: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None, *,
                kind: str = "l2", eps: float = 1e-6, interleaved: bool = False,
                workspace: Optional[torch.Tensor] = None, grads: Optional[dict] = None) -> dict:
    """Gradients of ``qk_norm`` (``kda_qk_norm_bwd``): a dict with dq, dk (dtype
    of q), dq_weight and dk_weight (fp32, None where there is no weight).
    ``grads`` may hold preallocated outputs, ``workspace`` a uint8 tensor of
    ``qk_norm_bwd_workspace_size`` bytes."""
    dt = _dtype(q, "q")
    n, hq, hk, d, rot, rows, (qs, ks), lead = _qk_common(q, k, q_weight, k_weight, table,
                                                         positions, kind)
    dev = q.device
    gqs = _rows(d_out_q, "d_out_q", q.dtype, q.shape, dev, lead)
    gks = _rows(d_out_k, "d_out_k", q.dtype, k.shape, dev, lead)
    g = dict(grads or {})
    g["dq"], dqs = _out_rows(g.get("dq"), "dq", q, dev, lead)
    g["dk"], dks = _out_rows(g.get("dk"), "dk", k, dev, lead)
    for name, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
        g[name] = None if w is None else _out(g.get(name), (d,), torch.float32, dev)
        _expect(g[name], name, torch.float32, (d,), dev)
    if q_weight is not None or k_weight is not None or workspace is not None:
        workspace = _workspace(workspace, lib().kda_qk_norm_bwd_workspace_size(n, hq, hk, d), dev)
    _call("kda_qk_norm_bwd", dev, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(table),
          _ptr(positions), _ptr(d_out_q), _ptr(d_out_k), _ptr(g["dq"]), _ptr(g["dk"]),
          _ptr(g["dq_weight"]), _ptr(g["dk_weight"]), n, hq, hk, d, rot, rows, qs, ks, gqs, gks,
          dqs, dks, eps, _NORMS[kind], int(bool(interleaved)), dt, _ptr(workspace),
          0 if workspace is None else workspace.numel())
    return g


# ---------------------------------------------------------------- state space scan
def _ssm_common(x, dt, A, B, C, D, lead):
    H, P = x.shape[lead:]
    if not isinstance(B, torch.Tensor) or B.dim() != lead + 2:
        raise ValueError("B must be [..., G, N] with the leading axes of x")
    G, N = B.shape[lead:]
    _fits(B, "B")
    dev, dtype = x.device, x.dtype
    if H % max(G, 1) or (H and not G):
        raise ValueError(f"{H} heads cannot share {G} groups of B and C")
    strides = (_rows(x, "x", dtype, x.shape, dev, lead),
               _rows(B, "B", dtype, (*x.shape[:lead], G, N), dev, lead),
               _rows(C, "C", dtype, (*x.shape[:lead], G, N), dev, lead))
    for t, name, shape in ((dt, "dt", x.shape[: lead + 1]), (A, "A", (H,))):
        if t is None:
            raise TypeError(f"{name} must be a tensor")
        _expect(t, name, torch.float32, shape, dev)
    _expect(D, "D", torch.float32, (H,), dev)
    return H, P, G, N, strides


def ssm_workspace_size(batch: int, seq_len: int, num_heads: int, head_dim: int, state_dim: int,
                       num_seqs: int = 0) -> int:
    """Bytes of workspace ``ssm_chunk_fwd`` needs (``num_seqs``: packed sequences,
    0 for a batch of equal rows)."""
    _sizes_fit("ssm_chunk_fwd", batch, seq_len, num_seqs, num_heads, head_dim, state_dim)
    n = lib().kda_ssm_chunk_fwd_workspace_size(batch, seq_len, num_seqs, num_heads, head_dim,
                                               state_dim)
    if n < 0:
        raise ValueError("invalid sizes")
    return int(n)


def ssm_chunk_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                  C: torch.Tensor, D: Optional[torch.Tensor] = None,
                  initial_state: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, *,
                  workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  final_state: Optional[torch.Tensor] = None, output_final_state: bool = True
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective state space scan over whole sequences (``kda_ssm_chunk_fwd``):
    S_t = exp(dt_t A) S_{t-1} + dt_t x_t B_t^T, y_t = S_t C_t + D x_t per head.

    x: [B, T, H, P], B, C: [B, T, G, N] float32 or bfloat16 (may be slices of
    wider rows), P and N 64 or 128, H a multiple of G (heads H / G * j .. share
    row j); dt: [B, T, H] fp32 as it enters the formula; A: [H], D: [H] or None,
    fp32, dt * A <= 0; initial_state: [n, H, P, N] fp32 or None; cu_seqlens as
    for ``chunk_fwd``.  Returns (out [B, T, H, P], final_state or None);
    ``final_state`` may be ``initial_state`` itself.
    """
    dtc = _dtype(x, "x")
    if x.dim() != 4:
        raise ValueError("x must be [B, T, H, P]")
    b, T = x.shape[:2]
    dev = x.device
    H, P, G, N, (xs, bs, cs) = _ssm_common(x, dt, A, B, C, D, 2)
    n = _num_seqs(cu_seqlens, b, dev)
    state = (n, H, P, N)
    _expect(initial_state, "initial_state", torch.float32, state, dev)
    out, os = _out_rows(out, "out", x, dev, 2)
    if final_state is None and output_final_state:
        final_state = torch.empty(state, dtype=torch.float32, device=dev)
    _expect(final_state, "final_state", torch.float32, state, dev)
    packed = n if cu_seqlens is not None else 0
    need = lib().kda_ssm_chunk_fwd_workspace_size(b, T, packed, H, P, N)
    ws = _workspace(workspace, max(need, 0), dev) if need or workspace is not None else None
    _call("kda_ssm_chunk_fwd", dev, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
          _ptr(initial_state), _ptr(cu_seqlens), _ptr(out), _ptr(final_state), b, T, H, G, P, N,
          xs, bs, cs, os, packed, dtc, _ptr(ws), 0 if ws is None else ws.numel())
    return out, final_state


def ssm_bwd_workspace_size(batch: int, seq_len: int, num_heads: int, num_groups: int,
                           head_dim: int, state_dim: int, dtype: torch.dtype,
                           num_seqs: int = 0) -> int:
    """Bytes of workspace ``ssm_chunk_bwd`` needs (``num_seqs``: packed sequences,
    0 for a batch of equal rows)."""
    _sizes_fit("ssm_chunk_bwd", batch, seq_len, num_seqs, num_heads, num_groups, head_dim, state_dim)
    n = lib().kda_ssm_chunk_bwd_workspace_size(batch, seq_len, num_seqs, num_heads, num_groups,
                                               head_dim, state_dim, _DTYPES[dtype])
    if n < 0:
        raise ValueError("invalid sizes")
    return int(n)


def ssm_chunk_bwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                  C: torch.Tensor, d_out: torch.Tensor, D: Optional[torch.Tensor] = None,
                  d_final_state: Optional[torch.Tensor] = None,
                  initial_state: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, *,
                  workspace: Optional[torch.Tensor] = None, grads: Optional[dict] = None,
                  output_initial_state_grad: bool = True) -> dict:
    """Gradients of ``ssm_chunk_fwd`` (``kda_ssm_chunk_bwd``): given dL/d out and
    dL/d final_state (None = zero), a dict with dx, dB, dC (dtype of x), ddt, dA,
    dD (fp32; dD None without D) and d_initial_state (fp32, or None when
    ``output_initial_state_grad`` is False).  ``grads`` may hold preallocated
    outputs, ``workspace`` a uint8 tensor of ``ssm_bwd_workspace_size`` bytes.
    """
    dtc = _dtype(x, "x")
    if x.dim() != 4:
        raise ValueError("x must be [B, T, H, P]")
    b, T = x.shape[:2]
    dev = x.device
    H, P, G, N, (xs, bs, cs) = _ssm_common(x, dt, A, B, C, D, 2)
    gs = _rows(d_out, "d_out", x.dtype, x.shape, dev, 2)
    n = _num_seqs(cu_seqlens, b, dev)
    state = (n, H, P, N)
    _expect(initial_state, "initial_state", torch.float32, state, dev)
    _expect(d_final_state, "d_final_state", torch.float32, state, dev)
    g = dict(grads or {})
    rows = []
    for name, like in (("dx", x), ("dB", B), ("dC", C)):
        g[name], row = _out_rows(g.get(name), name, like, dev, 2)
        rows.append(row)
    for name, shape in (("ddt", (b, T, H)), ("dA", (H,))):
        g[name] = _out(g.get(name), shape, torch.float32, dev)
        _expect(g[name], name, torch.float32, shape, dev)
    g["dD"] = None if D is None else _out(g.get("dD"), (H,), torch.float32, dev)
    _expect(g["dD"], "dD", torch.float32, (H,), dev)
    g.setdefault("d_initial_state", None)
    if g["d_initial_state"] is None and output_initial_state_grad:
        g["d_initial_state"] = torch.empty(state, dtype=torch.float32, device=dev)
    _expect(g["d_initial_state"], "d_initial_state", torch.float32, state, dev)
    packed = n if cu_seqlens is not None else 0
    need = lib().kda_ssm_chunk_bwd_workspace_size(b, T, packed, H, G, P, N, dtc)
    ws = _workspace(workspace, max(need, 0), dev)
    _call("kda_ssm_chunk_bwd", dev, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
          _ptr(initial_state), _ptr(cu_seqlens), _ptr(d_out), _ptr(d_final_state), _ptr(g["dx"]),
          _ptr(g["ddt"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
          _ptr(g["d_initial_state"]), b, T, H, G, P, N, xs, bs, cs, gs, *rows, packed, dtc,
          _ptr(ws), ws.numel())
    return g


def ssm_decode_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                    C: torch.Tensor, state: torch.Tensor, D: Optional[torch.Tensor] = None, *,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``ssm_chunk_fwd`` for one token per session (``kda_ssm_decode_step``): x
    [B, H, P], dt [B, H], B, C [B, G, N], state [B, H, P, N] fp32 updated in
    place.  Returns out [B, H, P]."""
    dtc = _dtype(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, H, P]")
    b, dev = x.shape[0], x.device
    H, P, G, N, (xs, bs, cs) = _ssm_common(x, dt, A, B, C, D, 1)
    if state is None:
        raise TypeError("state must be a tensor")
    _expect(state, "state", torch.float32, (b, H, P, N), dev)
    out, os = _out_rows(out, "out", x, dev, 1)
    _call("kda_ssm_decode_step", dev, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
          _ptr(state), _ptr(out), b, H, G, P, N, xs, bs, cs, os, dtc)
    return out
