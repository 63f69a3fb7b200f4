"""Kimi Delta Attention (KDA) forward on AMD Instinct MI355X (gfx950).

Python front end of ``libkda.so``; the C ABI is declared in include/kda.h.

    out, final_state = chunk_fwd(q, k, v, log_alpha, beta, initial_state, cu_seqlens)
    out, final_state, snapshots = chunk_fwd_snapshots(q, k, v, log_alpha, beta, every)
    out = decode_step(q, k, v, log_alpha, beta, state)   # state updated in place
    grads = chunk_bwd(q, k, v, log_alpha, beta, d_out, d_final_state, initial_state)

The operators around the recurrence (include/kda_layer.h):

    out, rows = short_conv(x, weight, bias, initial_state, cu_seqlens)
    q, k = qk_norm(q, k, q_weight, k_weight, table, positions)
    out, final_state = ssm_chunk_fwd(x, dt, A, B, C, D, initial_state, cu_seqlens)
    out = ssm_decode_step(x, dt, A, B, C, state, D)      # state updated in place
"""
from ._lib import KdaError, lib
from .layer import (qk_norm, qk_norm_bwd, qk_norm_bwd_workspace_size, short_conv, short_conv_bwd,
                    short_conv_bwd_workspace_size, short_conv_step, ssm_bwd_workspace_size,
                    ssm_chunk_bwd, ssm_chunk_fwd, ssm_decode_step, ssm_workspace_size)
from .ops import (bwd_workspace_size, chunk_bwd, chunk_fwd, chunk_fwd_segmented,
                  chunk_fwd_segmented_noalloc, chunk_fwd_snapshots, decode_step,
                  segmented_workspace_size)

__all__ = ["chunk_fwd", "chunk_fwd_segmented", "chunk_fwd_segmented_noalloc",
           "chunk_fwd_snapshots", "chunk_bwd", "decode_step", "segmented_workspace_size",
           "bwd_workspace_size", "short_conv", "short_conv_bwd",
           "short_conv_bwd_workspace_size", "short_conv_step", "qk_norm", "qk_norm_bwd",
           "qk_norm_bwd_workspace_size", "ssm_chunk_fwd", "ssm_chunk_bwd", "ssm_decode_step",
           "ssm_workspace_size", "ssm_bwd_workspace_size", "KdaError", "lib"]
