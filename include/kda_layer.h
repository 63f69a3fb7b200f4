/*
 * kda_layer.h -- C ABI of libkda, the operators around the KDA recurrence of a
 * layer (AMD Instinct MI355X, gfx950, hand-written HIP):
 *
 *   - the short causal convolution that a layer's q, k and v (or x, B and C)
 *     pass through before the recurrence (kda_short_conv_*);
 *   - the per-head norm of queries and keys with the position rotation in the
 *     same pass (kda_qk_norm_*);
 *   - the selective state space scan, the recurrence with one decay per token
 *     and head and no delta rule (kda_ssm_*).
 *
 * Conventions shared by every entry point (those of kda.h, where both apply):
 *   - Status codes, element types (enum kda_dtype), packed sequences
 *     (cu_seqlens: a DEVICE int32 array of num_seqs + 1 offsets, 0 first, not
 *     decreasing, T last; NULL = batch rows of seq_len tokens), streams and the
 *     debug mode are as in kda.h.  Malformed offsets give wrong results, never
 *     an access out of bounds.  Tokens behind the last offset are in no
 *     sequence: their outputs are left as they were.
 *   - Tensors with one row per token may be slices of wider rows: `*_stride`
 *     is the distance in elements between consecutive tokens (token t of batch
 *     row b is row b * seq_len + t), at least the row's own length.  Everything
 *     else is dense.  Offsets are 64-bit; tokens are counted in 32 bits (batch *
 *     seq_len at most 2^31 - 4096).  A launch holds less than 2^32 threads: where
 *     millions of sequences, sessions or channels need more, the call is
 *     refused (KDA_ERR_UNSUPPORTED) before any work.
 *   - Parameters (weights, biases, A, D), dt and scan states are fp32; sums,
 *     norms and states are held in fp32; outputs are rounded once.
 *   - A workspace is the caller's, 16-byte aligned, of at least the size its
 *     `_workspace_size` returns (-1: invalid sizes).  Nothing in it has to
 *     survive a call and no call reads what an earlier one left.  Calls that
 *     may overlap in time (two streams, two captured graphs) need one each.
 *   - Nothing is allocated and no host memory is read after the call returns:
 *     every call may be captured into a graph.  Results do not depend on the
 *     order in which workgroups run.
 *   - An output must not overlap an input or another output (KDA_ERR_ALIAS)
 *     except where said.  Slices of one wider row (the same distance between
 *     tokens, columns beside each other) do not overlap.
 */
#ifndef KDA_LAYER_H_
#define KDA_LAYER_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation behind the short convolution. */
enum kda_activation { KDA_ACT_NONE = 0, KDA_ACT_SILU = 1 };

/* What kda_qk_norm_* divides a head by: the root of its sum of squares, or of
 * their mean. */
enum kda_norm { KDA_NORM_L2 = 0, KDA_NORM_RMS = 1 };

/*
 * kda_short_conv_fwd -- depthwise causal convolution of width 2, 3 or 4 with
 * an optional bias and activation:
 *     z[t,c] = bias[c] + sum_j weight[c,j] * r[t - (width - 1) + j, c],
 *     out[t,c] = z, or z * sigmoid(z) (KDA_ACT_SILU),
 * where r holds the sequence's rows x and, before its first token, the
 * width - 1 rows of initial_state (zeros when NULL).
 *
 *   x, out          [batch, seq_len, channels]      dtype (rows x_stride, out_stride apart)
 *   weight          [channels, width]               fp32
 *   bias            [channels] or NULL              fp32
 *   initial_state,
 *   final_state     [N, width - 1, channels] or NULL  dtype
 *
 * final_state receives the last width - 1 rows of (initial_state, x) of each
 * sequence, unrounded copies: a sequence shorter than that keeps rows of its
 * initial state, an empty one all of them.  Any number of channels; rows whose
 * starts and lengths are multiples of 16 bytes are read in 16-byte pieces.
 */
int kda_short_conv_fwd(const void *x, const float *weight, const float *bias,
                       const void *initial_state, const int32_t *cu_seqlens, void *out,
                       void *final_state, int32_t batch, int32_t seq_len, int32_t channels,
                       int32_t width, int64_t x_stride, int64_t out_stride, int32_t num_seqs,
                       int32_t activation, int32_t dtype, hipStream_t stream);

/*
 * kda_short_conv_bwd -- gradients of kda_short_conv_fwd for d_out (of out) and
 * d_final_state (of final_state; NULL = zero).  z is computed again from x.
 *   dx               [batch, seq_len, channels]        dtype
 *   dweight          [channels, width]                 fp32
 *   dbias            [channels] or NULL                fp32
 *   d_initial_state  [N, width - 1, channels] or NULL  dtype
 */
int kda_short_conv_bwd(const void *x, const float *weight, const float *bias,
                       const void *initial_state, const int32_t *cu_seqlens, const void *d_out,
                       const void *d_final_state, void *dx, float *dweight, float *dbias,
                       void *d_initial_state, int32_t batch, int32_t seq_len, int32_t channels,
                       int32_t width, int64_t x_stride, int64_t d_out_stride, int64_t dx_stride,
                       int32_t num_seqs, int32_t activation, int32_t dtype, void *workspace,
                       int64_t workspace_bytes, hipStream_t stream);
int64_t kda_short_conv_bwd_workspace_size(int32_t batch, int32_t seq_len, int32_t channels,
                                          int32_t width);

/*
 * kda_short_conv_step -- one token of each of `batch` sessions: out as above
 * from (state, x), then state moves on by one row, in place.
 *   x, out  [batch, channels] dtype;  state  [batch, width - 1, channels] dtype
 */
int kda_short_conv_step(const void *x, const float *weight, const float *bias, void *state,
                        void *out, int32_t batch, int32_t channels, int32_t width,
                        int64_t x_stride, int64_t out_stride, int32_t activation, int32_t dtype,
                        hipStream_t stream);

/*
 * kda_qk_norm_fwd -- every head of q and k divided by its norm, times a weight
 * per channel, then its first rotary_dim channels rotated by the token's
 * position, in one pass:
 *     y = x * weight / sqrt(ss + eps),  ss = sum x^2 (L2) or mean x^2 (RMS),
 *     (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin) for each pair i,
 * with pairs (a, b) = (i, i + rotary_dim / 2), or (2 i, 2 i + 1) when
 * interleaved != 0, i < rotary_dim / 2, and cos | sin taken from row
 * positions[token] of the table:
 *   q, out_q   [tokens, q_heads, head_dim]   dtype (rows *_stride apart)
 *   k, out_k   [tokens, k_heads, head_dim]   dtype; k_heads may be 0
 *   q_weight, k_weight  [head_dim] or NULL (ones)                fp32
 *   table      [table_rows, rotary_dim]: cos, then sin           fp32
 *   positions  [tokens]  int32; values outside the table are moved into it
 * Squares are summed in fp32 as they are: heads whose ss + eps is no normal fp32
 * number (a norm over 1.8e19, or under 1.1e-19 with eps = 0) are not divided right.
 * head_dim is 64 or 128; rotary_dim a multiple of 16, at most head_dim, 0 = no
 * rotation (table and positions are then not read).  Row starts of q, k and
 * the outputs and the table are 16-byte aligned.
 */
int kda_qk_norm_fwd(const void *q, const void *k, const float *q_weight, const float *k_weight,
                    const float *table, const int32_t *positions, void *out_q, void *out_k,
                    int32_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                    int32_t rotary_dim, int32_t table_rows, int64_t q_stride, int64_t k_stride,
                    int64_t out_q_stride, int64_t out_k_stride, float eps, int32_t norm,
                    int32_t interleaved, int32_t dtype, hipStream_t stream);

/*
 * kda_qk_norm_bwd -- gradients of kda_qk_norm_fwd for d_out_q and d_out_k,
 * from its inputs:
 *   dq, dk like q and k;  dq_weight, dk_weight [head_dim] fp32 or NULL.
 * The workspace is read only when a weight's gradient is asked for.
 */
int kda_qk_norm_bwd(const void *q, const void *k, const float *q_weight, const float *k_weight,
                    const float *table, const int32_t *positions, const void *d_out_q,
                    const void *d_out_k, void *dq, void *dk, float *dq_weight, float *dk_weight,
                    int32_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                    int32_t rotary_dim, int32_t table_rows, int64_t q_stride, int64_t k_stride,
                    int64_t d_out_q_stride, int64_t d_out_k_stride, int64_t dq_stride,
                    int64_t dk_stride, float eps, int32_t norm, int32_t interleaved,
                    int32_t dtype, void *workspace, int64_t workspace_bytes, hipStream_t stream);
int64_t kda_qk_norm_bwd_workspace_size(int32_t tokens, int32_t q_heads, int32_t k_heads,
                                       int32_t head_dim);

/*
 * kda_ssm_chunk_fwd -- the selective state space scan over whole sequences:
 * per head, with one decay per token,
 *     S_t = exp(dt_t A) S_{t-1} + dt_t x_t B_t^T,   y_t = S_t C_t + D x_t,
 * computed in blocks of 64 tokens (fp32 inputs: 32), in parallel inside a block
 * and, for long sequences, in several pieces at once.
 *
 *   x, out   [batch, seq_len, num_heads, head_dim]    dtype (rows *_stride apart)
 *   B, C     [batch, seq_len, num_groups, state_dim]  dtype (rows *_stride apart)
 *   dt       [batch, seq_len, num_heads]              fp32
 *   A        [num_heads] fp32;  D  [num_heads] fp32 or NULL (zero)
 *   initial_state, final_state  [N, num_heads, head_dim, state_dim] fp32
 *                               (the [.., d_v, d_k] layout of every state) or NULL
 *
 * Heads num_heads / num_groups * j .. share row j of B and C.  head_dim and
 * state_dim are 64 or 128 each.  dt and A are finite, dt * A <= 0 (any size: a
 * decay of zero included); a token with dt = 0 leaves the state as it is.
 * NaN and infinities in x, B or C reach what the formula says they reach (never
 * an earlier token, another sequence or, from x, another row of a head), but may
 * turn into NaN where it has an infinity.  Row starts of x, B, C and out are
 * 16-byte aligned, and 64 rows of each span less than 2^31 bytes.  final_state
 * may be initial_state itself.
 */
int64_t kda_ssm_chunk_fwd_workspace_size(int32_t batch, int32_t seq_len, int32_t num_seqs,
                                         int32_t num_heads, int32_t head_dim, int32_t state_dim);
int kda_ssm_chunk_fwd(const void *x, const float *dt, const float *A, const void *B,
                      const void *C, const float *D, const float *initial_state,
                      const int32_t *cu_seqlens, void *out, float *final_state, int32_t batch,
                      int32_t seq_len, int32_t num_heads, int32_t num_groups, int32_t head_dim,
                      int32_t state_dim, int64_t x_stride, int64_t b_stride, int64_t c_stride,
                      int64_t out_stride, int32_t num_seqs, int32_t dtype, void *workspace,
                      int64_t workspace_bytes, hipStream_t stream);

/*
 * kda_ssm_chunk_bwd -- gradients of kda_ssm_chunk_fwd for d_out (of out) and
 * d_final_state (of final_state; NULL = zero), from its inputs:
 *   dx  like x;  dB, dC  like B and C (summed over the heads that share a row)
 *   ddt [batch, seq_len, num_heads], dA [num_heads], dD [num_heads] or NULL  fp32
 *   d_initial_state like initial_state, or NULL
 * With a NaN or an infinity in an input, any gradient of its sequence and dA and
 * dD may be NaN.  The workspace holds the state at every block of 64 (fp32: 32)
 * tokens from both sides: about seq_len / 32 (fp32: seq_len / 16) states per head,
 * and one or two a sequence more when packed; beside them twice the forward's
 * workspace and, where a group's heads are split into sets, dB and dC in fp32 of
 * each set.
 */
int64_t kda_ssm_chunk_bwd_workspace_size(int32_t batch, int32_t seq_len, int32_t num_seqs,
                                         int32_t num_heads, int32_t num_groups, int32_t head_dim,
                                         int32_t state_dim, int32_t dtype);
int kda_ssm_chunk_bwd(const void *x, const float *dt, const float *A, const void *B,
                      const void *C, const float *D, const float *initial_state,
                      const int32_t *cu_seqlens, const void *d_out, const float *d_final_state,
                      void *dx, float *ddt, float *dA, void *dB, void *dC, float *dD,
                      float *d_initial_state, int32_t batch, int32_t seq_len, int32_t num_heads,
                      int32_t num_groups, int32_t head_dim, int32_t state_dim, int64_t x_stride,
                      int64_t b_stride, int64_t c_stride, int64_t d_out_stride,
                      int64_t dx_stride, int64_t db_stride, int64_t dc_stride, int32_t num_seqs,
                      int32_t dtype, void *workspace, int64_t workspace_bytes,
                      hipStream_t stream);

/*
 * kda_ssm_decode_step -- one token of each of `batch` sessions, the state
 * updated in place.  x, out [batch, num_heads, head_dim], B, C [batch,
 * num_groups, state_dim], dt [batch, num_heads], state [batch, num_heads,
 * head_dim, state_dim] fp32; everything else as above.
 */
int kda_ssm_decode_step(const void *x, const float *dt, const float *A, const void *B,
                        const void *C, const float *D, float *state, void *out, int32_t batch,
                        int32_t num_heads, int32_t num_groups, int32_t head_dim,
                        int32_t state_dim, int64_t x_stride, int64_t b_stride, int64_t c_stride,
                        int64_t out_stride, int32_t dtype, hipStream_t stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* KDA_LAYER_H_ */
