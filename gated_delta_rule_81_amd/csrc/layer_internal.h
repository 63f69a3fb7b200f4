// layer_internal.h -- host-side launch functions of the operators around the
// recurrence (not part of the public ABI; see include/kda_layer.h).  Arguments
// are already validated.  Each returns 0, or -1 if a launch failed.
#pragma once

#include "kda_internal.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// Sequences of a call: num_seqs rows of seq_len tokens (cu == NULL), or the
// packed offsets cu; total tokens in all.
struct Seqs {
    const int32_t *cu;
    int32_t num, seq_len, total;
};

// Pieces of `len` tokens of the sequences.  Equal rows: piece j of row n has
// number n * per + j.  Packed: t0 / len + n + j, t0 the sequence's first token,
// so that numbers of different sequences never meet whatever the offsets hold
// (some belong to none).  An empty sequence has one (empty) piece.
__host__ __device__ inline int64_t pieces_per_row(const Seqs &q, int64_t len) {
    return q.seq_len > 0 ? (q.seq_len + len - 1) / len : 1;
}
__host__ __device__ inline int64_t piece_count(const Seqs &q, int64_t len) {
    return q.cu ? q.total / len + q.num + 1 : q.num * pieces_per_row(q, len);
}
__host__ __device__ inline int64_t first_piece(const Seqs &q, int64_t len, int64_t t0, int n) {
    return q.cu ? t0 / len + n : n * pieces_per_row(q, len);
}

// Places for the states of pieces, for sequences of two and more only.  Equal rows:
// the piece's number.  Packed: floor(2 t0 / len) + j.  A sequence of T > len tokens
// takes ceil(T / len) <= floor(2 T / len) places, so the next one's begin behind them
// and all are under 2 total / len, however many short sequences there are.
__host__ __device__ inline int64_t slot_count(const Seqs &q, int64_t len) {
    return q.cu ? 2 * (int64_t)q.total / len : q.num * pieces_per_row(q, len);
}
__host__ __device__ inline int64_t first_slot(const Seqs &q, int64_t len, int64_t t0, int n) {
    return q.cu ? 2 * t0 / len : n * pieces_per_row(q, len);
}

struct ConvArgs {
    const void *x, *state0, *d_out, *d_final;
    const float *weight, *bias;
    void *out, *final_state, *dx, *d_state0;
    float *dweight, *dbias, *partial;
    Seqs seqs;
    int32_t channels, width, silu, dtype;
    int64_t x_stride, out_stride, d_out_stride, dx_stride;
};
// Threads of a call's largest launch, which holds kMostThreads at most.
constexpr int64_t kMostThreads = UINT32_MAX;
int64_t conv_fwd_threads(const ConvArgs &a);
int64_t conv_bwd_threads(const ConvArgs &a);
int64_t conv_step_threads(const ConvArgs &a, const void *state, int32_t batch);
int launch_conv_fwd(const ConvArgs &a, hipStream_t stream);
int launch_conv_bwd(const ConvArgs &a, hipStream_t stream);
int64_t conv_bwd_workspace_floats(int64_t total, int64_t channels, int width);
int launch_conv_step(const ConvArgs &a, void *state, int32_t batch, hipStream_t stream);

struct QkArgs {
    const void *x[2], *dy[2];    // q, k and the gradients of their outputs
    void *y[2];                  // outputs, or dq and dk
    const float *weight[2];
    float *dweight[2], *partial;
    const float *table;
    const int32_t *positions;
    int32_t tokens, heads[2], head_dim, rot, table_rows;
    int64_t x_stride[2], dy_stride[2], y_stride[2];
    float eps;
    int32_t rms, interleaved, dtype;
};
int launch_qk_norm_fwd(const QkArgs &a, hipStream_t stream);
int launch_qk_norm_bwd(const QkArgs &a, hipStream_t stream);
int64_t qk_norm_bwd_workspace_floats(int64_t tokens, int64_t q_heads, int64_t k_heads,
                                     int head_dim);

// The scan's walk over the sequences.  With seg_states the sequences are cut into
// pieces of `piece` tokens that run at once (seg_states: a state per slot and
// head, seg_decay: a double each); without, `piece` is at least every sequence's
// length.
struct SsmScan {
    const void *x, *k, *c;
    const float *dt, *A, *D, *state0;
    void *out;
    float *final_state, *seg_states, *block_states;
    double *seg_decay;
    Seqs seqs;
    int32_t heads, groups, p, n, piece;
    int64_t x_stride, k_stride, c_stride, out_stride;
};
// Threads of the largest launch of launch_ssm_out (directions = 1) or
// launch_ssm_states (2).
int64_t ssm_scan_threads(const SsmScan &a, int dtype, int directions);
// y and the final states.
int launch_ssm_out(const SsmScan &a, int dtype, hipStream_t stream);
// The state entering every block to a.block_states; and from the right, to
// b.block_states, the loss gradient of the state behind every block (b: x =
// d_out, k = C, state0 = d_final_state, final_state = d_initial_state; pieces of
// its own).  a and b differ in nothing else.
int launch_ssm_states(const SsmScan &a, const SsmScan &b, int dtype, hipStream_t stream);

// The gradients from the states entering every block (s_states) and the loss
// gradients behind every block (e_states), both [block number][head][n][p]:
// a.blocks block numbers of 64 (bf16) or 32 tokens.  The heads of a group are
// worked on in `sets` sets; part_bc (sets > 1): dB and dC of each set, fp32
// [set][2][token][group][n]; part_a, part_d: [block number][head].
struct SsmGrad {
    const void *x, *B, *C, *dy;
    const float *dt, *A, *D, *s_states, *e_states;
    void *dx, *dB, *dC;
    float *ddt, *dA, *dD, *part_a, *part_d, *part_bc;
    Seqs seqs;
    int32_t heads, groups, p, n, sets;
    int64_t blocks, x_stride, b_stride, c_stride, dy_stride, dx_stride, db_stride, dc_stride;
};
int64_t ssm_grad_threads(const SsmGrad &a);
int launch_ssm_grad(const SsmGrad &a, int dtype, hipStream_t stream);

struct SsmStep {
    const void *x, *B, *C;
    const float *dt, *A, *D;
    float *state;
    void *out;
    int32_t batch, heads, groups, p, n;
    int64_t x_stride, b_stride, c_stride, out_stride;
};
constexpr int kSsmStepThreads = 256;  // of a workgroup; one per session and head
int launch_ssm_step(const SsmStep &a, int dtype, hipStream_t stream);

}  // namespace kda
