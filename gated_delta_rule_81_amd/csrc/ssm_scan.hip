// ssm_scan.hip -- the selective state space scan over whole sequences.
//
//   S_t = e^{dt_t A} S_{t-1} + dt_t x_t B_t^T,   y_t = S_t C_t + D x_t
//
// per head (S: P x N), B and C shared by the heads of a group.  In blocks of L
// tokens, with cum_t the sum of dt A from the block's first token to t,
//
//   y_t = sum_{s <= t} e^{cum_t - cum_s} (C_t . B_s) dt_s x_s + e^{cum_t} S0 C_t,
//   S_L = e^{cum_L} S0 + sum_s e^{cum_L - cum_s} dt_s x_s B_s^T,
//
// every exponent <= 0.  cum is summed in fp64, each step cut off at 2^-400 (which
// leaves nothing of any fp32 value): its differences are then exact to 2^-37
// whatever lies before them, so any dt A <= 0 is accepted.
//
// One workgroup walks the blocks of one (piece, head); wave w keeps the 16 state
// rows p = 16 w .. as fp32 accumulators of S^T tiles (N / 16 of them), which are
// the next block's operand as they stand.  A long sequence is cut into pieces
// that run at once: a first pass leaves each piece's own final state, a fold
// turns these into entering states (the transition of a piece is one number per
// head), and the second pass is the scan proper.  The first pass reads x and B
// once more and does 4 P N of the second's 4 P N + 2 L (P + N) operations a token.
#include "ssm_device.h"

#ifndef SCAN_OCC
#define SCAN_OCC (P == 64 && sizeof(T) == 2 ? 3 : 2)
#endif
#ifdef SCAN_SB
#define SB __builtin_amdgcn_sched_barrier(0)
#else
#define SB
#endif
namespace kda {
namespace {

enum Mode { kLocal, kOut, kStates };

// REV walks the blocks from the last to the first and the tokens' weights from
// the right: the gradient's recurrence E_{t-1} = e^{dt_t A} (E_t + x_t k_t^T).
template <typename T, int P, int N, int MODE, bool REV>
__global__ __launch_bounds__(P * 4, SCAN_OCC) void ssm_scan_kernel(SsmScan a) {
    constexpr int L = kSsmBlock<T>, NT = P * 4, NI = sizeof(T) == 2 ? 1 : 3;
    // Parts of y's fp32 operands, the block's weights M and the state: two for a
    // bf16 y (2^-15, nothing beside its own rounding), three for an fp32 one.
    constexpr int KM = sizeof(T) == 2 ? 2 : 3, KP = KM;
    constexpr bool OUT = MODE == kOut;
    typedef Tile<NI, L, N> TK;
    typedef Tile<NI, L, P> TX;
    typedef Tile<KM, L, L> TM;
    __shared__ __attribute__((aligned(16))) bf16 sk[TK::ELEMS];
    __shared__ __attribute__((aligned(16))) bf16 sc[OUT ? TK::ELEMS : 8];
    __shared__ __attribute__((aligned(16))) bf16 sx[TX::ELEMS];
    __shared__ __attribute__((aligned(16))) bf16 sm[OUT ? TM::ELEMS : 8];
    __shared__ __attribute__((aligned(16))) double s_cum[2][L];  // log2 of the decay up to t
    __shared__ __attribute__((aligned(16))) float s_dt[2][L], s_w[2][L], s_in[2][L];
    __shared__ double s_tot[2];

    const int64_t unit = xcd_unit(piece_count(a.seqs.total, a.seqs.num, a.piece) * a.heads);
    if (unit < 0) return;
    const int h = (int)(unit % a.heads);
    const int64_t number = unit / a.heads;
    const Piece pc = find_piece(a.seqs, number, a.piece);
    if (!pc.any) return;
    if (MODE == kLocal && (REV ? pc.first : pc.last)) return;  // nothing enters from it
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
    const RowsAt<TK> krow(lane);
    const RowsAt<TM> mrow(lane);
    int kcol[N / 16];
#pragma unroll
    for (int t = 0; t < N / 16; ++t) kcol[t] = cols_at<TK>(16 * t, lane);
    const int xcol = cols_at<TX>(16 * wave, lane);
    const int group = h / (a.heads / a.groups);
    const T *x = static_cast<const T *>(a.x) + (int64_t)h * P;
    const T *k = static_cast<const T *>(a.k) + (int64_t)group * N;
    const T *c = static_cast<const T *>(a.c) + (int64_t)group * N;
    const double A = (double)a.A[h] * kLog2eD;
    const int blocks = (pc.end - pc.beg + L - 1) / L;

    // S^T tiles: rows n = 16 t + 4 g + e, column p = 16 wave + r.  kStates, which
    // forms no outputs, keeps S tiles (rows p, column n = 16 t + r) instead: its
    // states are stored [N][P], four rows p a lane.
    f32x4 S[N / 16];
    constexpr bool TR = MODE == kStates;
    const int64_t lane_off = TR ? (int64_t)(16 * wave + 4 * g) * N + r
                                : (int64_t)(16 * wave + r) * N + 4 * g;
    const float *enter = nullptr;
    if (MODE != kLocal) {
        const bool edge = REV ? pc.last : pc.first;
        enter = a.seg_states && !edge
                    ? a.seg_states + (number * a.heads + h) * (int64_t)(P * N)
                    : (a.state0 ? a.state0 + ((int64_t)pc.seq * a.heads + h) * (P * N) : nullptr);
    }
#pragma unroll
    for (int t = 0; t < N / 16; ++t) {
        const float *at = enter + lane_off + 16 * t;
        S[t] = !enter ? zero4()
               : TR   ? f32x4{at[0], at[N], at[2 * N], at[3 * N]}
                      : *reinterpret_cast<const f32x4 *>(at);
    }

    Stage<T, L, N, NT> rk, rc;
    Stage<T, L, P, NT> rx;
    float rdt = 0.f;
    auto first_token = [&](int i) { return pc.beg + (REV ? blocks - 1 - i : i) * L; };
    auto load_rows = [&](int i) {
        const int t0 = first_token(i), n = pc.end - t0 < L ? pc.end - t0 : L;
        rk.load(k + t0 * a.k_stride, a.k_stride, n, tid);
        rx.load(x + t0 * a.x_stride, a.x_stride, n, tid);
        if constexpr (OUT) rc.load(c + t0 * a.c_stride, a.c_stride, n, tid);
    };
    auto load_dt = [&](int i) {  // lane = token; tokens past the end do nothing (dt = 0)
        const int t = first_token(i) + lane;
        rdt = lane < L && t < pc.end ? a.dt[(int64_t)t * a.heads + h] : 0.f;
    };
    double total = 0.0;
    auto weights = [&](int buf) {  // by the last wave
        const double step = (double)rdt * A;
        const double cum = wave_prefix(step < -400.0 ? -400.0 : step, lane);
        const double all = __shfl(cum, 63, 64);
        total += all;
        if (lane < L) {
            s_cum[buf][lane] = cum;
            s_dt[buf][lane] = rdt;
            s_in[buf][lane] = fast_exp2((float)cum);
            s_w[buf][lane] = REV ? fast_exp2((float)cum) : rdt * fast_exp2((float)(all - cum));
        }
        if (lane == 0) s_tot[buf] = all;
    };
    const bool weigher = wave == NT / 64 - 1;
    if (blocks > 0) {
        load_rows(0);
        if (weigher) {
            load_dt(0);
            weights(0);
        }
    }
    if constexpr (OUT) {  // tiles above the diagonal that a 32-wide step reads: zero for good
        for (int i = tid; i < TM::ELEMS; i += NT) sm[i] = static_cast<bf16>(0.f);
    }
    for (int i = 0; i < blocks; ++i) {
        const int buf = i & 1, t0 = first_token(i);
        rk.template store<TK>(sk, tid);
        rx.template store<TX>(sx, tid);
        if constexpr (OUT) rc.template store<TK>(sc, tid);
        lds_barrier();
        if (i + 1 < blocks) {
            load_rows(i + 1);
            if (weigher) load_dt(i + 1);
        }
        if constexpr (MODE == kStates) {
            const int64_t block = pc.seq_beg / L + pc.seq + (t0 - pc.seq_beg) / L;
            float *to = a.block_states + (block * a.heads + h) * (int64_t)(P * N) +
                        (int64_t)r * P + 16 * wave + 4 * g;
#pragma unroll
            for (int t = 0; t < N / 16; ++t)
                *reinterpret_cast<f32x4 *>(to + (int64_t)16 * t * P) = S[t];
        }
        f32x4 y[L / 16];
        const int ln = here(lane), r = ln & 15, g = ln >> 4;
        if constexpr (OUT) {
            // M[t][s] = e^{cum_t - cum_s} (C_t . B_s) dt_s, s <= t, formed as tiles of M^T
            int q = 0;
#pragma unroll
            for (int it = 0; it < L / 16; ++it)
#pragma unroll
                for (int is = 0; is <= it; ++is, ++q) {
                    if (q % (NT / 64) != wave) continue;
                    f32x4 m = zero4();
#pragma unroll
                    for (int ks = 0; ks < N / 32; ++ks)
                        m = mma(read_rows<TK, NI>(sk, 16 * is, ks, krow),
                                read_rows<TK, NI>(sc, 16 * it, ks, krow), m);
                    const int t = 16 * it + r, s = 16 * is + 4 * g;
                    const double ct = s_cum[buf][t];
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                    {
                        const float z = (float)(ct - s_cum[buf][s + e]);  // 0 above the diagonal
                        v[e] = m[e] * fast_exp2(s + e <= t ? z : -1e30f) * s_dt[buf][s + e];
                    }
#pragma unroll
                    for (int part = 0; part < KM; ++part) {
                        bf16x4 o;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float f = part < KM - 1 ? top_bits(v[e]) : v[e];
                            o[e] = static_cast<bf16>(f);
                            v[e] -= f;
                        }
                        *reinterpret_cast<bf16x4 *>(sm + part * TM::PLANE + TM::at(t, s)) = o;
                    }
                    SB;
                }
            // y^T = S C^T e^{cum}: rows p, columns t
#pragma unroll
            for (int it = 0; it < L / 16; ++it) y[it] = zero4();
#pragma unroll
            for (int ks = 0; ks < N / 32; ++ks) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = S[2 * ks][e], f[4 + e] = S[2 * ks + 1][e];
                const Parts<KP> sp = split<KP>(f);
#pragma unroll
                for (int it = 0; it < L / 16; ++it)
                    y[it] = mma(sp, read_rows<TK, NI>(sc, 16 * it, ks, krow), y[it]);
                SB;
            }
#pragma unroll
            for (int it = 0; it < L / 16; ++it) y[it] *= s_in[buf][16 * it + r];
            lds_barrier();
        }
        // x^T operands of this wave's rows p, and x^T weighted for the state
        Parts<NI> xt[L / 32];
        Parts<3> xw[L / 32];
#pragma unroll
        for (int ks = 0; ks < L / 32; ++ks) {
            xt[ks] = read_cols<TX, NI>(sx, ks, xcol);
            const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&s_w[buf][32 * ks + 4 * g]);
            const f32x4 w1 = *reinterpret_cast<const f32x4 *>(&s_w[buf][32 * ks + 16 + 4 * g]);
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = to_f32(xt[ks].v[0][e]);
                if constexpr (NI == 3) v += to_f32(xt[ks].v[1][e]) + to_f32(xt[ks].v[2][e]);
                f[e] = v * (e < 4 ? w0[e % 4] : w1[e % 4]);
            }
            xw[ks] = split<3>(f);
            SB;
        }
        if constexpr (OUT) {
            const int n = pc.end - t0;
            T *out = static_cast<T *>(a.out) + (int64_t)h * P + 16 * wave + 4 * g;
            const float D = a.D ? a.D[h] : 0.f;
#pragma unroll
            for (int it = 0; it < L / 16; ++it) {
#pragma unroll
                for (int ks = 0; ks <= it / 2; ++ks)
                    y[it] = mma(xt[ks], read_rows<TM, KM>(sm, 16 * it, ks, mrow), y[it]);
                const int t = 16 * it + r;
                if (a.D) {
                    const bf16 *row = sx + TX::at(t, 16 * wave + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = to_f32(row[e]);
                        if constexpr (NI == 3)
                            v += to_f32(row[TX::PLANE + e]) + to_f32(row[2 * TX::PLANE + e]);
                        y[it][e] += D * v;
                    }
                }
                if (t < n)
                    store4(out + (int64_t)(t0 + t) * a.out_stride, y[it][0], y[it][1], y[it][2],
                           y[it][3]);
                SB;
            }
        }
        const float decay = fast_exp2((float)s_tot[buf]);
#pragma unroll
        for (int t = 0; t < N / 16; ++t) {
            S[t] *= decay;
#pragma unroll
            for (int ks = 0; ks < L / 32; ++ks)
                S[t] = TR ? mma(xw[ks], read_cols<TK, NI>(sk, ks, kcol[t]), S[t])
                          : mma(read_cols<TK, NI>(sk, ks, kcol[t]), xw[ks], S[t]);
        }
        if (weigher && i + 1 < blocks) weights(buf ^ 1);
        lds_barrier();  // the tiles are read: the next block's may be written
    }
    float *to = nullptr;
    if (MODE == kLocal) {
        to = a.seg_states + (number * a.heads + h) * (int64_t)(P * N);
        if (weigher && lane == 0) a.seg_decay[number * a.heads + h] = total;
    } else if (a.final_state && (REV ? pc.first : pc.last)) {
        to = a.final_state + ((int64_t)pc.seq * a.heads + h) * (P * N);
    }
    if (to)
#pragma unroll
        for (int t = 0; t < N / 16; ++t) {
            float *at = to + lane_off + 16 * t;
            if constexpr (TR)
#pragma unroll
                for (int e = 0; e < 4; ++e) at[e * N] = S[t][e];
            else
                *reinterpret_cast<f32x4 *>(at) = S[t];
        }
}

// The pieces' own final states turned in place into entering states:
// enter[next] = e^{decay} enter + own.  One workgroup per 1024 values of a
// (sequence, head); the pieces one after the other, the next one's load ahead.
template <bool REV> __global__ __launch_bounds__(256) void ssm_fold_kernel(SsmScan a, int values) {
    const int per = values / 1024;
    const int64_t u = blockIdx.x / per;
    const int h = (int)(u % a.heads), n = (int)(u / a.heads);
    const int64_t off = (int64_t)(blockIdx.x % per) * 1024 + threadIdx.x * 4;
    const int beg = (int)seq_first_token(a.seqs.cu, a.seqs.seq_len, a.seqs.total, n);
    const int end = seq_end_token(a.seqs, n);
    const int count = end > beg ? (int)(((int64_t)end - beg + a.piece - 1) / a.piece) : 1;
    if (count < 2) return;
    const int64_t first = beg / a.piece + n;
    auto at = [&](int j) {
        return a.seg_states + ((first + (REV ? count - 1 - j : j)) * a.heads + h) * (int64_t)values + off;
    };
    f32x4 S = a.state0 ? *reinterpret_cast<const f32x4 *>(
                             a.state0 + ((int64_t)n * a.heads + h) * values + off)
                       : zero4();
    f32x4 own = *reinterpret_cast<const f32x4 *>(at(0));
    for (int j = 1; j < count; ++j) {
        const f32x4 now = own;
        if (j + 1 < count) own = *reinterpret_cast<const f32x4 *>(at(j));
        const double d = a.seg_decay[(first + (REV ? count - j : j - 1)) * a.heads + h];
        S = S * fast_exp2((float)d) + now;
        *reinterpret_cast<f32x4 *>(at(j)) = S;
    }
}

template <typename T, int P, int N, int MODE, bool REV>
void launch(const SsmScan &a, hipStream_t stream) {
    const int64_t units = piece_count(a.seqs.total, a.seqs.num, a.piece) * a.heads;
    hipLaunchKernelGGL((ssm_scan_kernel<T, P, N, MODE, REV>), dim3(xcd_blocks(units)), dim3(P * 4),
                       0, stream, a);
}

template <typename T, int P, int N> int scan(const SsmScan &args, int mode, hipStream_t stream) {
    SsmScan a = args;
    if (a.seg_states) {
        const int64_t folds = (int64_t)a.seqs.num * a.heads * (P * N / 1024);
        if (mode == kSsmStatesRev) {
            launch<T, P, N, kLocal, true>(a, stream);
            hipLaunchKernelGGL((ssm_fold_kernel<true>), dim3((unsigned)folds), dim3(256), 0, stream,
                               a, P * N);
        } else {
            launch<T, P, N, kLocal, false>(a, stream);
            hipLaunchKernelGGL((ssm_fold_kernel<false>), dim3((unsigned)folds), dim3(256), 0,
                               stream, a, P * N);
        }
    }
    if (mode == kSsmOut)
        launch<T, P, N, kOut, false>(a, stream);
    else if (mode == kSsmStates)
        launch<T, P, N, kStates, false>(a, stream);
    else
        launch<T, P, N, kStates, true>(a, stream);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T> int scan_dims(const SsmScan &a, int mode, hipStream_t stream) {
    if (a.p == 64)
        return a.n == 64 ? scan<T, 64, 64>(a, mode, stream) : scan<T, 64, 128>(a, mode, stream);
    return a.n == 64 ? scan<T, 128, 64>(a, mode, stream) : scan<T, 128, 128>(a, mode, stream);
}

}  // namespace

int launch_ssm_scan(const SsmScan &a, int mode, int dtype, hipStream_t stream) {
    return dtype == kDtypeBf16 ? scan_dims<bf16>(a, mode, stream)
                               : scan_dims<float>(a, mode, stream);
}

}  // namespace kda
