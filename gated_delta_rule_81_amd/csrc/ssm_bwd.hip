// ssm_bwd.hip -- gradients of the state space scan.
//
// With S0 the state entering a block of L tokens, E the loss gradient of the
// state behind it, G = C B^T, dP = dY X^T (both L x L) and L_ts = e^{cum_t - cum_s},
// s <= t (ssm_scan.hip):
//   du_s = e^{cum_L - cum_s} E B_s + sum_t G_ts L_ts dy_t,    dx = dt du + D dy
//   dC_t = e^{cum_t} S0^T dy_t + sum_s Q_ts B_s,   Q_ts = dP_ts L_ts dt_s
//   dB_s = dt_s e^{cum_L - cum_s} E^T x_s + sum_t Q_ts C_t
//   dl_r = sum_{s < r <= t} G_ts Q_ts + sum_{t >= r} z_t + sum_{s < r} v_s
//          + e^{cum_L} <E, S0>            (l_r = dt_r A)
//     z_t = e^{cum_t} dy_t . S0 C_t,  v_s = dt_s e^{cum_L - cum_s} x_s . E B_s
//   ddt = x . du + A dl,  dA = sum dt dl,  dD = sum x . dy
// dB and dC summed over the heads of the group.  dl adds the pairs that l_r
// stands between: no term is added and taken away again, so it is exact at any
// decay (as a suffix sum of dy y - u du it would lose e^-l of its digits).
//
// Three steps.  The scan (ssm_scan.hip) writes S0 of every block, then, from the
// right, E of every block, both fp32 and transposed ([N][P]).  Then one
// workgroup per (block, group, set of heads) loops over its heads with dB and dC
// in registers: 8 waves, each the owner of 16 columns n of dB and dC and of a
// 16-token s-tile of du.  dP and M stay in its registers; in LDS lie G (fp32, the
// same for all heads of the group), and, as bf16 parts, Q (for dB's and dC's
// waves) and E (read by columns n, needed by rows too).  A head of 128 rows is
// two of 64 that share dt and A: every sum above is linear in the rows.
//
// 2 x 4096 tokens x 64 heads of 64 x 128 bf16, 0.29 GB of inputs and gradients:
// 550 us a call; in a trace of warm calls pieces 60, fold 17, states 161 (writes
// 1.07 GB of block states and reads the inputs once), gradients 308, dA and dD 4.6.
// HBM bounds the states pass.  In the gradient kernel VALU issues in 45% of the
// cycles, LDS works in 29% and the matrix unit in 17%; its waves wait 45% of their
// time, at two barriers a head and for LDS, with one workgroup of 8 waves a CU, the most that
// 145 KB of LDS and 230 registers leave.  Fewer VALU instructions do not help it
// (weights below the diagonal as products, as the scan has them: 538 us where 534
// stood).  fp32: 992 us.
#include "ssm_device.h"

namespace kda {
namespace {

constexpr int kPB = 64;        // state rows a workgroup works on at a time
constexpr int kGradWaves = 8;

template <typename T, int N>
__global__ __launch_bounds__(kGradWaves * 64) void ssm_grad_kernel(SsmGrad a) {
    constexpr int L = kSsmBlock<T>, NT = kGradWaves * 64, NI = sizeof(T) == 2 ? 1 : 3;
    constexpr int KQ = 3;                        // parts of Q (2: 535 us where 3 take 549)
    constexpr int TL = L / 16, PT = TL / 2;      // token tiles; row tiles of du a wave owns
    constexpr int NTN = N / 16, TG = kGradWaves / NTN, TPW = TL / TG;  // tiles of dB, dC a wave owns
    constexpr int KT = L / 32;                   // 32-wide steps over tokens
    constexpr int PG = kGradWaves / TL;          // waves of one s-tile
    typedef Tile<NI, L, N> TK;
    typedef Tile<NI, L, kPB> TX;
    typedef Tile<KQ, L, L> TQ;
    typedef Tile<3, N, kPB> TE;
    __shared__ __attribute__((aligned(16))) bf16 sb[TK::ELEMS];
    __shared__ __attribute__((aligned(16))) bf16 sc[TK::ELEMS];
    __shared__ __attribute__((aligned(16))) bf16 sx[TX::ELEMS];
    __shared__ __attribute__((aligned(16))) bf16 sy[TX::ELEMS];
    __shared__ __attribute__((aligned(16))) bf16 sq[TQ::ELEMS];  // Q^T: [s][t]
    __shared__ __attribute__((aligned(16))) bf16 se[TE::ELEMS];  // E: [n][p]
    // of three heads: the one worked on, the next, and the one whose sums are left
    __shared__ __attribute__((aligned(16))) double s_cum[3][L];
    __shared__ __attribute__((aligned(16))) float s_dt[3][L], s_out[3][L], s_in[3][L];
    __shared__ __attribute__((aligned(16))) float s_g[TL * (TL + 1) / 2][64][4];  // G's tiles
    __shared__ float s_all[3], s_D[3], s_A[3];
    // the waves' shares of ddt, dA and dD, of two heads
    __shared__ float s_pair[2][TL][L], s_z[2][NTN][L], s_xdu[2][PG][L], s_v[2][PG][L];
    __shared__ float s_k[2][NTN], s_d[2][TL];

    const int64_t unit = blockIdx.x;
    const int set = (int)(unit % a.sets), group = (int)(unit / a.sets % a.groups);
    const int64_t number = unit / a.sets / a.groups;
    const int per_group = a.heads / a.groups, per_set = (per_group + a.sets - 1) / a.sets;
    const int h0 = group * per_group + set * per_set;
    const int h1 = set * per_set + per_set < per_group ? h0 + per_set : (group + 1) * per_group;
    const Piece pc = find_piece(a.seqs, number, L);
    const int tid = threadIdx.x, lane0 = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = lane0, r = lane & 15, g = lane >> 4;
    const int n = pc.any ? pc.end - pc.beg : 0, t0 = pc.beg;
    if (n <= 0) {  // no token: nothing to add to dA and dD
        for (int h = h0 + tid; h < h1; h += NT) {
            a.part_a[number * a.heads + h] = 0.f;
            a.part_d[number * a.heads + h] = 0.f;
        }
        return;
    }
    const int P = a.p, halves = P / kPB;
    const int count = (h1 > h0 ? h1 - h0 : 0) * halves;  // (head, 64 of its rows) to work on
    // s-tile and row tiles of du.  An early s-tile has more tiles below it: the
    // two waves of a SIMD (w, w + 4) take one from either end.
    const int is = wave & 4 ? TL - 1 - wave % TL : wave % TL, pg = wave / TL;
    const int nt = wave % NTN, tg = wave / NTN;  // columns and token tiles of dB, dC
    // of the waves with the last s-tile, one forms the next head's decays and one
    // adds up the last head's shares
    const bool weigher = wave == 3, summer = wave == 4;

    const T *x = static_cast<const T *>(a.x) + t0 * a.x_stride;
    const T *dy = static_cast<const T *>(a.dy) + t0 * a.dy_stride;
    Stage<T, L, kPB, NT> rx, ry;
    auto load_rows = [&](int i) {
        const int64_t off = (int64_t)(h0 + i / halves) * P + (i % halves) * kPB;
        rx.load(x + off, a.x_stride, n, tid);
        ry.load(dy + off, a.dy_stride, n, tid);
    };
    // operand of index n (columns 16 nt ..), k = rows p (read_wide's order), of a state
    // stored [N][P]
    auto load_state = [&](const float *states, int i, float (&f)[kPB / 32][8]) {
        const float *at = states + (number * a.heads + h0 + i / halves) * (int64_t)(P * N) +
                          (int64_t)(16 * nt + r) * P + (i % halves) * kPB + 8 * g;
#pragma unroll
        for (int ks = 0; ks < kPB / 32; ++ks)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const f32x4 v = __builtin_nontemporal_load(
                    reinterpret_cast<const f32x4 *>(at + 32 * ks + 4 * q));
#pragma unroll
                for (int e = 0; e < 4; ++e) f[ks][4 * q + e] = v[e];
            }
    };
    float rdt = 0.f, rA = 0.f, rD = 0.f;  // the weigher's head
    auto load_dt = [&](int i) {
        const int h = h0 + i / halves;
        rdt = lane < n ? a.dt[(int64_t)(t0 + lane) * a.heads + h] : 0.f;
        rA = a.A[h];
        rD = a.D ? a.D[h] : 0.f;
    };
    auto weights = [&](int buf) {
        const double step = (double)rdt * ((double)rA * kLog2eD);
        const double cum = wave_prefix(step < -400.0 ? -400.0 : step, lane);
        const double all = from_lane(cum, 63);
        if (lane < L) {
            s_cum[buf][lane] = cum;
            s_dt[buf][lane] = rdt;
            s_in[buf][lane] = fast_exp2((float)cum);
            s_out[buf][lane] = fast_exp2((float)(all - cum));
        }
        if (lane == 0) s_all[buf] = fast_exp2((float)all), s_D[buf] = rD, s_A[buf] = rA;
    };
    float ev[kPB / 32][8], sv[kPB / 32][8], kdot = 0.f;
    auto store_e = [&]() {  // E's parts to LDS, and this wave's share of <E, S0>
        kdot = 0.f;
#pragma unroll
        for (int ks = 0; ks < kPB / 32; ++ks) {
#pragma unroll
            for (int e = 0; e < 8; ++e) kdot += ev[ks][e] * sv[ks][e];
            const Parts<3> ep = split<3>(ev[ks]);
            if (tg == 0)
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    *reinterpret_cast<bf16x8 *>(se + q * TE::PLANE +
                                                TE::at(16 * nt + r, 32 * ks + 8 * g)) = ep.v[q];
        }
    };

    // the group's rows, and the first head's
    {
        Stage<T, L, N, NT> rb, rc;
        rb.load(static_cast<const T *>(a.B) + t0 * a.b_stride + (int64_t)group * N, a.b_stride, n, tid);
        rc.load(static_cast<const T *>(a.C) + t0 * a.c_stride + (int64_t)group * N, a.c_stride, n, tid);
        if (count > 0) {
            load_rows(0);
            load_state(a.e_states, 0, ev);
            load_state(a.s_states, 0, sv);
            if (weigher) load_dt(0);
        }
        rb.template store<TK>(sb, tid);
        rc.template store<TK>(sc, tid);
        for (int i = tid; i < TQ::ELEMS; i += NT) sq[i] = static_cast<bf16>(0.f);
        if (count > 0) {
            rx.template store<TX>(sx, tid);
            ry.template store<TX>(sy, tid);
            store_e();
            if (weigher) weights(0);
        }
    }
    lds_barrier();

    // G's tiles it >= is (rows t = 16 it + 4 g + e, column s = 16 is + r), by lane
    auto tile_of = [](int it, int js) { return it * (it + 1) / 2 + js; };
    {
        const WideAt<TK> kwide(lane);
#pragma unroll
        for (int it = 0; it < TL; ++it) {
            if (it < is || pg != it % PG) continue;
            f32x4 v = zero4();
#pragma unroll
            for (int ks = 0; ks < N / 32; ++ks)
                v = mma(read_wide<TK, NI>(sc, 16 * it, ks, kwide),
                        read_wide<TK, NI>(sb, 16 * is, ks, kwide), v);
            *reinterpret_cast<f32x4 *>(s_g[tile_of(it, is)][lane]) = v;
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    lds_barrier();
    f32x4 dB[TPW], dC[TPW];  // rows n = 16 nt + 4 g + e, column token 16 (tg TPW + i) + r
#pragma unroll
    for (int i = 0; i < TPW; ++i) dB[i] = dC[i] = zero4();
    // Head i's shares added up: ddt, and its parts of dA and dD (by the summer; over
    // the head's halves in registers).
    float sum_dl = 0.f, sum_xdu = 0.f, sum_d = 0.f;
    auto add_up = [&](int i) {
        const int buf = i % 3, par = i & 1, h = h0 + i / halves;
        float dl = 0.f, xdu = 0.f, z = 0.f, v = 0.f, k = 0.f, d = 0.f;
        if (lane < L) {
#pragma unroll
            for (int q = 0; q < TL; ++q) dl += q <= lane / 16 ? s_pair[par][q][lane] : 0.f;
#pragma unroll
            for (int q = 0; q < NTN; ++q) z += s_z[par][q][lane];
#pragma unroll
            for (int q = 0; q < PG; ++q) xdu += s_xdu[par][q][lane], v += s_v[par][q][lane];
        }
#pragma unroll
        for (int q = 0; q < NTN; ++q) k += s_k[par][q];
#pragma unroll
        for (int q = 0; q < TL; ++q) d += s_d[par][q];
        z = wave_suffix(z, lane);
        v = __shfl_up(wave_prefix(v, lane), 1, 64);
        dl += z + (lane > 0 ? v : 0.f) + s_all[buf] * k;
        const bool fresh = i % halves == 0;
        sum_dl = fresh ? dl : sum_dl + dl;
        sum_xdu = fresh ? xdu : sum_xdu + xdu;
        sum_d = fresh ? d : sum_d + d;
        if (i % halves != halves - 1) return;
        if (lane < n) a.ddt[(int64_t)(t0 + lane) * a.heads + h] = sum_xdu + s_A[buf] * sum_dl;
        const float tot = rows4_sum(row16_total(lane < n ? s_dt[buf][lane] * sum_dl : 0.f));
        if (lane == 0) {
            a.part_a[number * a.heads + h] = tot;
            a.part_d[number * a.heads + h] = sum_d;
        }
    };

    // The waves with more tiles below their s-tile issue first: the barriers wait for
    // them (539 us without, 534 with).
    if (is == 0)
        __builtin_amdgcn_s_setprio(3);
    else if (is == 1)
        __builtin_amdgcn_s_setprio(2);
    else if (is == 2)
        __builtin_amdgcn_s_setprio(1);
    for (int i = 0; i < count; ++i) {
        const int buf = i % 3, par = i & 1, h = h0 + i / halves;
        const bool more = i + 1 < count;
        lane = here(lane0), r = lane & 15, g = lane >> 4;
        const RowsAt<TK> krow(lane);
        const WideAt<TX> xwide(lane);
        // ---- phase A: everything but the products with Q
        {   // dC_t += e^{cum_t} S0^T dy_t and z_t;  dB_s += dt_s e^{cum_L - cum_s} E^T x_s
            Parts<3> sp[kPB / 32], ep[kPB / 32];
            const WideAt<TE> ewide(lane);
#pragma unroll
            for (int ks = 0; ks < kPB / 32; ++ks) {
                sp[ks] = split<3>(sv[ks]);
                ep[ks] = read_wide<TE, 3>(se, 16 * nt, ks, ewide);
            }
            if (more) {
                load_rows(i + 1);
                if (weigher) load_dt(i + 1);
            }
#pragma unroll
            for (int q = 0; q < TPW; ++q) {
                const int it = tg * TPW + q, t = 16 * it + r;
                f32x4 u = zero4(), v = zero4();
#pragma unroll
                for (int ks = 0; ks < kPB / 32; ++ks) {
                    u = mma(sp[ks], read_wide<TX, NI>(sy, 16 * it, ks, xwide), u);
                    v = mma(ep[ks], read_wide<TX, NI>(sx, 16 * it, ks, xwide), v);
                }
                const float win = s_in[buf][t];
                const bf16 *row = sc + TK::at(t, 16 * nt + 4 * g);
                float z = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float cv = to_f32(row[e]);
                    if constexpr (NI == 3)
                        cv += to_f32(row[TK::PLANE + e]) + to_f32(row[2 * TK::PLANE + e]);
                    u[e] *= win;
                    z += u[e] * cv;
                }
                z = rows4_sum(z);
                if (g == 0) s_z[par][nt][t] = z;
                dC[q] += u;
                dB[q] += v * (s_out[buf][t] * s_dt[buf][t]);
            }
            const float ks = rows4_sum(row16_total(kdot));
            if (tg == 0 && lane == 0) s_k[par][nt] = ks;
            // E's loads here and S0's after the pairs: both there 547 us, both here 566
            if (more) load_state(a.e_states, i + 1, ev);
        }
        {   // this wave's s-tile: dP, M, Q, the pairs, and du
            const int s = 16 * is + r;
            const double cs = s_cum[buf][s];
            const float dts = s_dt[buf][s];
            Parts<3> mp[KT];
            float mf[8], diag = 0.f, tail = 0.f;  // tail: pairs of the tiles below, per column s
#pragma unroll
            for (int it = TL - 1; it >= 0; --it) {
                float *m = mf + 4 * (it % 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e] = 0.f;
                if (it >= is) {
                    f32x4 dp = zero4();
#pragma unroll
                    for (int ks = 0; ks < kPB / 32; ++ks)
                        dp = mma(read_wide<TX, NI>(sy, 16 * it, ks, xwide),
                                 read_wide<TX, NI>(sx, 16 * is, ks, xwide), dp);
                    const f32x4 G = *reinterpret_cast<const f32x4 *>(s_g[tile_of(it, is)][lane]);
                    float qv[4], w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = 16 * it + 4 * g + e;
                        const float z = (float)(s_cum[buf][t] - cs);
                        const float d = fast_exp2(s <= t ? z : -1e30f);  // 0 above the diagonal
                        diag += s == t ? dp[e] : 0.f;  // of tile it == is
                        qv[e] = dp[e] * d * dts;
                        m[e] = G[e] * d;
                        w[e] = G[e] * qv[e];
                    }
                    // Q to LDS, and the pairs: the sum over t' >= t of a column, then over
                    // the columns s < t.  The waves of an s-tile take its tiles in turn.
#pragma unroll
                    for (int e = 2; e >= 0; --e) w[e] += w[e + 1];
                    float v[4];
                    rows4_gather(w[0], v);
                    const float below = (g < 1 ? v[1] : 0.f) + (g < 2 ? v[2] : 0.f) +
                                        (g < 3 ? v[3] : 0.f) + tail;
                    tail += v[0] + v[1] + v[2] + v[3];
                    if (pg == it % PG) {
                        store_parts<TQ::PLANE>(sq + TQ::at(s, 16 * it + 4 * g), qv);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = 16 * it + 4 * g + e;
                            const float sum = row16_total(s < t ? w[e] + below : 0.f);
                            if (r == 0) s_pair[par][is][t] = sum;
                        }
                    }
                }
                if (it % 2 == 0) mp[it / 2] = split<3>(mf);
            }
            diag = rows4_sum(row16_total(diag));
            if (pg == 0 && lane == 0) s_d[par][is] = diag;
            if (more) {
                load_state(a.s_states, i + 1, sv);
                if (weigher) weights((i + 1) % 3);
            }
            if (summer && i > 0) add_up(i - 1);
            float xdu = 0.f, vs = 0.f;
            const float wout = s_out[buf][s], D = s_D[buf];
            T *dx = static_cast<T *>(a.dx) + (int64_t)(t0 + s) * a.dx_stride + (int64_t)h * P +
                    (i % halves) * kPB;
#pragma unroll
            for (int q = 0; q < PT; ++q) {
                const int pt = pg * PT + q;
                f32x4 du = zero4();
#pragma unroll
                for (int ks = 0; ks < N / 32; ++ks)
                    du = mma(read_cols<TE, 3>(se, ks, cols_at<TE>(16 * pt, lane)),
                             read_rows<TK, NI>(sb, 16 * is, ks, krow), du);
                du *= wout;
                const int at = TX::at(s, 16 * pt + 4 * g);
                float xv[4], yv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xv[e] = to_f32(sx[at + e]);
                    yv[e] = to_f32(sy[at + e]);
                    if constexpr (NI == 3) {
                        xv[e] += to_f32(sx[TX::PLANE + at + e]) + to_f32(sx[2 * TX::PLANE + at + e]);
                        yv[e] += to_f32(sy[TX::PLANE + at + e]) + to_f32(sy[2 * TX::PLANE + at + e]);
                    }
                    vs += du[e] * xv[e];
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
                    if (2 * kt + 1 >= is)
                        du = mma(read_cols<TX, NI>(sy, kt, cols_at<TX>(16 * pt, lane)), mp[kt], du);
#pragma unroll
                for (int e = 0; e < 4; ++e) xdu += du[e] * xv[e];
                if (s < n)
                    store4(dx + 16 * pt + 4 * g, dts * du[0] + D * yv[0], dts * du[1] + D * yv[1],
                           dts * du[2] + D * yv[2], dts * du[3] + D * yv[3]);
            }
            xdu = rows4_sum(xdu);
            vs = rows4_sum(vs);
            if (g == 0) s_xdu[par][pg][s] = xdu, s_v[par][pg][s] = vs * dts;
        }
        lds_barrier();
        // ---- phase B: the products with Q, and the next head's rows into LDS
        Parts<NI> bt[KT], ct[KT];  // B^T and C^T of this wave's columns n
#pragma unroll
        for (int ks = 0; ks < KT; ++ks) {
            bt[ks] = read_cols<TK, NI>(sb, ks, cols_at<TK>(16 * nt, lane));
            ct[ks] = read_cols<TK, NI>(sc, ks, cols_at<TK>(16 * nt, lane));
        }
#pragma unroll
        for (int q = 0; q < TPW; ++q) {
            const int it = tg * TPW + q;
#pragma unroll
            for (int ks = 0; ks < KT; ++ks) {
                if (ks <= it / 2) dC[q] = mma(bt[ks], read_cols<TQ, KQ>(sq, ks, cols_at<TQ>(16 * it, lane)), dC[q]);
                if (ks >= it / 2) dB[q] = mma(ct[ks], read_rows<TQ, KQ>(sq, 16 * it, ks, RowsAt<TQ>(lane)), dB[q]);
            }
        }
        if (more) {
            rx.template store<TX>(sx, tid);
            ry.template store<TX>(sy, tid);
            store_e();
        }
        lds_barrier();
    }
    if (summer && count > 0) add_up(count - 1);
    // dB and dC of this group, or of this set of its heads
#pragma unroll
    for (int q = 0; q < TPW; ++q) {
        const int t = 16 * (tg * TPW + q) + r;
        if (t >= n) continue;
        const int64_t token = t0 + t, col = (int64_t)group * N + 16 * nt + 4 * g;
        if (a.sets == 1) {
            store4(static_cast<T *>(a.dB) + token * a.db_stride + col, dB[q][0], dB[q][1], dB[q][2],
                   dB[q][3]);
            store4(static_cast<T *>(a.dC) + token * a.dc_stride + col, dC[q][0], dC[q][1], dC[q][2],
                   dC[q][3]);
        } else {
            const int64_t row = (int64_t)a.groups * N;
            float *p = a.part_bc + (2 * set * (int64_t)a.seqs.total + token) * row + col;
            *reinterpret_cast<f32x4 *>(p) = dB[q];
            *reinterpret_cast<f32x4 *>(p + a.seqs.total * row) = dC[q];
        }
    }
}

// dB and dC: the sets' parts summed in order, four values a thread.
template <typename T> __global__ __launch_bounds__(256) void ssm_sets_kernel(SsmGrad a) {
    const int64_t row = (int64_t)a.groups * a.n, values = (int64_t)a.seqs.total * row;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= 2 * values) return;
    const int which = at >= values;
    const int64_t v = at - which * values, token = v / row, col = v % row;
    if (token >= seq_end_token(a.seqs, a.seqs.num - 1)) return;  // in no sequence
    const float *p = a.part_bc + at;
    f32x4 s = zero4();
    for (int k = 0; k < a.sets; ++k) s += *reinterpret_cast<const f32x4 *>(p + 2 * k * values);
    T *out = which ? static_cast<T *>(a.dC) + token * a.dc_stride : static_cast<T *>(a.dB) + token * a.db_stride;
    store4(out + col, s[0], s[1], s[2], s[3]);
}

// dA and dD of one head: its blocks' parts summed in fp64, 256 side by side.
__global__ __launch_bounds__(256) void ssm_params_kernel(SsmGrad a) {
    __shared__ double sum[2][256];
    const int h = blockIdx.x, tid = threadIdx.x;
    double s = 0.0, d = 0.0;
    for (int64_t i = tid; i < a.blocks; i += 256) {
        s += a.part_a[i * a.heads + h];
        d += a.part_d[i * a.heads + h];
    }
    sum[0][tid] = s;
    sum[1][tid] = d;
    __syncthreads();
    for (int k = 128; k > 0; k >>= 1) {
        if (tid < k)
            for (int q = 0; q < 2; ++q) sum[q][tid] += sum[q][tid + k];
        __syncthreads();
    }
    if (tid == 0) {
        a.dA[h] = (float)sum[0][0];
        if (a.dD) a.dD[h] = (float)sum[1][0];
    }
}

template <typename T> int grad(const SsmGrad &a, hipStream_t stream) {
    if (a.blocks == 0) {  // no sequence: dA and dD are zero
        hipLaunchKernelGGL(ssm_params_kernel, dim3(a.heads), dim3(256), 0, stream, a);
        return hipGetLastError() == hipSuccess ? 0 : -1;
    }
    const unsigned blocks = (unsigned)(a.blocks * a.groups * a.sets);
    if (a.n == 64)
        hipLaunchKernelGGL((ssm_grad_kernel<T, 64>), dim3(blocks), dim3(kGradWaves * 64), 0, stream, a);
    else
        hipLaunchKernelGGL((ssm_grad_kernel<T, 128>), dim3(blocks), dim3(kGradWaves * 64), 0, stream, a);
    if (a.sets > 1) {
        const int64_t quads = 2 * (int64_t)a.seqs.total * a.groups * a.n / 4;
        if (quads > 0)
            hipLaunchKernelGGL((ssm_sets_kernel<T>), dim3((unsigned)((quads + 255) / 256)), dim3(256),
                               0, stream, a);
    }
    hipLaunchKernelGGL(ssm_params_kernel, dim3(a.heads), dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int64_t ssm_grad_threads(const SsmGrad &a) { return a.blocks * a.groups * a.sets * kGradWaves * 64; }
int launch_ssm_grad(const SsmGrad &a, int dtype, hipStream_t stream) {
    return dtype == kDtypeBf16 ? grad<bf16>(a, stream) : grad<float>(a, stream);
}

}  // namespace kda
