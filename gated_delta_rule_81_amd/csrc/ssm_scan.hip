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
// One workgroup walks the blocks of a piece for 128 state rows (fp32: one head);
// a wave keeps 32 of them (fp32: 16) as fp32 accumulators of S^T tiles, which are
// the next block's operand as they stand.  D x is a term on the diagonal of the
// block's weights.  A long sequence is cut into pieces that run at once: a first
// pass leaves each piece's own final state, a fold turns these into entering
// states (the transition of a piece is one number per head), and the second pass
// is the scan proper.  The first pass reads x and B once more and does 4 P N of
// the second's 4 P N + 2 L (P + N) operations a token.
//
// Bound by issue, not by HBM: fp32 operands (the state, its updates, the block's
// weights) enter the matrix unit as three bf16 parts, so a token costs 3 times the
// products above, and the parts (5.5 VALU instructions a value) and decays take as
// many cycles again.  Two parts of the state and the weights where they enter y
// would take 383 us where three take 432, but then sums that cancel to less than
// 2^-8 of their terms lose more to the parts than to a bf16 output's own rounding.
// 32K tokens x 64 heads of 64 x 128 bf16, 0.68 GB: 427 to 451 us a call; in a trace
// of warm calls pieces 109, fold 13 (67 MB, 5 TB/s), scan 319.  The scan's SIMDs
// issue VALU in 55% of the cycles and the matrix unit works in 34%.  fp32: 990 us.
// Wave rows: a 32-row wave reads every row of B, C and M from LDS once for two tiles
// of products (with two parts: 16 rows 452 us, 32 rows 384).
#include "ssm_device.h"

#include <algorithm>
#include <type_traits>

namespace kda {
namespace {

enum Mode { kLocal, kOut, kStates };

// LDS of one block's tiles.
template <typename T, int P, int N, int HEADS, int MODE> struct ScanLds {
    static constexpr int L = kSsmBlock<T>, NI = sizeof(T) == 2 ? 1 : 3;
    static constexpr bool OUT = MODE == kOut;
    typedef Tile<NI, L, N> TK;
    typedef Tile<NI, L, HEADS * P> TX;
    // Row tiles 0 and 1 have nothing right of column 32: of 64 rows, 1 lies beside 0.
    static constexpr bool PACK = L == 64;
    // The weights M in three parts; of 64 rows as fp32 (a value takes two elements),
    // split where they are read: three parts of each would leave one workgroup a CU.
    typedef std::conditional_t<PACK, Tile<1, 48, 2 * L>, Tile<3, L, L>> TM;
    typedef std::conditional_t<PACK, FloatRowsAt<TM>, RowsAt<TM>> MRows;
    __device__ static constexpr int m_row(int it) { return PACK && it > 0 ? it - 1 : it; }
    __device__ static constexpr int m_step(int it) { return PACK && it == 1; }  // 32 columns each
    __attribute__((aligned(16))) bf16 k[TK::ELEMS];
    __attribute__((aligned(16))) bf16 c[OUT ? TK::ELEMS : 8];
    __attribute__((aligned(16))) bf16 x[TX::ELEMS];
    __attribute__((aligned(16))) bf16 m[OUT ? HEADS * TM::ELEMS : 8];
    __attribute__((aligned(16))) double cum[2][HEADS][L];  // log2 of the decay up to t
    __attribute__((aligned(16))) float dt[2][HEADS][L], w[2][HEADS][L], in[2][HEADS][L];
    // Weights of M's tiles below the diagonal as products, from the last token before
    // the tile's rows: row[t] = e^{cum_t - cum_ref}, col[at(it) + s] = dt_s e^{cum_ref - cum_s}.
    static constexpr int TL = L / 16;
    __device__ static constexpr int col_at(int it) { return 8 * it * (it - 1); }
    __attribute__((aligned(16))) float row[OUT ? 2 : 1][HEADS][OUT ? L : 1];
    __attribute__((aligned(16))) float col[OUT ? 2 : 1][HEADS][OUT ? col_at(TL) : 4];
    double tot[2][HEADS];
    // whether a wave staged a NaN or an infinity of x; a row's first such token, or L
    __attribute__((aligned(4))) unsigned char odd[8], from[OUT ? HEADS * P : 4];
};

// REV walks the blocks from the last to the first and the tokens' weights from
// the right: the gradient's recurrence E_{t-1} = e^{dt_t A} (E_t + x_t k_t^T).
template <typename T, int P, int N, int HEADS, int RT, int MODE, bool REV>
__device__ __forceinline__ void scan_body(const SsmScan &a, int64_t unit,
                                          ScanLds<T, P, N, HEADS, MODE> &lds) {
    typedef ScanLds<T, P, N, HEADS, MODE> S_;
    constexpr int L = S_::L, NT = HEADS * P * 4 / RT, NW = NT / 64, WPH = NW / HEADS, NI = S_::NI;
    constexpr bool OUT = S_::OUT;
    typedef typename S_::TK TK;
    typedef typename S_::TX TX;
    typedef typename S_::TM TM;
    bf16 *sk = lds.k, *sc = lds.c, *sx = lds.x, *sm = lds.m;
    auto &s_cum = lds.cum;
    auto &s_dt = lds.dt, &s_w = lds.w, &s_in = lds.in;
    auto &s_tot = lds.tot;

    const int h0 = (int)(unit % (a.heads / HEADS)) * HEADS;
    const int64_t number = unit / (a.heads / HEADS);
    const Piece pc = find_piece<MODE == kLocal>(a.seqs, number, a.piece);
    if (!pc.any) return;
    if (MODE == kLocal && (REV ? pc.first : pc.last)) return;  // nothing enters from it
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
    const RowsAt<TK> krow(lane);
    const WideAt<TK> kwide(lane);
    const typename S_::MRows mrow(lane);
    int kcol[N / 16];
#pragma unroll
    for (int t = 0; t < N / 16; ++t) kcol[t] = cols_at<TK>(16 * t, lane);
    // this wave's rows, counted over the workgroup's heads, and their head
    const int row0 = 16 * RT * wave, mine = wave / WPH;
    int xcol[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) xcol[rt] = cols_at<TX>(row0 + 16 * rt, lane);
    const int group = h0 / (a.heads / a.groups);
    const T *x = static_cast<const T *>(a.x) + (int64_t)h0 * P;
    const T *k = static_cast<const T *>(a.k) + (int64_t)group * N;
    const T *c = static_cast<const T *>(a.c) + (int64_t)group * N;
    // the last waves, one for each head, form the decays (the first ones have a tile
    // of M more)
    const bool weigher = wave >= NW - HEADS;
    const int wh = weigher ? wave - (NW - HEADS) : 0;
    const double A = (double)a.A[h0 + wh] * kLog2eD;
    const int blocks = (pc.end - pc.beg + L - 1) / L;

    // S^T tiles: rows n = 16 t + 4 g + e, column p = row0 + 16 rt + r.  kStates, which
    // forms no outputs, keeps S tiles (rows p, column n = 16 t + r) instead: its
    // states are stored [N][P], four rows p a lane.
    f32x4 S[RT][N / 16];
    constexpr bool TR = MODE == kStates;
    const int lane_off = TR ? (row0 + 4 * g) * N + r : (row0 + r) * N + 4 * g;
    const float *enter = nullptr;
    if (MODE != kLocal) {
        // Of a sequence in several pieces the fold has written every entering state,
        // the first too: final_state may be state0, and another workgroup writes it.
        enter = a.seg_states && !(pc.first && pc.last)
                    ? a.seg_states + (pc.slot * a.heads + h0) * (int64_t)(P * N)
                    : (a.state0 ? a.state0 + ((int64_t)pc.seq * a.heads + h0) * (P * N) : nullptr);
    }
#pragma unroll
    for (int i = 0; i < RT * (N / 16); ++i) {
        const int rt = i / (N / 16), t = i % (N / 16);
        const float *at = enter + lane_off + 16 * rt * N + 16 * t;
        S[rt][t] = !enter ? zero4()
               : TR   ? f32x4{at[0], at[N], at[2 * N], at[3 * N]}
                      : *reinterpret_cast<const f32x4 *>(at);
    }

    Stage<T, L, N, NT> rk, rc;
    Stage<T, L, HEADS * P, NT> rx;
    float rdt = 0.f;
    // kLocal walks against the recurrence: a token's weight in the state behind the
    // piece is known from the blocks before it in that order, and the sums need no
    // decay from block to block.
    constexpr bool FROM_END = REV != (MODE == kLocal);
    auto first_token = [&](int i) { return pc.beg + (FROM_END ? blocks - 1 - i : i) * L; };
    auto load_rows = [&](int i) {
        const int t0 = first_token(i), n = pc.end - t0 < L ? pc.end - t0 : L;
        rk.load(k + t0 * a.k_stride, a.k_stride, n, tid);
        rx.load(x + t0 * a.x_stride, a.x_stride, n, tid);
        if constexpr (OUT) rc.load(c + t0 * a.c_stride, a.c_stride, n, tid);
    };
    auto load_dt = [&](int i) {  // lane = token; tokens past the end do nothing (dt = 0)
        const int t = first_token(i) + lane;
        rdt = lane < L && t < pc.end ? a.dt[(int64_t)t * a.heads + h0 + wh] : 0.f;
    };
    float D[HEADS];
#pragma unroll
    for (int hh = 0; hh < HEADS; ++hh) D[hh] = OUT && a.D ? a.D[h0 + hh] : 0.f;
    double total = 0.0;
    auto weights = [&](int buf) {
        const double step = (double)rdt * A;
        const double cum = wave_prefix(step < -400.0 ? -400.0 : step, lane);
        const double all = from_lane(cum, 63), behind = MODE == kLocal ? total : 0.0;
        total += all;
        if (lane < L) {
            s_cum[buf][wh][lane] = cum;
            s_dt[buf][wh][lane] = rdt;
            s_in[buf][wh][lane] = fast_exp2((float)cum);
            s_w[buf][wh][lane] = REV ? fast_exp2((float)(behind + cum))
                                     : rdt * fast_exp2((float)(behind + (all - cum)));
        }
        if constexpr (OUT) {
            double ref = 0.0;
#pragma unroll
            for (int it = 1; it < S_::TL; ++it) {
                const double before = from_lane(cum, 16 * it - 1);
                if (lane >= 16 * it) ref = before;
                else lds.col[buf][wh][S_::col_at(it) + lane] = rdt * fast_exp2((float)(before - cum));
            }
            if (lane < L) lds.row[buf][wh][lane] = fast_exp2((float)(cum - ref));
        }
        if (lane == 0) s_tot[buf][wh] = all;
    };
    if (blocks > 0) {
        load_rows(0);
        if (weigher) {
            load_dt(0);
            weights(0);
        }
    }
    if constexpr (OUT) {  // tiles above the diagonal that a 32-wide step reads: zero for good
        for (int i = tid; i < HEADS * TM::ELEMS; i += NT) sm[i] = static_cast<bf16>(0.f);
    }
    for (int i = 0; i < blocks; ++i) {
        const int buf = i & 1, t0 = first_token(i);
        rk.template store<TK>(sk, tid);
        rx.template store<TX>(sx, tid);
        if constexpr (OUT) {
            rc.template store<TK>(sc, tid);
            const bool any = __builtin_amdgcn_ballot_w64(!finite(rx.sum())) != 0;
            if (lane == 0) lds.odd[wave] = any;
        }
        lds_barrier();
        if (i + 1 < blocks) {
            load_rows(i + 1);
            if (weigher) load_dt(i + 1);
        }
        if constexpr (MODE == kStates) {
            const int64_t block = first_piece(a.seqs, L, pc.seq_beg, pc.seq) + (t0 - pc.seq_beg) / L;
            float *to = a.block_states + (block * a.heads + h0 + mine) * (int64_t)(P * N) +
                        (int64_t)r * P + row0 % P + 4 * g;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int t = 0; t < N / 16; ++t)
                    *reinterpret_cast<f32x4 *>(to + (int64_t)16 * t * P + 16 * rt) = S[rt][t];
        }
        f32x4 y[RT][L / 16];
        const int ln = here(lane), r = ln & 15, g = ln >> 4;
        // A product with a zero weight still passes on a NaN or an infinity of x, so a
        // token's would reach earlier ones.  They enter the products as zeros; y of the
        // row is NaN from that token on, and the row of the state behind the block.
        bool odd = false;
        if constexpr (OUT) {
            static_assert(NW == 4 || NW == 8, "flags of the waves as words");
            const unsigned *f = reinterpret_cast<const unsigned *>(lds.odd);
            odd = __builtin_amdgcn_readfirstlane(NW == 4 ? f[0] : f[0] | f[1]) != 0;
            if (__builtin_expect(odd, 0)) {  // every wave its own rows
                constexpr int ROWS = 16 * RT, SPAN = L * ROWS / 64;  // tokens of a lane
                const int col = row0 + ln % ROWS, begin = ln / ROWS * SPAN;
                int first = L;
#pragma unroll 1
                for (int t = begin + SPAN - 1; t >= begin; --t) {
                    bf16 *at = sx + TX::at(t, col);
                    if (finite(to_f32(*at))) continue;
                    first = t;
                    for (int q = 0; q < NI; ++q) at[q * TX::PLANE] = static_cast<bf16>(0.f);
                }
                if (RT == 1) first = min(first, __shfl_xor(first, 16, 64));
                first = min(first, __shfl_xor(first, 32, 64));
                lds.from[col] = (unsigned char)first;
            }
        }
        if constexpr (OUT) {
            // M[t][s] = e^{cum_t - cum_s} (C_t . B_s) dt_s, s <= t, formed as tiles of M^T
            int q = 0;
#pragma unroll
            for (int it = 0; it < L / 16; ++it)
#pragma unroll
                for (int is = 0; is <= it; ++is, ++q) {
                    if (q % NW != wave) continue;
                    f32x4 m = zero4();
#pragma unroll
                    for (int ks = 0; ks < N / 32; ++ks)
                        m = mma(read_wide<TK, NI>(sk, 16 * is, ks, kwide),
                                read_wide<TK, NI>(sc, 16 * it, ks, kwide), m);
                    const int t = 16 * it + r, s = 16 * is + 4 * g;
                    const int to = TM::at(16 * S_::m_row(it) + r,
                                          (S_::PACK ? 2 : 1) * (s + 32 * S_::m_step(it)));
#pragma unroll
                    for (int hh = 0; hh < HEADS; ++hh) {
                        float v[4];
                        if (is < it) {
                            const float row = lds.row[buf][hh][t];
                            const f32x4 col =
                                *reinterpret_cast<const f32x4 *>(&lds.col[buf][hh][S_::col_at(it) + s]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] = m[e] * row * col[e];
                        } else {  // 0 above the diagonal, D's term on it
                            const double ct = s_cum[buf][hh][t];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float z = (float)(ct - s_cum[buf][hh][s + e]);
                                const float on = m[e] * fast_exp2(z) * s_dt[buf][hh][s + e];
                                v[e] = s + e > t ? 0.f : s + e == t ? on + D[hh] : on;
                            }
                        }
                        bf16 *at = sm + hh * TM::ELEMS + to;
                        if constexpr (S_::PACK)
                            *reinterpret_cast<f32x4 *>(at) = f32x4{v[0], v[1], v[2], v[3]};
                        else
                            store_parts<TM::PLANE>(at, v);
                    }
                }
            // y^T = S C^T e^{cum}: rows p, columns t
#pragma unroll
            for (int i = 0; i < RT * (L / 16); ++i) y[i % RT][i / RT] = zero4();
#pragma unroll
            for (int ks = 0; ks < N / 32; ++ks) {
                Parts<3> sp[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = S[rt][2 * ks][e], f[4 + e] = S[rt][2 * ks + 1][e];
                    sp[rt] = split<3>(f);
                }
#pragma unroll
                for (int it = 0; it < L / 16; ++it) {
                    const Parts<NI> ct = read_rows<TK, NI>(sc, 16 * it, ks, krow);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) y[rt][it] = mma(sp[rt], ct, y[rt][it]);
                }
            }
#pragma unroll
            for (int it = 0; it < L / 16; ++it)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) y[rt][it] *= s_in[buf][mine][16 * it + r];
            // the next block's decays, by a wave that had a tile of M less to form
            if (weigher && i + 1 < blocks) weights(buf ^ 1);
            lds_barrier();
        }
        // x^T operands of this wave's rows p, and x^T weighted for the state
        Parts<NI> xt[RT][L / 32];
        Parts<3> xw[RT][L / 32];
#pragma unroll
        for (int ks = 0; ks < L / 32; ++ks) {
            const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&s_w[buf][mine][32 * ks + 4 * g]);
            const f32x4 w1 = *reinterpret_cast<const f32x4 *>(&s_w[buf][mine][32 * ks + 16 + 4 * g]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const Parts<NI> &xv = xt[rt][ks] = read_cols<TX, NI>(sx, ks, xcol[rt]);
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v = to_f32(xv.v[0][e]);
                    if constexpr (NI == 3) v += to_f32(xv.v[1][e]) + to_f32(xv.v[2][e]);
                    f[e] = v * (e < 4 ? w0[e % 4] : w1[e % 4]);
                }
                xw[rt][ks] = split<3>(f);
            }
        }
        if constexpr (OUT) {
            const int n = pc.end - t0;
            T *out = static_cast<T *>(a.out) + (int64_t)h0 * P + row0 + 4 * g;
            const bf16 *weights_of = sm + mine * TM::ELEMS;
#pragma unroll
            for (int it = 0; it < L / 16; ++it) {
#pragma unroll
                for (int ks = 0; ks <= it / 2; ++ks) {
                    const Parts<3> mt = read_rows<TM, 3>(weights_of, 16 * S_::m_row(it),
                                                         ks + S_::m_step(it), mrow);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) y[rt][it] = mma(xt[rt][ks], mt, y[rt][it]);
                }
                const int t = 16 * it + r;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    f32x4 &o = y[rt][it];
                    if (__builtin_expect(odd, 0))
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = t < lds.from[row0 + 16 * rt + 4 * g + e] ? o[e] : __builtin_nanf("");
                    if (t < n)
                        store4(out + (int64_t)(t0 + t) * a.out_stride + 16 * rt, o[0], o[1], o[2],
                               o[3]);
                }
            }
        }
        const float decay = fast_exp2((float)s_tot[buf][mine]);
#pragma unroll
        for (int t = 0; t < N / 16; ++t) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                if (MODE != kLocal) S[rt][t] *= decay;
#pragma unroll
            for (int ks = 0; ks < L / 32; ++ks) {
                const Parts<NI> kt = read_cols<TK, NI>(sk, ks, kcol[t]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    S[rt][t] = TR ? mma(xw[rt][ks], kt, S[rt][t]) : mma(kt, xw[rt][ks], S[rt][t]);
            }
        }
        if (OUT && __builtin_expect(odd, 0)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                if (lds.from[row0 + 16 * rt + r] < L)
#pragma unroll
                    for (int t = 0; t < N / 16; ++t) S[rt][t] = zero4() + __builtin_nanf("");
        }
        if (!OUT && weigher && i + 1 < blocks) weights(buf ^ 1);
        lds_barrier();  // the tiles are read: the next block's may be written
    }
    float *to = nullptr;
    if (MODE == kLocal) {
        to = a.seg_states + (pc.slot * a.heads + h0) * (int64_t)(P * N);
        if (weigher && lane == 0) a.seg_decay[pc.slot * a.heads + h0 + wh] = total;
    } else if (a.final_state && (REV ? pc.first : pc.last)) {
        to = a.final_state + ((int64_t)pc.seq * a.heads + h0) * (P * N);
    }
    if (to)
#pragma unroll
        for (int i = 0; i < RT * (N / 16); ++i) {
            const int rt = i / (N / 16), t = i % (N / 16);
            float *at = to + lane_off + 16 * rt * N + 16 * t;
            if constexpr (TR)
#pragma unroll
                for (int e = 0; e < 4; ++e) at[e * N] = S[rt][t][e];
            else
                *reinterpret_cast<f32x4 *>(at) = S[rt][t];
        }
}

template <typename T, int P, int N, int HEADS, int RT>
__global__ __launch_bounds__(HEADS * P * 4 / RT, 2) void ssm_out_kernel(SsmScan a) {
    __shared__ ScanLds<T, P, N, HEADS, kOut> lds;
    const int64_t unit =
        xcd_unit(blockIdx.x, piece_count(a.seqs, a.piece), a.heads / HEADS, a.groups);
    if (unit >= 0) scan_body<T, P, N, HEADS, RT, kOut, false>(a, unit, lds);
}

template <typename T, int P, int N, int HEADS, int RT>
__global__ __launch_bounds__(HEADS * P * 4 / RT, 2) void ssm_local_kernel(SsmScan a) {
    __shared__ ScanLds<T, P, N, HEADS, kLocal> lds;
    const int64_t unit =
        xcd_unit(blockIdx.x, slot_count(a.seqs, a.piece), a.heads / HEADS, a.groups);
    if (unit >= 0) scan_body<T, P, N, HEADS, RT, kLocal, false>(a, unit, lds);
}

// Both directions of the backward's walk in one launch (half the workgroups
// each): neither alone has enough workgroups to hide its own latencies.
template <typename T, int P, int N, int HEADS, int RT, int MODE>
__global__ __launch_bounds__(HEADS * P * 4 / RT, 2) void ssm_both_kernel(SsmScan a, SsmScan b) {
    __shared__ ScanLds<T, P, N, HEADS, MODE> lds;
    const bool rev = blockIdx.x >= gridDim.x / 2;
    const int64_t numbers =
        MODE == kLocal ? slot_count(a.seqs, a.piece) : piece_count(a.seqs, a.piece);
    const int64_t unit = xcd_unit(rev ? blockIdx.x - gridDim.x / 2 : blockIdx.x, numbers,
                                  a.heads / HEADS, a.groups);
    if (unit < 0) return;
    if (!rev)
        scan_body<T, P, N, HEADS, RT, MODE, false>(a, unit, lds);
    else
        scan_body<T, P, N, HEADS, RT, MODE, true>(b, unit, lds);
}

// The pieces' own final states turned in place into entering states:
// enter[next] = e^{decay} enter + own.  One workgroup per 1024 values of a
// (sequence, head); the pieces one after the other, eight loads ahead.  Packed
// sequences in several pieces are found by the tokens i * piece: each holds one at
// least, its first is its own, and there are few beside many short sequences.
template <bool REV>
__device__ __forceinline__ void fold_body(const SsmScan &a, int values, int64_t block) {
    const int per = values / 1024;
    const int64_t u = block / per;
    const int h = (int)(u % a.heads);
    int n = (int)(u / a.heads), beg, end;
    const int64_t off = block % per * 1024 + threadIdx.x * 4;
    if (a.seqs.cu) {
        const int i = n;
        n = seq_of_token(a.seqs, i * a.piece, &beg, &end);
        if (n < 0 || ((int64_t)beg + a.piece - 1) / a.piece != i) return;
    } else {
        beg = seq_first(a.seqs, n);
        end = seq_end_token(a.seqs, n);
    }
    const int count = end > beg ? (int)(((int64_t)end - beg + a.piece - 1) / a.piece) : 1;
    if (count < 2) return;
    const int64_t first = first_slot(a.seqs, a.piece, beg, n);
    auto at = [&](int j) {
        return a.seg_states + ((first + (REV ? count - 1 - j : j)) * a.heads + h) * (int64_t)values + off;
    };
    f32x4 S = a.state0 ? *reinterpret_cast<const f32x4 *>(
                             a.state0 + ((int64_t)n * a.heads + h) * values + off)
                       : zero4();
    constexpr int U = 8;  // pieces whose loads are in flight together
    for (int j0 = 0; j0 < count - 1; j0 += U) {
        f32x4 own[U];
        float decay[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = j0 + i < count - 1 ? j0 + i : count - 2;
            own[i] = *reinterpret_cast<const f32x4 *>(at(j));
            decay[i] = fast_exp2(
                (float)a.seg_decay[(first + (REV ? count - 1 - j : j)) * a.heads + h]);
        }
        f32x4 kept = S;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const f32x4 enter = kept;
            if (j0 + i < count - 1) {
                kept = enter * decay[i] + own[i];
                *reinterpret_cast<f32x4 *>(at(j0 + i)) = enter;
            }
        }
        S = kept;
    }
    *reinterpret_cast<f32x4 *>(at(count - 1)) = S;
}

__global__ __launch_bounds__(256) void ssm_fold_kernel(SsmScan a, int values) {
    fold_body<false>(a, values, blockIdx.x);
}
__global__ __launch_bounds__(256) void ssm_fold_both_kernel(SsmScan a, SsmScan b, int values,
                                                            unsigned blocks) {
    if (blockIdx.x < blocks)
        fold_body<false>(a, values, blockIdx.x);
    else
        fold_body<true>(b, values, blockIdx.x - blocks);
}

template <typename T, int P, int N, int HEADS, int RT> struct Scan {
    static constexpr int NT = HEADS * P * 4 / RT;
    static int64_t pieces(const SsmScan &a) {
        return xcd_blocks(piece_count(a.seqs, a.piece), a.heads / HEADS, a.groups);
    }
    static int64_t slots(const SsmScan &a) {
        return xcd_blocks(slot_count(a.seqs, a.piece), a.heads / HEADS, a.groups);
    }
    static int64_t folds(const SsmScan &a) {
        const int64_t seqs =
            a.seqs.cu ? ((int64_t)a.seqs.total + a.piece - 1) / a.piece : a.seqs.num;
        return seqs * a.heads * (P * N / 1024);
    }
    static int64_t threads(const SsmScan &a, int directions) {
        const int64_t walk = pieces(a) * NT;
        if (!a.seg_states) return directions * walk;
        const int64_t local = slots(a) * NT, fold = folds(a) * 256;
        return directions * std::max(walk, std::max(local, fold));
    }
    static int out(const SsmScan &a, hipStream_t stream) {
        if (a.seg_states) {
            hipLaunchKernelGGL((ssm_local_kernel<T, P, N, HEADS, RT>), dim3((unsigned)slots(a)),
                               dim3(NT), 0, stream, a);
            hipLaunchKernelGGL(ssm_fold_kernel, dim3((unsigned)folds(a)), dim3(256), 0, stream, a,
                               P * N);
        }
        hipLaunchKernelGGL((ssm_out_kernel<T, P, N, HEADS, RT>), dim3((unsigned)pieces(a)), dim3(NT),
                           0, stream, a);
        return hipGetLastError() == hipSuccess ? 0 : -1;
    }
    static int both(const SsmScan &a, const SsmScan &b, hipStream_t stream) {
        if (a.seg_states) {
            hipLaunchKernelGGL((ssm_both_kernel<T, P, N, HEADS, RT, kLocal>),
                               dim3((unsigned)(2 * slots(a))), dim3(NT), 0, stream, a, b);
            const unsigned f = (unsigned)folds(a);
            hipLaunchKernelGGL(ssm_fold_both_kernel, dim3(2 * f), dim3(256), 0, stream, a, b, P * N,
                               f);
        }
        hipLaunchKernelGGL((ssm_both_kernel<T, P, N, HEADS, RT, kStates>),
                           dim3((unsigned)(2 * pieces(a))), dim3(NT), 0, stream, a, b);
        return hipGetLastError() == hipSuccess ? 0 : -1;
    }
};

// bf16: 128 rows a workgroup and 32 a wave, two heads of 64 that share B and C
// together.  Measured with two parts of y's operands: 32K x 64 heads of 64 x 128 384
// us, with one head a workgroup and 16 rows a wave 452; heads of 128 rows 690 and 814
// (with three parts 806); 1,227 tokens x 8 heads of 64 x 64,
// where the launches count, 28 and 29.  An odd number of heads a group leaves one
// head a workgroup; fp32 has no LDS for two (three parts of every tile).
template <typename T, int P, typename F> auto by_state(const SsmScan &a, F f) {
    typedef decltype(f(Scan<T, 64, 64, 1, 1>())) R;
    if constexpr (sizeof(T) == 2) {
        constexpr int HEADS = 128 / P;
        if (a.heads / a.groups % HEADS == 0)
            return a.n == 64 ? f(Scan<T, P, 64, HEADS, 2>()) : f(Scan<T, P, 128, HEADS, 2>());
    }
    if constexpr (sizeof(T) == 2 && P == 128) return R(-1);  // HEADS = 1 divides any number
    else return a.n == 64 ? f(Scan<T, P, 64, 1, 1>()) : f(Scan<T, P, 128, 1, 1>());
}
template <typename F> auto by_dims(const SsmScan &a, int dtype, F f) {
    if (dtype == kDtypeBf16) return a.p == 64 ? by_state<bf16, 64>(a, f) : by_state<bf16, 128>(a, f);
    return a.p == 64 ? by_state<float, 64>(a, f) : by_state<float, 128>(a, f);
}

}  // namespace

int64_t ssm_scan_threads(const SsmScan &a, int dtype, int directions) {
    return by_dims(a, dtype, [&](auto s) { return s.threads(a, directions); });
}
int launch_ssm_out(const SsmScan &a, int dtype, hipStream_t stream) {
    return by_dims(a, dtype, [&](auto s) { return s.out(a, stream); });
}
int launch_ssm_states(const SsmScan &a, const SsmScan &b, int dtype, hipStream_t stream) {
    return by_dims(a, dtype, [&](auto s) { return s.both(a, b, stream); });
}

}  // namespace kda
