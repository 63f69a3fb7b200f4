// qk_norm.hip -- queries and keys divided by each head's norm, weighted, and
// rotated by position in the same pass; forward and backward.
//
//   y = R (x w inv),  inv = 1 / sqrt(ss / m + eps),  m = 1 (L2) or d (RMS);
//   backward: g = R^T dy, dw = sum g x inv, h = g w,
//             dx = inv h - x inv^3 (h . x) / m.
//
// Every value is read once and written once (backward: two reads, one write),
// so HBM bounds both.  A head is d / 8 lanes with eight channels each (16 bytes
// of bf16); a wave works on 64 / (d / 8) heads of ONE token at a time, so the
// token's cos | sin row is read once into registers for all of its heads, q's
// and k's alike.  The sum over a head stays in its 8 or 16 lanes (DPP); pairs
// half the rotated width apart come from the partner lane.  32K tokens x 192 heads
// x 128 bf16 (3.2 GB): 572 us, 5.6 TB/s; backward with weights and rotation of 8K x
// 40 heads (0.25 GB): 55 us with the sum of its parts (4), 4.6 TB/s.
#include "layer_device.h"

namespace kda {
namespace {

// Passes (of 4 or 8 heads each) of one unit, whose loads are in flight together,
// and waves of a workgroup.  Measured, us: forward 32K x 192 heads x 128 bf16 with
// 4 passes and 1, 4, 8 waves 571, 581, 586, with 2 and 8 passes 584, 586; backward
// 8K x 40 heads (4 waves) with 2, 4, 8 passes 55, 58, 132, with 1 and 8 waves 105, 68.
constexpr int kFwdPasses = 4, kFwdWaves = 1;
constexpr int kBwdPasses = 2, kBwdWaves = 4;

// Sum over aligned groups of LPR (8 or 16) lanes, in every lane of the group.
template <int LPR> __device__ __forceinline__ float head_sum(float x) {
    auto dpp = [](float v, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value,
                                                          0xf, 0xf, true));
    };
    x += dpp(x, std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
    x += dpp(x, std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
    x += dpp(x, std::integral_constant<int, 0x141>{});  // row_half_mirror: the other quad of 8
    if constexpr (LPR == 16) x += dpp(x, std::integral_constant<int, 0x140>{});  // row_mirror
    return x;
}

// What a lane does to its eight channels: cos and sin per channel (or per
// channel pair when interleaved) and the lane that holds the other halves.
struct Turn {
    float cs[8], sn[8];  // sn carries the sign of the sine's term
    int partner;
    bool on;
};

template <int D>
__device__ __forceinline__ Turn load_turn(const QkArgs &a, int64_t token, int lane, bool back) {
    constexpr int LPR = D / 8;
    Turn r;
    const int e0 = 8 * (lane % LPR), half = a.rot / 2;
    r.on = e0 < a.rot;
    r.partner = lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.cs[i] = 1.f, r.sn[i] = 0.f;
    if (!r.on) return r;
    int pos = a.positions[token];
    pos = pos < 0 ? 0 : (pos >= a.table_rows ? a.table_rows - 1 : pos);
    const float *row = a.table + (int64_t)pos * a.rot;
    if (a.interleaved) {
        const f32x4 c = *reinterpret_cast<const f32x4 *>(row + e0 / 2);
        const f32x4 s = *reinterpret_cast<const f32x4 *>(row + half + e0 / 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r.cs[i] = c[i / 2];
            r.sn[i] = (i % 2 == 0) != back ? -s[i / 2] : s[i / 2];
        }
        return r;
    }
    const bool low = e0 < half;
    const int at = low ? e0 : e0 - half;
    r.partner = low ? lane + half / 8 : lane - half / 8;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const f32x4 c = *reinterpret_cast<const f32x4 *>(row + at + i);
        const f32x4 s = *reinterpret_cast<const f32x4 *>(row + half + at + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r.cs[i + e] = c[e];
            r.sn[i + e] = low != back ? -s[e] : s[e];
        }
    }
    return r;
}

// y <- R y (or R^T y when the turn was loaded so).  Every lane of the wave
// takes part in the exchange.
__device__ __forceinline__ void rotate(const Turn &r, int interleaved, float (&y)[8]) {
    float o[8];
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = y[i ^ 1];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl(y[i], r.partner, 64);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = r.on ? y[i] * r.cs[i] + o[i] * r.sn[i] : y[i];
}

__device__ __forceinline__ float inv_norm(float ss, bool rms, int d, float eps) {
    return __builtin_amdgcn_rsqf((rms ? ss * (1.f / d) : ss) + eps);
}

// Eight channels of both weights (ones where there is none).
__device__ __forceinline__ void load_weights(const QkArgs &a, int e0, float (&w)[2][8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[k][e] = a.weight[k] ? a.weight[k][e0 + e] : 1.f;
}

// The heads of one token in passes of HPP heads, q's first, then k's: a pass is
// never of both, so which of the two it is is the same for the whole wave.
struct Pass {
    int which, head;  // tensor, this lane's head in it
    bool on, any;     // whether there is such a head; whether there is such a pass
};
template <int HPP>
__device__ __forceinline__ Pass pass_of(const QkArgs &a, int pass, int sub) {
    const int pq = (a.heads[0] + HPP - 1) / HPP, pk = (a.heads[1] + HPP - 1) / HPP;
    Pass p;
    p.which = pass >= pq;
    p.any = pass < pq + pk;
    p.head = (p.which ? pass - pq : pass) * HPP + sub;
    p.on = p.any && p.head < (p.which ? a.heads[1] : a.heads[0]);
    return p;
}

// Row of this lane's eight channels in a tensor of the pass: scalar base, 32-bit
// offset (a token's heads span less than 2^31 bytes).
template <typename T>
__device__ __forceinline__ T *row_of(const void *q, const void *k, const int64_t (&stride)[2],
                                     const Pass &p, int64_t token, int d, int e0) {
    const char *base = static_cast<const char *>(p.which ? k : q) +
                       token * (p.which ? stride[1] : stride[0]) * (int64_t)sizeof(T);
    return (T *)(base + (unsigned)(p.head * d + e0) * (unsigned)sizeof(T));
}

// Unit: (token, group of kFwdPasses passes).  One wave per unit.
template <typename T, int D>
__global__ __launch_bounds__(64 * kFwdWaves) void qk_norm_fwd_kernel(QkArgs a, int groups,
                                                                     int64_t unit0) {
    constexpr int LPR = D / 8, HPP = 64 / LPR;  // lanes per head, heads per pass
    const int lane = threadIdx.x & 63;
    const int64_t unit = unit0 + (int64_t)blockIdx.x * kFwdWaves +
                         __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t token = unit / groups;
    if (token >= a.tokens) return;
    const int pass0 = (int)(unit % groups) * kFwdPasses, e0 = 8 * (lane % LPR);
    typename Vec8<T>::raw raw[kFwdPasses];
#pragma unroll
    for (int i = 0; i < kFwdPasses; ++i) {
        const Pass p = pass_of<HPP>(a, pass0 + i, lane / LPR);
        raw[i] = p.on ? load8(row_of<T>(a.x[0], a.x[1], a.x_stride, p, token, D, e0))
                      : Vec8<T>::zero();
    }
    const bool weights = a.weight[0] || a.weight[1];
    float wt[2][8];
    if (weights) load_weights(a, e0, wt);
    Turn turn;
    if (a.rot) turn = load_turn<D>(a, token, lane, false);
#pragma unroll
    for (int i = 0; i < kFwdPasses; ++i) {
        const Pass p = pass_of<HPP>(a, pass0 + i, lane / LPR);
        float x[8];
        Vec8<T>::to_float(raw[i], x);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
        const float inv = inv_norm(head_sum<LPR>(ss), a.rms, D, a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv;
        if (weights) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= p.which ? wt[1][e] : wt[0][e];
        }
        if (a.rot) rotate(turn, a.interleaved, x);
        if (p.on) store8(row_of<T>(a.y[0], a.y[1], a.y_stride, p, token, D, e0), x);
    }
}

// The same walk; the gradients of the two weights of all of a workgroup's heads go
// to its row of `partial` ([row][2][D]), summed afterwards in row order.
template <typename T, int D>
__global__ __launch_bounds__(64 * kBwdWaves, 4) void qk_norm_bwd_kernel(QkArgs a, int groups) {
    constexpr int LPR = D / 8, HPP = 64 / LPR;
    __shared__ float sum[kBwdWaves][2][HPP][D];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e0 = 8 * (lane % LPR);
    const int64_t units = (int64_t)a.tokens * groups;
    const bool weights = a.weight[0] || a.weight[1];
    float dw[2][8], wt[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
    if (weights) load_weights(a, e0, wt);
    for (int64_t unit = (int64_t)blockIdx.x * kBwdWaves + wave; unit < units;
         unit += (int64_t)gridDim.x * kBwdWaves) {
        const int64_t token = unit / groups;
        const int pass0 = (int)(unit % groups) * kBwdPasses;
        typename Vec8<T>::raw rx[kBwdPasses], rg[kBwdPasses];
#pragma unroll
        for (int i = 0; i < kBwdPasses; ++i) {
            const Pass p = pass_of<HPP>(a, pass0 + i, lane / LPR);
            rx[i] = p.on ? load8(row_of<T>(a.x[0], a.x[1], a.x_stride, p, token, D, e0))
                         : Vec8<T>::zero();
            rg[i] = p.on ? load8(row_of<T>(a.dy[0], a.dy[1], a.dy_stride, p, token, D, e0))
                         : Vec8<T>::zero();
        }
        Turn turn;
        if (a.rot) turn = load_turn<D>(a, token, lane, true);
#pragma unroll
        for (int i = 0; i < kBwdPasses; ++i) {
            const Pass p = pass_of<HPP>(a, pass0 + i, lane / LPR);
            if (!p.any) break;
            float x[8], g[8];
            Vec8<T>::to_float(rx[i], x);
            Vec8<T>::to_float(rg[i], g);
            if (a.rot) rotate(turn, a.interleaved, g);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
            const float inv = inv_norm(head_sum<LPR>(ss), a.rms, D, a.eps);
            if (weights) {
                // a lane without a head adds nothing (0 * inf where eps is 0)
                const float k = p.on ? inv : 0.f;
                if (p.which) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[1][e] += g[e] * (x[e] * k), g[e] *= wt[1][e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[0][e] += g[e] * (x[e] * k), g[e] *= wt[0][e];
                }
            }
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) dot += g[e] * x[e];
            // inv^2 first: x inv stays in range where inv^3 may not
            const float k = head_sum<LPR>(dot) * inv * (a.rms ? 1.f / D : 1.f) * inv;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = inv * (g[e] - x[e] * k);
            if (p.on) store8(row_of<T>(a.y[0], a.y[1], a.y_stride, p, token, D, e0), x);
        }
    }
    if (!a.partial) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sum[wave][0][lane / LPR][e0 + e] = dw[0][e];
        sum[wave][1][lane / LPR][e0 + e] = dw[1][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += 64 * kBwdWaves) {
        float s = 0.f;
#pragma unroll
        for (int wv = 0; wv < kBwdWaves; ++wv)
#pragma unroll
            for (int r = 0; r < HPP; ++r) s += sum[wv][i / D][r][i % D];
        a.partial[(int64_t)blockIdx.x * 2 * D + i] = s;
    }
}

// dq_weight and dk_weight: `rows` rows of [2][D], eight columns per workgroup,
// 128 rows side by side.
__global__ __launch_bounds__(1024) void qk_reduce_kernel(const float *partial, int rows, int D,
                                                         float *dq, float *dk) {
    __shared__ float part[128][8];
    const int col = blockIdx.x * 8 + threadIdx.x;
    float s = 0.f;
#pragma unroll 4
    for (int r = threadIdx.y; r < rows; r += 128) s += partial[(int64_t)r * 2 * D + col];
    part[threadIdx.y][threadIdx.x] = s;
    for (int k = 64; k > 0; k >>= 1) {
        __syncthreads();
        if (threadIdx.y < k) part[threadIdx.y][threadIdx.x] += part[threadIdx.y + k][threadIdx.x];
    }
    if (threadIdx.y) return;
    float *out = col < D ? dq : dk;
    if (out) out[col % D] = part[0][threadIdx.x];
}

int groups_of(int64_t q_heads, int64_t k_heads, int d, int per_unit) {
    const int hpp = 512 / d;  // heads per pass
    const int64_t passes = (q_heads + hpp - 1) / hpp + (k_heads + hpp - 1) / hpp;
    return (int)((passes + per_unit - 1) / per_unit);
}
// Workgroups of the backward: enough to fill the chip several times over,
// few enough that their partial sums stay small beside the data.
constexpr int kBwdBlocks = 1024;
int bwd_blocks(int64_t units) {
    const int64_t b = (units + kBwdWaves - 1) / kBwdWaves;
    return (int)(b < kBwdBlocks ? b : kBwdBlocks);
}

template <typename T, int D> int fwd(const QkArgs &a, hipStream_t stream) {
    const int groups = groups_of(a.heads[0], a.heads[1], D, kFwdPasses);
    const int64_t units = (int64_t)a.tokens * groups;
    constexpr int64_t kMost = (int64_t)1 << 25;  // a launch holds less than 2^32 threads
    for (int64_t u = 0; u < units; u += kMost) {
        const int64_t now = units - u < kMost ? units - u : kMost;
        hipLaunchKernelGGL((qk_norm_fwd_kernel<T, D>),
                           dim3((unsigned)((now + kFwdWaves - 1) / kFwdWaves)), dim3(64 * kFwdWaves),
                           0, stream, a, groups, u);
    }
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T, int D> int bwd(const QkArgs &args, hipStream_t stream) {
    QkArgs a = args;
    const bool weights = a.dweight[0] || a.dweight[1];
    if (!weights) a.partial = nullptr;
    const int groups = groups_of(a.heads[0], a.heads[1], D, kBwdPasses);
    const int blocks = bwd_blocks((int64_t)a.tokens * groups);
    if (blocks > 0)
        hipLaunchKernelGGL((qk_norm_bwd_kernel<T, D>), dim3(blocks), dim3(64 * kBwdWaves), 0, stream, a,
                           groups);
    if (weights)
        hipLaunchKernelGGL(qk_reduce_kernel, dim3(2 * D / 8), dim3(8, 128), 0, stream, a.partial,
                           blocks, D, a.dweight[0], a.dweight[1]);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

#define KDA_QK_DISPATCH(fn)                                                      \
    (a.dtype == kDtypeBf16                                                       \
         ? (a.head_dim == 128 ? fn<bf16, 128>(a, stream) : fn<bf16, 64>(a, stream)) \
         : (a.head_dim == 128 ? fn<float, 128>(a, stream) : fn<float, 64>(a, stream)))

}  // namespace

int launch_qk_norm_fwd(const QkArgs &a, hipStream_t stream) { return KDA_QK_DISPATCH(fwd); }
int launch_qk_norm_bwd(const QkArgs &a, hipStream_t stream) { return KDA_QK_DISPATCH(bwd); }

int64_t qk_norm_bwd_workspace_floats(int64_t tokens, int64_t q_heads, int64_t k_heads,
                                     int head_dim) {
    return (int64_t)bwd_blocks(tokens * groups_of(q_heads, k_heads, head_dim, kBwdPasses)) * 2 * head_dim;
}

}  // namespace kda
