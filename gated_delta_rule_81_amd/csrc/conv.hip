// conv.hip -- short depthwise causal convolution: forward, backward and the
// single-token step.
//
//   z[t] = bias + sum_j w[j] r[t - (W-1) + j],  out = z or z sigmoid(z),
//
// with r = the sequence's rows and, before them, its state's W - 1 rows.  Every
// value is read once and written once with about 2 W operations in between, so
// HBM bounds all three.  A lane keeps VEC neighbouring channels and walks a
// run of tokens with the last W - 1 rows in registers; a wave therefore reads
// and writes whole 1 KiB pieces of a row, and the only rows read twice are the
// W - 1 before each run.  Sequence boundaries inside a run are a wave-uniform
// branch per token that reloads the window from the next sequence's state.
//
// Measured, bf16: 32K x 12288 channels (1.6 GB) 334 us, 4.8 TB/s; backward of 2 x
// 4096 x 4096 (0.2 GB) 54 us with the sum of its parts (4), 3.7 TB/s; a token of 256
// sessions (0.15 GB) 28 to 33 us, 4.6 to 5.4 TB/s.  Few tokens (3,923 x 2184 channels
// in 7 sequences, 34 MB: 15 to 17 us) are one round of waves and hardly more than
// the call: there runs of 4, 8 or 16 tokens and 2, 4 or 8 rows loaded together
// measure 16.7 to 19.3 us.
#include "layer_device.h"

namespace kda {
namespace {

constexpr int kWaves = 4;  // runs of one workgroup (one per wave)

// A wave's run of tokens is the same for its 64 lanes; said so, the token, its
// sequence and its row's address stay in scalar registers and branches.
__device__ __forceinline__ int wave_of_block() {
    return __builtin_amdgcn_readfirstlane(threadIdx.y);
}
// Channel c of a row: a scalar base and a 32-bit offset per lane.
template <typename T> __device__ __forceinline__ const T *col(const T *row, int c) {
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(row) +
                                       (unsigned)c * (unsigned)sizeof(T));
}
template <typename T> __device__ __forceinline__ T *col(T *row, int c) {
    return reinterpret_cast<T *>(reinterpret_cast<char *>(row) + (unsigned)c * (unsigned)sizeof(T));
}

// Row `r` of the sequence that begins at token `beg`, as floats: a token's, or
// row r - beg + W - 1 of the sequence's state for the W - 1 rows before it.
template <typename T, int VEC, int W>
__device__ __forceinline__ void seq_row(const T *x, int64_t xs, const T *state0, int64_t n, int C,
                                        int c, int r, int beg, float (&f)[VEC]) {
    typedef Row<T, VEC> R;
    if (r >= beg) {
        R::get(R::raw(col(x + (int64_t)(r) * xs, c)), f);
    } else if (state0) {
        R::get(R::raw(col(state0 + (n * (W - 1) + (r - beg + W - 1)) * (int64_t)C, c)), f);
    } else {
        R::get(R::zero(), f);
    }
}

// The channels' taps and biases, in 16-byte pieces where VEC allows.
template <int VEC, int W>
__device__ __forceinline__ void load_params(const ConvArgs &a, int c, float (&w)[W][VEC],
                                            float (&b)[VEC]) {
    const float *wp = a.weight + (int64_t)c * W;
    if constexpr (VEC % 4 == 0) {
        f32x4 v[VEC * W / 4];
#pragma unroll
        for (int i = 0; i < VEC * W / 4; ++i) v[i] = *reinterpret_cast<const f32x4 *>(wp + 4 * i);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = v[(i * W + j) / 4][(i * W + j) % 4];
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const f32x4 q = a.bias ? *reinterpret_cast<const f32x4 *>(a.bias + c + i) : zero4();
#pragma unroll
            for (int e = 0; e < 4; ++e) b[i + e] = q[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = wp[i * W + j];
            b[i] = a.bias ? a.bias[c + i] : 0.f;
        }
    }
}

// A workgroup is 64 channel vectors x kWaves runs of `run` tokens; workgroups
// at and past `run_blocks` copy the final states, kWaves rows each.
template <typename T, int VEC, int W>
__global__ __launch_bounds__(64 * kWaves) void conv_fwd_kernel(ConvArgs a, int cblocks,
                                                               int run_blocks, int run) {
    typedef Row<T, VEC> R;
    constexpr int U = 2;  // rows loaded together, the next ones' loads ahead (32K: 334 us, with 8 346)
    const T *x = static_cast<const T *>(a.x), *state0 = static_cast<const T *>(a.state0);
    const int C = a.channels, wave = wave_of_block();
    const int c = ((int)(blockIdx.x % cblocks) * 64 + (int)threadIdx.x) * VEC;
    if (c >= C) return;
    const int64_t blk = blockIdx.x / cblocks;
    if (blk >= run_blocks) {
        const int64_t unit = (blk - run_blocks) * kWaves + wave;
        const int64_t n = unit / (W - 1);
        const int j = (int)(unit % (W - 1));
        if (n >= a.seqs.num) return;
        const int beg = seq_first(a.seqs, (int)n);
        int end = seq_end_token(a.seqs, (int)n);
        end = end < beg ? beg : end;
        float f[VEC];
        // row j of the last W - 1 of (state, x)
        seq_row<T, VEC, W>(x, a.x_stride, state0, n, C, c, end - (W - 1) + j, beg, f);
        R::put(static_cast<T *>(a.final_state) + (n * (W - 1) + j) * (int64_t)C + c, f);
        return;
    }
    const int64_t first = (blk * kWaves + wave) * (int64_t)run;
    if (first >= a.seqs.total) return;
    const int t0 = (int)first;
    const int t1 = first + run < a.seqs.total ? (int)(first + run) : a.seqs.total;
    T *out = static_cast<T *>(a.out);

    float w[W][VEC], b[VEC], win[W][VEC];  // win: rows t - (W-1) .. t
    load_params<VEC, W>(a, c, w, b);
    int beg = 0, end = 0, n = -1;
    typename R::vec next[U];
    auto load = [&](int t) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            next[i] = t + i < t1 ? R::raw(col(x + (int64_t)(t + i) * a.x_stride, c)) : R::zero();
    };
    auto token = [&](int t, const typename R::vec &raw) {
        R::get(raw, win[W - 1]);
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float z = b[e];
#pragma unroll
            for (int j = 0; j < W; ++j) z += w[j][e] * win[j][e];
            y[e] = a.silu ? z * sigmoid(z) : z;
        }
        R::put(col(out + (int64_t)t * a.out_stride, c), y);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) win[j][e] = win[j + 1][e];
    };
    // Token t's sequence and the rows before t; n < 0 where none holds it.
    auto enter = [&](int t) {
        n = seq_of_token(a.seqs, t, &beg, &end);
        if (n < 0) {
            end = t + 1;
            return;
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            seq_row<T, VEC, W>(x, a.x_stride, state0, n, C, c, t - (W - 1) + j, beg, win[j]);
    };
    load(t0);
    enter(t0);
    for (int t = t0; t < t1; t += U) {
        typename R::vec raw[U];
#pragma unroll
        for (int i = 0; i < U; ++i) raw[i] = next[i];
        load(t + U);
        if (t + U <= t1 && t + U <= end && n >= 0) {  // inside one sequence
#pragma unroll
            for (int i = 0; i < U; ++i) token(t + i, raw[i]);
            continue;
        }
#pragma unroll 1
        for (int tt = t; tt < t + U && tt < t1; ++tt) {
            if (tt >= end) enter(tt);
            if (n < 0) continue;
            token(tt, R::raw(col(x + (int64_t)tt * a.x_stride, c)));
        }
    }
}

// d(out)/dz times d_out, from the window ending at the token.
template <int VEC, int W>
__device__ __forceinline__ void grad_z(const float (&w)[W][VEC], const float (&b)[VEC],
                                       const float (&win)[W][VEC], bool silu, float (&g)[VEC]) {
    if (!silu) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float z = b[e];
#pragma unroll
        for (int j = 0; j < W; ++j) z += w[j][e] * win[j][e];
        const float s = sigmoid(z);
        g[e] *= s * (1.f + z * (1.f - s));
    }
}

// dz[t] = d_out act'(z); dx[s] = sum_j w[j] dz[s + (W-1) - j] over its own
// sequence (+ d_final for the last W - 1 rows); dw[j] = sum_t dz[t] r[t-(W-1)+j].
// A run emits dx of its own tokens, so it walks W - 1 tokens past its end (dz
// only); dw and db of the run go to the workgroup's row of `partial`
// ([row][W + 1][C]), summed afterwards in row order.
template <typename T, int VEC, int W>
__global__ __launch_bounds__(64 * kWaves) void conv_bwd_kernel(ConvArgs a, int cblocks,
                                                               int run_blocks, int run) {
    typedef Row<T, VEC> R;
    constexpr int U = 4;
    __shared__ float sum[kWaves - 1][W + 1][VEC][64];
    const T *x = static_cast<const T *>(a.x), *state0 = static_cast<const T *>(a.state0);
    const T *dy = static_cast<const T *>(a.d_out), *d_final = static_cast<const T *>(a.d_final);
    const int C = a.channels, wave = wave_of_block();
    const int c = ((int)(blockIdx.x % cblocks) * 64 + (int)threadIdx.x) * VEC;
    const bool on = c < C;
    const int64_t blk = blockIdx.x / cblocks;
    float w[W][VEC], b[VEC];
    if (on) load_params<VEC, W>(a, c, w, b);

    if (blk >= run_blocks) {  // gradient of the initial states: kWaves sequences each
        const int64_t n = (blk - run_blocks) * kWaves + wave;
        if (!on || n >= a.seqs.num) return;
        const int beg = seq_first(a.seqs, (int)n);
        int end = seq_end_token(a.seqs, (int)n);
        const int len = end < beg ? 0 : end - beg;
        float dz[W - 1][VEC];  // of the first W - 1 tokens
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
            R::get(R::zero(), dz[t]);
            if (t < len) {
                float win[W][VEC];
#pragma unroll
                for (int j = 0; j < W; ++j)
                    seq_row<T, VEC, W>(x, a.x_stride, state0, n, C, c, beg + t - (W - 1) + j, beg,
                                       win[j]);
                R::get(R::raw(col(dy + (int64_t)(beg + t) * a.d_out_stride, c)), dz[t]);
                grad_z<VEC, W>(w, b, win, a.silu, dz[t]);
            }
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            float g[VEC];
            R::get(R::zero(), g);
            if (d_final && j >= len)  // this row is still there in the final state
                R::get(R::raw(d_final + (n * (W - 1) + (j - len)) * (int64_t)C + c), g);
#pragma unroll
            for (int i = 0; i <= j; ++i)  // tap i of token j - i
#pragma unroll
                for (int e = 0; e < VEC; ++e) g[e] += w[i][e] * dz[j - i][e];
            R::put(static_cast<T *>(a.d_state0) + (n * (W - 1) + j) * (int64_t)C + c, g);
        }
        return;
    }

    const int64_t first = (blk * kWaves + wave) * (int64_t)run;
    float dw[W][VEC], db[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
    }
    if (on && first < a.seqs.total) {
        const int t0 = (int)first;
        const int t1 = first + run < a.seqs.total ? (int)(first + run) : a.seqs.total;
        const int t2 = t1 + (W - 1) < a.seqs.total ? t1 + (W - 1) : a.seqs.total;
        T *dx = static_cast<T *>(a.dx);
        float win[W][VEC], dz[W][VEC];  // dz: of tokens t - (W-1) .. t
        int beg = 0, end = t0, n = -1;

        // dx of token s, whose dz window begins at s
        auto emit = [&](int s, int row) {
            float g[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[e] = 0.f;
            if (row >= 0 && d_final)
                R::get(R::raw(d_final + ((int64_t)n * (W - 1) + row) * C + c), g);
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) g[e] += w[W - 1 - i][e] * dz[i][e];
            R::put(col(dx + (int64_t)s * a.dx_stride, c), g);
        };
        auto shift = [&]() {
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) dz[i][e] = dz[i + 1][e];
        };
        // the last W - 1 rows of the sequence that ends: no dz behind it
        auto flush = [&]() {
            for (int k = 0; k < W - 1; ++k) {
                shift();
#pragma unroll
                for (int e = 0; e < VEC; ++e) dz[W - 1][e] = 0.f;
                const int s = end - (W - 1) + k;
                if (s >= beg && s >= t0 && s < t1) emit(s, k);
            }
        };

        bool done = false;
        typename R::vec nx[U], ng[U];  // the next rows, their loads ahead
        auto load = [&](int t) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const bool in = t + i < t2;
                nx[i] = in ? R::raw(col(x + (int64_t)(t + i) * a.x_stride, c)) : R::zero();
                ng[i] = in ? R::raw(col(dy + (int64_t)(t + i) * a.d_out_stride, c)) : R::zero();
            }
        };
        auto token = [&](int t, const typename R::vec &rx, const typename R::vec &rg, bool own) {
            R::get(rx, win[W - 1]);
            shift();
            R::get(rg, dz[W - 1]);
            grad_z<VEC, W>(w, b, win, a.silu, dz[W - 1]);
            if (own) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    db[e] += dz[W - 1][e];
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j][e] += dz[W - 1][e] * win[j][e];
                }
            }
            const int s = t - (W - 1);
            if (s >= beg && s >= t0) emit(s, -1);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) win[j][e] = win[j + 1][e];
        };
        auto enter = [&](int t) {
            n = seq_of_token(a.seqs, t, &beg, &end);
            if (n < 0) {
                end = t + 1;
                return;
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                seq_row<T, VEC, W>(x, a.x_stride, state0, n, C, c, t - (W - 1) + j, beg, win[j]);
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) dz[j][e] = 0.f;
        };
        load(t0);
        enter(t0);
        for (int t = t0; t < t2 && !done; t += U) {
            typename R::vec rx[U], rg[U];
#pragma unroll
            for (int i = 0; i < U; ++i) rx[i] = nx[i], rg[i] = ng[i];
            load(t + U);
            if (t + U <= t1 && t + U <= end && n >= 0) {  // inside one sequence
#pragma unroll
                for (int i = 0; i < U; ++i) token(t + i, rx[i], rg[i], true);
                continue;
            }
#pragma unroll 1
            for (int tt = t; tt < t + U && tt < t2; ++tt) {
                if (tt >= end) {
                    if (n >= 0) flush();
                    if (tt >= t1) {  // what follows is another sequence's
                        n = -1;
                        done = true;
                        break;
                    }
                    enter(tt);
                }
                if (n < 0) continue;
                token(tt, R::raw(col(x + (int64_t)tt * a.x_stride, c)),
                      R::raw(col(dy + (int64_t)tt * a.d_out_stride, c)), tt < t1);
            }
        }
        // the walk ended where its sequence does (t2 = total, or the next begins at t2)
        if (!done && n >= 0 && end <= t2) flush();
    }
    if (wave > 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sum[wave - 1][W][e][threadIdx.x] = db[e];
#pragma unroll
            for (int j = 0; j < W; ++j) sum[wave - 1][j][e][threadIdx.x] = dw[j][e];
        }
    }
    __syncthreads();
    if (wave == 0 && on) {
        float *p = a.partial + blk * (W + 1) * (int64_t)C + c;
#pragma unroll
        for (int j = 0; j <= W; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float v = j < W ? dw[j][e] : db[e];
#pragma unroll
                for (int k = 0; k < kWaves - 1; ++k) v += sum[k][j][e][threadIdx.x];
                p[j * (int64_t)C + e] = v;
            }
    }
}

// dweight and dbias: the rows of `partial` summed, 16 rows side by side.
__global__ __launch_bounds__(1024) void conv_reduce_kernel(const float *partial, int rows, int C,
                                                           int W, float *dweight, float *dbias) {
    __shared__ float part[16][64];
    const int64_t col = (int64_t)blockIdx.x * 64 + threadIdx.x, cols = (int64_t)(W + 1) * C;
    float s = 0.f;
    if (col < cols)
        for (int r = threadIdx.y; r < rows; r += 16) s += partial[r * cols + col];
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || col >= cols) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += part[k][threadIdx.x];
    const int j = (int)(col / C);
    const int64_t c = col % C;
    if (j < W)
        dweight[c * W + j] = s;
    else if (dbias)
        dbias[c] = s;
}

template <typename T, int VEC, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a, T *state, int cblocks,
                                                        int batch) {
    typedef Row<T, VEC> R;
    const int C = a.channels, wave = wave_of_block();
    const int c = ((int)(blockIdx.x % cblocks) * 64 + (int)threadIdx.x) * VEC;
    const int64_t n = (int64_t)(blockIdx.x / cblocks) * kWaves + wave;
    if (c >= C || n >= batch) return;
    T *st = state + n * (W - 1) * (int64_t)C + c;
    typename R::vec raw[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j] = R::raw(st + j * (int64_t)C);
    raw[W - 1] = R::raw(static_cast<const T *>(a.x) + n * a.x_stride + c);
    float w[W][VEC], y[VEC];
    load_params<VEC, W>(a, c, w, y);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float f[VEC];
        R::get(raw[j], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] += w[j][e] * f[e];
        if (j > 0) *reinterpret_cast<typename R::vec *>(st + (j - 1) * (int64_t)C) = raw[j];
    }
    if (a.silu)
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] *= sigmoid(y[e]);
    R::put(static_cast<T *>(a.out) + n * a.out_stride + c, y);
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens of one wave's run.  Long runs read fewer rows twice, short ones fill
// the chip when there is little to do: about 8 waves per SIMD's worth of runs,
// 8 to 128 tokens each.
int run_tokens(int64_t total, int cblocks) {
    int64_t run = total * cblocks / (256 * 32);
    run = (run + 7) / 8 * 8;
    return (int)(run < 8 ? 8 : (run > 128 ? 128 : run));
}
// The backward's runs read 2 (W - 1) rows twice and are worth more length: 16 to
// 64 tokens, for 2048 waves (8K x 4096 channels bf16: 53 us with 64, 60 with
// 32, 61 with 16).
int bwd_run_tokens(int64_t total, int cblocks) {
    int64_t run = total * cblocks / 2048;
    run = (run + 7) / 8 * 8;
    return (int)(run < 16 ? 16 : (run > 64 ? 64 : run));
}

// Workgroups: channel blocks x (runs of tokens + rows of states).
struct Grid {
    int64_t cb, rb, sb;
    int run;
    int64_t blocks() const { return cb * (rb + sb); }
};
Grid fwd_grid(const ConvArgs &a, int vec) {
    Grid g = {div_up(a.channels, 64 * vec), 0, 0, 0};
    g.run = run_tokens(a.seqs.total, (int)g.cb);
    g.rb = div_up(a.seqs.total, (int64_t)g.run * kWaves);
    g.sb = a.final_state ? div_up((int64_t)a.seqs.num * (a.width - 1), kWaves) : 0;
    return g;
}
Grid bwd_grid(const ConvArgs &a, int vec) {
    Grid g = {div_up(a.channels, 64 * vec), 0, 0, 0};
    g.run = bwd_run_tokens(a.seqs.total, (int)g.cb);
    g.rb = div_up(a.seqs.total, (int64_t)g.run * kWaves);
    g.sb = a.d_state0 ? div_up(a.seqs.num, kWaves) : 0;
    return g;
}
Grid step_grid(const ConvArgs &a, int32_t batch, int vec) {
    return {div_up(a.channels, 64 * vec), div_up(batch, kWaves), 0, 0};
}
int64_t reduce_blocks(const ConvArgs &a) { return div_up((int64_t)a.channels * (a.width + 1), 64); }

template <typename T, int VEC, int W> int fwd(const ConvArgs &a, hipStream_t stream) {
    const Grid g = fwd_grid(a, VEC);
    if (g.blocks() == 0) return 0;
    hipLaunchKernelGGL((conv_fwd_kernel<T, VEC, W>), dim3((unsigned)g.blocks()), dim3(64, kWaves), 0,
                       stream, a, (int)g.cb, (int)g.rb, g.run);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T, int VEC, int W> int bwd(const ConvArgs &a, hipStream_t stream) {
    const Grid g = bwd_grid(a, VEC);
    if (g.blocks() > 0)
        hipLaunchKernelGGL((conv_bwd_kernel<T, VEC, W>), dim3((unsigned)g.blocks()),
                           dim3(64, kWaves), 0, stream, a, (int)g.cb, (int)g.rb, g.run);
    hipLaunchKernelGGL(conv_reduce_kernel, dim3((unsigned)reduce_blocks(a)), dim3(64, 16), 0, stream,
                       a.partial, (int)g.rb, a.channels, W, a.dweight, a.dbias);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T, int VEC, int W>
int step(const ConvArgs &a, void *state, int batch, hipStream_t stream) {
    const Grid g = step_grid(a, batch, VEC);
    hipLaunchKernelGGL((conv_step_kernel<T, VEC, W>), dim3((unsigned)g.blocks()), dim3(64, kWaves), 0,
                       stream, a, static_cast<T *>(state), (int)g.cb, batch);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

// Whether every row of every tensor of the call starts on a multiple of
// VEC elements (16 bytes, or 8 for the bf16 backward) and holds whole vectors.
bool wide(const ConvArgs &a, const void *state, int vec) {
    const int esz = a.dtype == kDtypeBf16 ? 2 : 4;
    const void *p[] = {a.x, a.state0, a.d_out, a.d_final, a.out, a.final_state, a.dx, a.d_state0,
                       state};
    for (const void *q : p)
        if (reinterpret_cast<uintptr_t>(q) % (uintptr_t)(vec * esz)) return false;
    if ((reinterpret_cast<uintptr_t>(a.weight) | reinterpret_cast<uintptr_t>(a.bias)) % 16)
        return false;
    return a.channels % vec == 0 && a.x_stride % vec == 0 && a.out_stride % vec == 0 &&
           a.d_out_stride % vec == 0 && a.dx_stride % vec == 0;
}

// Channels of a lane: 16-byte pieces, 8 in the bf16 backward, or one channel.
int vec_of(const ConvArgs &a, const void *state, bool backward) {
    const int vec = a.dtype == kDtypeBf16 && !backward ? 8 : 4;
    return wide(a, state, vec) ? vec : 1;
}

#define KDA_CONV_WIDTHS(fn, T, VEC, ...)                       \
    (a.width == 4   ? fn<T, VEC, 4>(__VA_ARGS__)               \
     : a.width == 3 ? fn<T, VEC, 3>(__VA_ARGS__)               \
                    : fn<T, VEC, 2>(__VA_ARGS__))

}  // namespace

int64_t conv_fwd_threads(const ConvArgs &a) {
    return fwd_grid(a, vec_of(a, nullptr, false)).blocks() * 64 * kWaves;
}
int64_t conv_bwd_threads(const ConvArgs &a) {
    const int64_t runs = bwd_grid(a, vec_of(a, nullptr, true)).blocks() * 64 * kWaves;
    const int64_t sums = reduce_blocks(a) * 1024;
    return runs > sums ? runs : sums;
}
int64_t conv_step_threads(const ConvArgs &a, const void *state, int32_t batch) {
    return step_grid(a, batch, vec_of(a, state, false)).blocks() * 64 * kWaves;
}

int launch_conv_fwd(const ConvArgs &a, hipStream_t stream) {
    if (a.dtype == kDtypeBf16)
        return vec_of(a, nullptr, false) == 8 ? KDA_CONV_WIDTHS(fwd, bf16, 8, a, stream)
                                   : KDA_CONV_WIDTHS(fwd, bf16, 1, a, stream);
    return vec_of(a, nullptr, false) == 4 ? KDA_CONV_WIDTHS(fwd, float, 4, a, stream)
                               : KDA_CONV_WIDTHS(fwd, float, 1, a, stream);
}

int launch_conv_bwd(const ConvArgs &a, hipStream_t stream) {
    if (a.dtype == kDtypeBf16)
        return vec_of(a, nullptr, true) == 4 ? KDA_CONV_WIDTHS(bwd, bf16, 4, a, stream)
                                   : KDA_CONV_WIDTHS(bwd, bf16, 1, a, stream);
    return vec_of(a, nullptr, true) == 4 ? KDA_CONV_WIDTHS(bwd, float, 4, a, stream)
                               : KDA_CONV_WIDTHS(bwd, float, 1, a, stream);
}

int64_t conv_bwd_workspace_floats(int64_t total, int64_t channels, int width) {
    // runs are 16 tokens or longer (bwd_run_tokens)
    const int64_t rows = (total + 16 * kWaves - 1) / (16 * kWaves);
    return rows * channels * (width + 1);
}

int launch_conv_step(const ConvArgs &a, void *state, int32_t batch, hipStream_t stream) {
    if (a.dtype == kDtypeBf16)
        return vec_of(a, state, false) == 8 ? KDA_CONV_WIDTHS(step, bf16, 8, a, state, batch, stream)
                                 : KDA_CONV_WIDTHS(step, bf16, 1, a, state, batch, stream);
    return vec_of(a, state, false) == 4 ? KDA_CONV_WIDTHS(step, float, 4, a, state, batch, stream)
                             : KDA_CONV_WIDTHS(step, float, 1, a, state, batch, stream);
}

}  // namespace kda
