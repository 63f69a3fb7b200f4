// ssm_step.hip -- one token of the state space scan for every session: stream
// each state row once, update it in place, read the output.
//
//   m_p <- e^{dt A} m_p + (dt x_p) B,   y_p = <m_p, C> + D x_p
//
// on the state's rows m_p (N floats each).  Every state byte is read once and
// written once with 3 operations a value, so HBM bounds it: 16-byte loads and
// stores, all of a workgroup's rows in flight before the arithmetic, and the
// sum over a row's N / 4 lanes by DPP and permlane, off the LDS pipe.  256 sessions
// x 96 heads of 128 x 128, 3.2 GB: 556 us, 5.8 TB/s (a copy of such a size: 4.9).
// 3 sessions x 10 heads of 64 x 128: 3 us, the latency of one load and one store.
#include "kda_lanes.h"
#include "layer_device.h"

namespace kda {
namespace {

// Sum over the N / 4 = 16 or 32 lanes of a row, in every lane of it.
template <int LANES> __device__ __forceinline__ float row_sum(float x) {
    x = row16_total(x);
    return LANES == 32 ? xor16_sum(x) : x;
}

// One workgroup (4 waves) per (session, head, ROWS state rows).
template <typename T, int P, int N, int ROWS>
__global__ __launch_bounds__(kSsmStepThreads) void ssm_step_kernel(SsmStep a) {
    constexpr int LANES = N / 4, PER = 64 / LANES, STEPS = ROWS / (4 * PER);
    static_assert(STEPS * 4 * PER == ROWS, "rows over waves");
    const int64_t unit = blockIdx.x / (P / ROWS);  // session * heads + head
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = 4 * (lane % LANES);
    const int row0 = (int)(blockIdx.x % (P / ROWS)) * ROWS + wave * (ROWS / 4) + lane / LANES;
    float *S = a.state + unit * (int64_t)(P * N) + n0;
    f32x4 m[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        m[i] = __builtin_nontemporal_load(
            reinterpret_cast<const f32x4 *>(S + (int64_t)(row0 + i * PER) * N));
    const int64_t b = unit / a.heads;
    const int h = (int)(unit % a.heads), group = h / (a.heads / a.groups);
    const T *x = static_cast<const T *>(a.x) + b * a.x_stride + (int64_t)h * P;
    float Bf[4], Cf[4];
    Row<T, 4>::get(Row<T, 4>::raw(static_cast<const T *>(a.B) + b * a.b_stride + group * N + n0), Bf);
    Row<T, 4>::get(Row<T, 4>::raw(static_cast<const T *>(a.C) + b * a.c_stride + group * N + n0), Cf);
    const float dt = a.dt[unit], decay = fast_exp2(dt * a.A[h] * kLog2e);
    const float D = a.D ? a.D[h] : 0.f;
    T *out = static_cast<T *>(a.out) + b * a.out_stride + (int64_t)h * P;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int row = row0 + i * PER;
        const float xv = to_f32(x[row]), u = dt * xv;
        float y = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            m[i][e] = m[i][e] * decay + u * Bf[e];
            y += m[i][e] * Cf[e];
        }
        __builtin_nontemporal_store(m[i], reinterpret_cast<f32x4 *>(S + (int64_t)row * N));
        y = row_sum<LANES>(y);
        if (n0 == 0) out[row] = from_f32<T>(a.D ? y + D * xv : y);
    }
}

template <typename T, int P, int N> int step(const SsmStep &a, hipStream_t stream) {
    const int64_t units = (int64_t)a.batch * a.heads;
    // few units: a quarter of the rows each, so that four times the CUs take part
    if (units * 4 <= 1024)
        hipLaunchKernelGGL((ssm_step_kernel<T, P, N, P / 4>), dim3((unsigned)(units * 4)),
                           dim3(kSsmStepThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((ssm_step_kernel<T, P, N, P>), dim3((unsigned)units), dim3(kSsmStepThreads), 0,
                           stream, a);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T> int step_dims(const SsmStep &a, hipStream_t stream) {
    if (a.p == 64) return a.n == 64 ? step<T, 64, 64>(a, stream) : step<T, 64, 128>(a, stream);
    return a.n == 64 ? step<T, 128, 64>(a, stream) : step<T, 128, 128>(a, stream);
}

}  // namespace

int launch_ssm_step(const SsmStep &a, int dtype, hipStream_t stream) {
    return dtype == kDtypeBf16 ? step_dims<bf16>(a, stream) : step_dims<float>(a, stream);
}

}  // namespace kda
