// layer_device.h -- device helpers shared by the operators around the
// recurrence: vector loads and stores by element count, and the packed
// sequence a token belongs to.
#pragma once

#include "kda_device.h"
#include "kda_slots.h"
#include "layer_internal.h"

namespace kda {

// VEC consecutive elements of type T as floats.  VEC > 1 needs the address
// aligned to the vector's size (16 bytes at most per access).
template <typename T, int VEC> struct Row {
    typedef T vec __attribute__((ext_vector_type(VEC)));
    __device__ static vec raw(const T *p) { return *reinterpret_cast<const vec *>(p); }
    __device__ static void get(const vec &r, float (&f)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = to_f32(r[i]);
    }
    __device__ static void put(T *p, const float (&f)[VEC]) {
        vec r;
#pragma unroll
        for (int i = 0; i < VEC; ++i) r[i] = from_f32<T>(f[i]);
        *reinterpret_cast<vec *>(p) = r;
    }
    __device__ static vec zero() { return vec(T(0.f)); }
};
template <typename T> struct Row<T, 1> {
    typedef T vec;
    __device__ static vec raw(const T *p) { return *p; }
    __device__ static void get(const vec &r, float (&f)[1]) { f[0] = to_f32(r); }
    __device__ static void put(T *p, const float (&f)[1]) { *p = from_f32<T>(f[0]); }
    __device__ static vec zero() { return T(0.f); }
};

// End of sequence m, clamped into [0, total].
__device__ __forceinline__ int seq_end_token(const Seqs &q, int m) {
    if (!q.cu) return (m + 1) * q.seq_len;
    const int a = q.cu[m + 1];
    return a < 0 ? 0 : (a > q.total ? q.total : a);
}

// The sequence that holds token t (its tokens are [beg, end)): the last one
// that begins at or before t.  Returns -1 where none holds it (t behind the
// last offset, or malformed offsets).  q.num >= 1.
__device__ __forceinline__ int seq_of_token(const Seqs &q, int t, int *beg, int *end) {
    int m;
    if (!q.cu) {
        m = t / q.seq_len;
    } else {
        int lo = 0, hi = q.num - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_first_token(q.cu, q.seq_len, q.total, mid) <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        m = lo;
    }
    *beg = (int)seq_first_token(q.cu, q.seq_len, q.total, m);
    *end = seq_end_token(q, m);
    return t >= *beg && t < *end ? m : -1;
}

// 1 / (1 + e^-z) in fp32 (exp2 and reciprocal to one step of their result; e^-z
// may overflow to inf, which gives 0).
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-z * kLog2e));
}

}  // namespace kda
