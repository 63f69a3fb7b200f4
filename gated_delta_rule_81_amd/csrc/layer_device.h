// layer_device.h -- device helpers shared by the operators around the
// recurrence: vector loads and stores by element count, and the packed
// sequence a token belongs to.
#pragma once

#include "kda_device.h"
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

// Packed offset i, clamped into [0, total].  Offsets are not written while a kernel
// runs: read as constants, at an index that is the same for the whole wave they
// come through scalar loads, which do not queue behind the wave's row loads.
__device__ __forceinline__ int offset_at(const Seqs &q, int i) {
    typedef const __attribute__((address_space(4))) int32_t constant_i32;
    const int a = ((constant_i32 *)(uintptr_t)q.cu)[i];
    return a < 0 ? 0 : (a > q.total ? q.total : a);
}
// First token of sequence m and the one behind its last.
__device__ __forceinline__ int seq_first(const Seqs &q, int m) {
    return q.cu ? offset_at(q, m) : m * q.seq_len;
}
__device__ __forceinline__ int seq_end_token(const Seqs &q, int m) {
    return q.cu ? offset_at(q, m + 1) : (m + 1) * q.seq_len;
}

// The sequence that holds token t (its tokens are [beg, end)): the last one
// that begins at or before t.  Returns -1 where none holds it (t behind the
// last offset, or malformed offsets).  q.num >= 1.
__device__ __forceinline__ int seq_of_token(const Seqs &q, int t, int *beg, int *end) {
    int lo = 0, hi = q.num - 1;
    if (!q.cu) lo = hi = t / q.seq_len;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offset_at(q, mid) <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    *beg = seq_first(q, lo);
    *end = seq_end_token(q, lo);
    return t >= *beg && t < *end ? lo : -1;
}

// 1 / (1 + e^-z) in fp32 (exp2 and reciprocal to one step of their result; e^-z
// may overflow to inf, which gives 0).
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-z * kLog2e));
}

}  // namespace kda
