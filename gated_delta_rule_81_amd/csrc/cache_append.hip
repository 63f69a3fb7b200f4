// cache_append.hip -- new keys and values into a paged cache, the keys (and the
// queries beside them) rotated by position on the way.
//
//   (a, b) <- (a cos - b sin, b cos + a sin) on channel pairs of a window
//
// Every value is read once and written once, so HBM bounds long calls and the
// latency of one chain (lens, page, cache row) short ones.  A lane takes sixteen
// channels of a head as two 16-byte pieces (of bf16) that lie half the window, or half of
// what is outside it, apart: both members of its pairs, so that no value crosses
// lanes.  A wave works on ONE token, whose session, page and cos | sin row are
// then the same for all of its lanes.  Two pieces a lane are loaded before the
// place they go to is known, so that both chains run beside each other.
//
// Measured: 32K tokens of 32 + 8 + 8 heads of 128, bf16, 0.77 GB read and written: 151 us,
// 5.1 TB/s, the rate of a large copy.  One token of 256 sessions: 4.5 us, of three: 3.1.
#include "cache_device.h"

namespace kda {
namespace {

// Pieces of a wave's unit whose loads are in flight together, and waves of a workgroup.
constexpr int kSteps = 2, kWaves = 4;

// Sixteen channels of a head: two pieces of eight, and where in the cos | sin row
// their angles begin (non-rotated: turn < 0).
struct Piece {
    int a, b, turn;
};
template <int D> __device__ __forceinline__ Piece piece_of(int u, int rot, int rot_at) {
    Piece p;
    if (u * 16 < rot) {
        p.a = rot_at + 8 * u, p.b = p.a + rot / 2, p.turn = 8 * u;
        return p;
    }
    const int k = u - rot / 16, m = (D - rot) / 16;  // pieces k and k + m of those outside
    p.a = 8 * k, p.b = 8 * (k + m), p.turn = -1;
    if (p.a >= rot_at) p.a += rot;
    if (p.b >= rot_at) p.b += rot;
    return p;
}

__device__ __forceinline__ void turn_pairs(const float *row, int rot, const Piece &p,
                                           bool interleaved, float (&x)[8], float (&y)[8]) {
    const int half = rot / 2;
    if (interleaved) {  // channels 2 i, 2 i + 1 of both pieces
        const f32x4 ca = *reinterpret_cast<const f32x4 *>(row + p.turn / 2);
        const f32x4 sa = *reinterpret_cast<const f32x4 *>(row + half + p.turn / 2);
        const f32x4 cb = *reinterpret_cast<const f32x4 *>(row + half / 2 + p.turn / 2);
        const f32x4 sb = *reinterpret_cast<const f32x4 *>(row + half + half / 2 + p.turn / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1], c = y[2 * i], d = y[2 * i + 1];
            x[2 * i] = a * ca[i] - b * sa[i], x[2 * i + 1] = b * ca[i] + a * sa[i];
            y[2 * i] = c * cb[i] - d * sb[i], y[2 * i + 1] = d * cb[i] + c * sb[i];
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 4) {  // x and y are the pairs' two channels
        const f32x4 c = *reinterpret_cast<const f32x4 *>(row + p.turn + j);
        const f32x4 s = *reinterpret_cast<const f32x4 *>(row + half + p.turn + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[j + i], b = y[j + i];
            x[j + i] = a * c[i] - b * s[i], y[j + i] = b * c[i] + a * s[i];
        }
    }
}

// Unit: (token, group of kSteps * 64 pieces of its heads of q, k and v).
template <typename T, int D>
__global__ __launch_bounds__(64 * kWaves) void append_kernel(AppendArgs a, int groups,
                                                             int64_t unit0) {
    constexpr int PER = D / 16;  // pieces of a head
    typedef typename Vec8<T>::raw Raw;
    const int lane = threadIdx.x & 63;
    const int64_t unit = unit0 + (int64_t)blockIdx.x * kWaves +
                         __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t token = unit / groups;
    if (token >= a.seqs.tokens) return;
    const Sessions &q = a.seqs;
    const int s = q.cu ? session_search(q, token, lane, [](int first, int) { return first; })
                       : (int)(token / q.each);
    const int beg = session_first(q, s), end = session_first(q, s + 1);
    if (token < beg || token >= end) return;  // in no session
    const int hq = a.q_heads, hk = a.kv_heads, heads = hq + (a.v ? 2 : 1) * hk;
    const int i0 = (int)(unit % groups) * kSteps * 64 + lane;
    Raw ra[kSteps], rb[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int idx = i0 + 64 * i, head = idx / PER;
        ra[i] = rb[i] = Vec8<T>::zero();
        if (head >= heads) continue;
        const Piece p = piece_of<D>(idx % PER, head < hq + hk ? a.rot : 0, a.rot_at);
        const T *x = head < hq ? static_cast<const T *>(a.q) + token * a.q_stride + (int64_t)head * D
                     : head < hq + hk
                         ? static_cast<const T *>(a.k) + token * a.k_stride + (int64_t)(head - hq) * D
                         : static_cast<const T *>(a.v) + token * a.v_stride +
                               (int64_t)(head - hq - hk) * D;
        ra[i] = load8(x + p.a), rb[i] = load8(x + p.b);
    }
    // the token's place in the cache
    const int at = own_tokens(q, a.pages, s) - (end - beg) + (int)(token - beg);
    int page = -1;
    if (at >= 0) page = word_at(q.table, (int64_t)s * q.width + at / a.pages.size);
    const bool kept = page >= 0 && page < a.pages.count;
    const int64_t place = (int64_t)page * a.pages.page + (int64_t)(at % a.pages.size) * a.pages.token;
    const float *row = nullptr;
    if (a.rot) {
        int pos = word_at(a.positions, token);
        pos = pos < 0 ? 0 : (pos >= a.table_rows ? a.table_rows - 1 : pos);
        row = a.table + (int64_t)pos * a.rot;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int idx = i0 + 64 * i, head = idx / PER;
        if (head >= heads || (head >= hq && !kept)) continue;
        const Piece p = piece_of<D>(idx % PER, head < hq + hk ? a.rot : 0, a.rot_at);
        T *y;
        if (head < hq) {
            y = static_cast<T *>(a.out_q) + token * a.out_q_stride + (int64_t)head * D;
        } else {
            char *cache = static_cast<char *>(head < hq + hk ? a.k_cache : a.v_cache);
            y = reinterpret_cast<T *>(cache + place +
                                      (int64_t)(head < hq + hk ? head - hq : head - hq - hk) *
                                          a.pages.head);
        }
        if (p.turn < 0) {  // as it is, NaN included
            *reinterpret_cast<Raw *>(y + p.a) = ra[i];
            *reinterpret_cast<Raw *>(y + p.b) = rb[i];
            continue;
        }
        float u[8], v[8];
        Vec8<T>::to_float(ra[i], u);
        Vec8<T>::to_float(rb[i], v);
        turn_pairs(row, a.rot, p, a.interleaved, u, v);
        store8(y + p.a, u), store8(y + p.b, v);
    }
}

int groups_of(const AppendArgs &a) {
    const int64_t heads = (int64_t)a.q_heads + (int64_t)(a.v ? 2 : 1) * a.kv_heads;
    const int64_t pieces = heads * (a.head_dim / 16);
    return (int)((pieces + 64 * kSteps - 1) / (64 * kSteps));
}

template <typename T, int D> int append(const AppendArgs &a, hipStream_t stream) {
    const int groups = groups_of(a);
    const int64_t units = (int64_t)a.seqs.tokens * groups;
    constexpr int64_t kMost = (int64_t)1 << 25;  // a launch holds less than 2^32 threads
    for (int64_t u = 0; u < units; u += kMost) {
        const int64_t now = units - u < kMost ? units - u : kMost;
        hipLaunchKernelGGL((append_kernel<T, D>), dim3((unsigned)((now + kWaves - 1) / kWaves)),
                           dim3(64 * kWaves), 0, stream, a, groups, u);
    }
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T> int append_dims(const AppendArgs &a, hipStream_t stream) {
    if (a.head_dim == 64) return append<T, 64>(a, stream);
    return a.head_dim == 128 ? append<T, 128>(a, stream) : append<T, 576>(a, stream);
}

}  // namespace

int launch_cache_append(const AppendArgs &a, hipStream_t stream) {
    return a.dtype == kDtypeBf16 ? append_dims<bf16>(a, stream) : append_dims<float>(a, stream);
}

}  // namespace kda
