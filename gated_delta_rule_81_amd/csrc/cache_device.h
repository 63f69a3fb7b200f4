// cache_device.h -- device helpers shared by the operators on a paged cache: the
// session a new token belongs to, and places in the cache.
#pragma once

#include "cache_internal.h"
#include "kda_device.h"

namespace kda {

// Read-only words at an index that is the same for the whole wave: scalar loads.
__device__ __forceinline__ int word_at(const int32_t *p, int64_t i) {
    typedef const __attribute__((address_space(4))) int32_t constant_i32;
    return ((constant_i32 *)(uintptr_t)p)[i];
}

// First new token of session s (s up to num), inside [0, tokens] whatever cu holds.
__device__ __forceinline__ int session_first(const Sessions &q, int s) {
    if (!q.cu) return s * q.each;
    const int a = word_at(q.cu, s);
    return a < 0 ? 0 : (a > q.tokens ? q.tokens : a);
}

// The last session s of [0, num) for which f(session_first(s), s) <= x, 0 if there
// is none; f does not fall as s grows.  64 sessions a step: the lanes of a wave
// look at one each.  Called by whole waves with the same x.
template <typename F>
__device__ __forceinline__ int session_search(const Sessions &q, int64_t x, int lane, F f) {
    int lo = 0, n = q.num;  // the session is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int64_t at = lo + (int64_t)lane * step;  // 64 * step may pass 2^31
        bool le = false;
        if (at < (int64_t)lo + n) {
            int first = (int)at * q.each;
            if (q.cu) {
                first = q.cu[at];
                first = first < 0 ? 0 : (first > q.tokens ? q.tokens : first);
            }
            le = f(first, (int)at) <= x;
        }
        const unsigned long long m = __ballot(le);
        const int hit = m ? 63 - __builtin_clzll(m) : 0;
        const int64_t left = (int64_t)n - (int64_t)hit * step;
        lo += hit * step;
        n = left < step ? (int)left : step;
    }
    return lo;
}

// Own tokens of session s, inside what its pages hold.
__device__ __forceinline__ int own_tokens(const Sessions &q, const Pages &p, int s) {
    const int64_t most = (int64_t)q.width * p.size;
    const int len = word_at(q.lens, s);
    return len < 0 ? 0 : (len > most ? (int)most : len);
}

}  // namespace kda
