// attn_device.h -- building blocks of the attention kernels over a paged cache:
// tiles of the cache in LDS, the products of a tile with 32 query rows, and the
// running maximum and sum of their softmax.
//
// Orientation.  Scores are formed as S^T = K Q^T in 32 x 32 tiles: lane l holds
// query row l % 32 and the sixteen tokens 8 (i / 4) + 4 (l / 32) + i % 4.  A
// row's maximum and sum are then in-lane operations and one exchange of the two
// halves, and the probabilities already lie as the second operand of
// O^T = V^T P^T, whose k order they set: for the 16 tokens of a step, slots
// 0..3 and 4..7 of a lane are tokens 4 (l / 32) + {0..3} and 8 on.
//
// Tiles.  The rows of K and V go from the cache to LDS without registers
// (global_load_lds, 16 bytes a lane), in the cache's order except that the
// 16-byte chunks of a row change places by an XOR with turn(row), done by the
// choice of each lane's source.  Rows 0..15 at one chunk (the reads of K) and
// four rows of four neighbouring chunks (the transposing reads of V) then fall
// on different banks.
#pragma once

#include "cache_device.h"

#include <type_traits>

namespace kda {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

// A tile of rows of C 16-byte chunks in LDS.
template <int C> __device__ __forceinline__ int tile_turn(int row) {
    return C % 16 == 0 ? ((row & 3) << 2) | ((row >> 2) & 3)
                       : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
}
template <int C> __device__ __forceinline__ int tile_at(int row, int chunk) {
    return (row * C + (chunk ^ tile_turn<C>(row))) * 16;
}

// The lane number as a value the compiler cannot trace: what is formed from it in a rare
// path is formed there and does not fill the registers as a constant of the loop around.
__device__ __forceinline__ int here(int lane) {
    asm volatile("" : "+v"(lane));
    return lane;
}

__device__ __forceinline__ float half_max(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Where the 16-byte chunks of a lane's row (token l % 32 of a tile) lie: pairs of them from
// pair c0 on, a half wave each; classes by the period of turn(), as for values.
template <int C> struct Keys {
    static constexpr int NK = C % 16 == 0 ? 8 : 4;
    int at[NK];
    __device__ __forceinline__ Keys(int c0, int lane) {
#pragma unroll
        for (int k = 0; k < NK; ++k) at[k] = tile_at<C>(lane & 31, 2 * (c0 + k) + (lane >> 5));
    }
    // Pair c0 + c of token 32 j + l % 32.
    __device__ __forceinline__ u32x4 read(lds_char *tile, int j, int c) const {
        return *(lds_u32x4 *)(tile + at[c % NK] + 32 * j * C * 16 + c / NK * NK * 32);
    }
};

// Products of one type of element.  chunk(): acc += over the channels of one
// 16-byte chunk per half wave.  Values: the operand of V^T for 16 tokens and 32
// channels of a tile of CH chunks a row; mma(): its product.
template <typename T> struct AttnMma;

template <> struct AttnMma<bf16> {
    struct Value { bf16x8 a; };
    typedef bf16x8 Prob;
    __device__ static f32x16 chunk(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    // Where the transposing reads of 32 channels from 32 d0 on, tokens 0..3 and 8..11 of each
    // half, lie for this lane.  turn() repeats after 16 rows and 8 or 16 chunks: NV classes of
    // d, the others by immediate offsets.
    template <int CH> struct Values {
        static constexpr int NV = CH % 16 == 0 ? 4 : 2;
        int at[NV][2];
        __device__ __forceinline__ Values(int d0, int lane) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int second = 0; second < 2; ++second) {
                    const int row = 8 * second + 4 * (lane >> 5) + ((lane & 15) >> 2);
                    const int col = 32 * (d0 + k) + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                    at[k][second] = tile_at<CH>(row, col >> 3) + (col & 7) * 2;
                }
        }
        // Tokens 16 j .. 16 j + 15, channels 32 (d0 + d) on (d0 a multiple of NV).
        __device__ __forceinline__ Value read(lds_char *tile, int j, int d) const {
            typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
            const int off = 16 * j * CH * 16 + d / NV * NV * 64;
            const bf16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                (lds_bf16x4 *)(tile + at[d % NV][0] + off));
            const bf16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                (lds_bf16x4 *)(tile + at[d % NV][1] + off));
            return {__builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7)};
        }
    };
    // Rounded once, by at most 2^-8 of each: an output is off by 2^-8 of sum p |v| at most beside
    // its own rounding (2.3e-3 of it on average against 1.7e-3).  A second part of what that leaves
    // out and a product more for it cost prompts 634 to 930 us, drafts 173 to 241, latent rows 170 to
    // 201, and of few rows alone 256K 208 to 213, 256 sessions behind 16K 271 to 289.
    __device__ static Prob prob(const f32x16 &s, int step) {
        Prob p;
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = static_cast<bf16>(s[8 * step + j]);
        return p;
    }
    __device__ static f32x16 mma(const Value &v, const Prob &p, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.a, p, c, 0, 0, 0);
    }
    // The operand with zeros where it is no number.
    __device__ static Value numbers(const Value &v) {
        u32x4 w = __builtin_bit_cast(u32x4, v.a);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = (w[e] & 0x7f80u) == 0x7f80u ? w[e] & 0xffff0000u : w[e];
            w[e] = (w[e] & 0x7f800000u) == 0x7f800000u ? w[e] & 0xffffu : w[e];
        }
        return {__builtin_bit_cast(bf16x8, w)};
    }
};

template <> struct AttnMma<float> {
    struct Value { float a[8]; };
    struct Prob { float p[8]; };
    __device__ static f32x16 chunk(u32x4 a, u32x4 b, f32x16 c) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c,
                                                     0, 0, 0);
        return c;
    }
    // Row 8 (e / 4) + 4 (l / 32) + e % 4, channel l % 32 on from 32 d.  What of turn(row) the
    // lane does not set is a constant, whose XOR with the lane's part is formed at each read: kept,
    // those of all reads would fill the registers.
    template <int CH> struct Values {
        static_assert(CH % 16 == 0, "rows over all banks");
        int base;
        __device__ __forceinline__ Values(int d0, int lane)
            : base((((lane & 31) >> 2) ^ (lane >> 5)) * 16 + (lane & 3) * 4 +
                   4 * (lane >> 5) * CH * 16 + d0 * 128) {}  // d0 even
        __device__ __forceinline__ Value read(lds_char *tile, int j, int d) const {
            typedef __attribute__((address_space(3))) float lds_float;
            Value v;
            const int at = here(base);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v.a[e] = *(lds_float *)(tile + (at ^ (((e % 4) << 2 ^ e / 4 << 1 ^ (d & 1) << 3) * 16)) +
                                        (16 * j + 8 * (e / 4) + e % 4) * CH * 16 + d / 2 * 256);
            return v;
        }
    };
    __device__ static Prob prob(const f32x16 &s, int step) {
        Prob p;
#pragma unroll
        for (int j = 0; j < 8; ++j) p.p[j] = s[8 * step + j];
        return p;
    }
    __device__ static f32x16 mma(const Value &v, const Prob &p, f32x16 c) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(v.a[e], p.p[e], c, 0, 0, 0);
        return c;
    }
    __device__ static Value numbers(const Value &v) {
        Value o;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o.a[e] = __builtin_fabsf(v.a[e]) < __builtin_inff() ? v.a[e] : 0.f;
        return o;
    }
};

// Splits.  A length of `units` (of kSplitTokens tokens) in at most `splits` parts
// of `per` units each, the last one shorter.
__device__ __forceinline__ int split_units(int units, int splits) {
    return splits > 0 ? (units + splits - 1) / splits : 0;
}
__device__ __forceinline__ int units_of(int tokens) {
    return (tokens + kSplitTokens - 1) / kSplitTokens;
}

__device__ __forceinline__ int prefix_tokens(const AttnArgs &a) {
    if (!a.prefix_width) return 0;
    const int64_t most = (int64_t)a.prefix_width * a.pages.size;
    const int n = word_at(a.prefix_len, 0);
    return n < 0 ? 0 : (n > most ? (int)most : n);
}

// Place of token `tok` in the page `entry`, in units of 2^shift bytes behind the start of its
// head; 0 (the first page's first token, which is there) for an entry that is no page.
__device__ __forceinline__ uint32_t token_place(const Pages &p, int entry, int tok, bool *there) {
    *there = entry >= 0 && entry < p.count;
    const uint32_t in = tok - p.by_size(tok) * (uint32_t)p.size;
    return *there ? (uint32_t)entry * p.page_units + in * p.token_units : 0;
}

// The first of `len` tokens (of a prefix, or of a session's own) whose page is there, len if none
// is.  A row whose exponentials come to a sum of zero asks this: it sees nothing where that token
// is not under its limit, and otherwise scores of -inf alone, whose softmax is no number.  64
// entries a step; called by whole waves with the same table and length.
__device__ __forceinline__ int first_there(const Pages &p, const int32_t *table, int len, int lane) {
    const int n = len > 0 ? p.by_size(len - 1) + 1 : 0;
#pragma unroll 1
    for (int i = 0; i < n; i += 64) {
        const int entry = i + lane < n ? table[i + lane] : -1;
        const unsigned long long m = __ballot(entry >= 0 && entry < p.count);
        if (m) return (i + __builtin_ctzll(m)) * p.size;
    }
    return len;
}

// 16 bytes a lane from memory to LDS at `to` + 16 * lane.  In assembly, so that the compiler
// does not wait for all loads on their way before each read of LDS; what is read is
// waited for by wait_loads().  m0 is read one wait state after it is written.
__device__ __forceinline__ void load_lds16(const char *from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(from), "s"(to)
                 : "memory");
}
// The same from an address that is the wave's and an offset under 2^32 that is the lane's.
__device__ __forceinline__ void load_lds16(const char *from, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %0"
                 :
                 : "s"(from), "v"(offset), "s"(to)
                 : "memory");
}
// Until at most N of this wave's loads are on their way.  The compiler knows this instruction:
// it does not wait again for its own loads from before.
template <int N> __device__ __forceinline__ void wait_loads() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | 15 << 8 | (N >> 4) << 14);
    asm volatile("" ::: "memory");
}

// The loads of rows of C chunks of ROWS tokens into a tile, 64 chunks each, wave `wave` of NW
// taking every NW-th.  set(): from each token's place, at its lane; load(): from any cache of
// that layout.  NEAR: every value of a head lies under 2^32 bytes behind its first.
template <int C, int ROWS, int NW, bool NEAR> struct TileLoads {
    static constexpr int LOADS = ROWS * C / 64, N = (LOADS + NW - 1) / NW;
    uint32_t at[N];
    __device__ static bool mine(int i, int wave) { return LOADS % NW == 0 || NW * i + wave < LOADS; }
    // Row and byte in the row of what this lane reads with load i.  (Rows that are no power of
    // two: formed again each time, to keep registers free.)
    __device__ static void part(int i, int wave, int lane, int *row, int *byte) {
        const int p = 64 * (NW * i + wave) + ((C & (C - 1)) != 0 ? here(lane) : lane);
        *row = p / C, *byte = ((p % C) ^ tile_turn<C>(*row)) * 16;
    }
    __device__ __forceinline__ void set(const Pages &pages, uint32_t place, int wave, int lane) {
        if (NEAR) place <<= pages.shift;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int row, byte;
            part(i, wave, lane, &row, &byte);
            at[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (row < ROWS ? row : 0), (int)place);
        }
    }
    __device__ __forceinline__ void load(const Pages &pages, const char *cache, lds_char *tile,
                                         int wave, int lane) const {
        const uint32_t to = (uint32_t)(uintptr_t)tile + 1024 * wave;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!mine(i, wave)) break;
            int row, byte;
            part(i, wave, lane, &row, &byte);
            if (NEAR)
                load_lds16(cache, at[i] + byte, to + 1024 * NW * i);
            else
                load_lds16(cache + ((uint64_t)at[i] << pages.shift) + byte, to + 1024 * NW * i);
        }
    }
};
// Rows of tokens that are not there (valid) to zeros: their product with a probability of zero
// has to be zero.  Each wave clears what it has loaded, once that has come.
template <int C, int ROWS, int NW>
__device__ __forceinline__ void clear_rows(lds_char *tile, uint64_t valid, int wave, int lane) {
    constexpr int LOADS = ROWS * C / 64;
#pragma unroll 1
    for (int load = wave; load < LOADS; load += NW) {
        const int p = 64 * load + here(lane), row = p / C;
        if (!((valid >> row) & 1)) *(lds_u32x4 *)(tile + 16 * p) = u32x4{0u, 0u, 0u, 0u};
    }
}

// Whether one of the 16-byte chunks lane, lane + 64, .. under `chunks` of a tile holds a NaN
// or an infinity, of any lane.
template <typename T>
__device__ __forceinline__ bool any_odd(lds_char *tile, int chunks, int lane) {
    bool odd = false;
    for (int i = lane; i < chunks; i += 64) {
        const u32x4 w = *(lds_u32x4 *)(tile + 16 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            odd |= (w[e] & 0x7f800000u) == 0x7f800000u ||
                   (sizeof(T) == 2 && (w[e] & 0x7f80u) == 0x7f80u);
    }
    return __ballot(odd) != 0;
}

// Workgroup barrier that waits for this wave's LDS operations only: loads stay on their way.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A maximum that may stand in an exponent's difference.
__device__ __forceinline__ float usable(float m) { return m == -__builtin_inff() ? 0.f : m; }

// Scores of tokens that are not there (valid) or lie at or behind the row's `ahead`-th of
// the tile's become -inf.
template <int TT>
__device__ __forceinline__ void hide_scores(f32x16 (&s)[TT], uint64_t valid, int ahead, int lane) {
    // bit 8 (e / 4) + e % 4 of word j: whether this lane's row sees its token e
    uint64_t see = ahead <= 0 ? 0 : (ahead < 32 * TT ? valid & ~(~0ull << ahead) : valid);
    see >>= 4 * (here(lane) >> 5);
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const uint32_t word = (uint32_t)(see >> (32 * j));
#pragma unroll
        for (int e = 0; e < 16; ++e)
            s[j][e] = word & (1u << (8 * (e / 4) + e % 4)) ? s[j][e] : -__builtin_inff();
    }
}

// The running maximum m over a tile's scores; what stands against the old one moves with it.
template <int TT, int DT>
__device__ __forceinline__ void move_maximum(const f32x16 (&s)[TT], float &m, float &l,
                                             f32x16 (&o)[DT], float sl) {
    float top = s[0][0];
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = __builtin_fmaxf(top, s[j][e]);
    top = half_max(top);
    // The maximum moves on only where a score passes it by 2^8 (at first by any): exponents
    // up to 8 lose nothing in fp32, and the steps of their bf16 values are relative.
    if (__ballot((top - m) * sl > 8.f)) {
        const float to = __builtin_fmaxf(m, top), f = fast_exp2((m - usable(to)) * sl);
        m = to, l *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= f;
    }
}
// Scores to probabilities relative to m, their sum into l.
template <int TT>
__device__ __forceinline__ void soften(f32x16 (&s)[TT], float m, float &l, float sl) {
    const float ms = usable(m) * sl;
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            s[j][e] = fast_exp2(s[j][e] * sl - ms);
            l += s[j][e];
        }
}

// S^T of 32 * TT tokens: KS chunk pairs of their rows with those of the queries, q(pair).
template <typename T, int KS, int C, int TT, typename Q>
__device__ __forceinline__ void scores(lds_char *tile, const Keys<C> &keys, Q q, f32x16 (&s)[TT]) {
#pragma unroll
    for (int c = 0; c < KS; ++c)
#pragma unroll
        for (int j = 0; j < TT; ++j)
            s[j] = AttnMma<T>::chunk(keys.read(tile, j, c), q(c), c ? s[j] : f32x16(0.f));
}

// o += V^T P^T over a tile's tokens, DT * 32 channels.  NUMBERS: what is no number (an infinity
// or a NaN) is left out: a product would carry it to rows that do not see its token (0 * inf).
template <typename T, bool NUMBERS, int TT, int DT, typename V>
__device__ __forceinline__ void add_values(const f32x16 (&s)[TT], lds_char *tile, const V &values,
                                           f32x16 (&o)[DT]) {
    typedef AttnMma<T> M;
#pragma unroll
    for (int j = 0; j < 2 * TT; ++j) {
        const typename M::Prob p = M::prob(s[j / 2], j % 2);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const typename M::Value v = values.read(tile, j, d);
            o[d] = M::mma(NUMBERS ? M::numbers(v) : v, p, o[d]);
        }
    }
}

// What add_values has left out of tokens [from, to) of one session, added for the rows that
// see it: row l % 32 of this wave sees the tokens under lim.  Values from the cache itself.
template <typename T, int DT>
__device__ __forceinline__ void add_others(const Pages &pages, const int32_t *table, const char *vc,
                                           int from, int to, int d0, int lim, int lane,
                                           f32x16 (&o)[DT]) {
    const int half = lane >> 5;
#pragma unroll 1
    for (int tok = from; tok < to; ++tok) {
        bool there;
        const uint32_t place = token_place(pages, table[pages.by_size(tok)], tok, &there);
        if (!there) continue;
        const T *row = reinterpret_cast<const T *>(vc + ((uint64_t)place << pages.shift));
        const bool see = tok < lim;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = to_f32(row[32 * (d0 + d) + 8 * k + 4 * half + i]);
                    o[d][4 * k + i] += see && !(__builtin_fabsf(x) < __builtin_inff()) ? x : 0.f;
                }
    }
}

// A tile's probabilities (s, against m) and their products with its values, and beside them the
// scores of the next tile, in one stream that keeps the matrix unit fed: operands are read from
// LDS kAhead products before they are used, and the exponentials stand between the products of
// the next scores, which do not depend on them.  The fences keep the compiler from moving each
// read to its product, where its latency would be waited for.  beside(i): what else is done
// with product i of the values, which have little beside them.
constexpr int kAhead = 4;
template <typename T, int C, int TT, int KS, int DT, typename V, typename F>
__device__ __forceinline__ void turn_over(lds_char *kt, lds_char *vt, const Keys<C> &keys,
                                          const V &values, const u32x4 (&q)[KS], f32x16 (&s)[TT],
                                          f32x16 (&next)[TT], float m, float &l, f32x16 (&o)[DT],
                                          float sl, F beside) {
    typedef AttnMma<T> M;
    constexpr int QK = TT * KS, PV = 2 * TT * DT, E = 16 * TT;
    static_assert(QK >= kAhead && PV >= kAhead, "operands ahead");
    u32x4 k[kAhead];
    typename M::Value v[kAhead];
    typename M::Prob p[2 * TT];
    const float ms = usable(m) * sl;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) k[i] = keys.read(kt, i % TT, i / TT);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < QK; ++i) {
        const int j = i % TT, c = i / TT, to = i + kAhead;
        next[j] = M::chunk(k[i % kAhead], q[c], c ? next[j] : f32x16(0.f));
        if (to < QK)
            k[i % kAhead] = keys.read(kt, to % TT, to / TT);
        else
            v[to - QK] = values.read(vt, (to - QK) / DT, (to - QK) % DT);
#pragma unroll
        for (int e = i * E / QK; e < (i + 1) * E / QK; ++e) {
            const float x = fast_exp2(s[e / 16][e % 16] * sl - ms);
            s[e / 16][e % 16] = x;
            l += x;
            if (e % 8 == 7) p[e / 8] = M::prob(s[e / 16], e / 8 % 2);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < PV; ++i) {
        const int d = i % DT, to = i + kAhead;
        o[d] = M::mma(v[i % kAhead], p[i / DT], o[d]);
        if (to < PV) v[i % kAhead] = values.read(vt, to / DT, to % DT);
        beside(i);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The two halves of that on their own.  Scores of 32 tokens, operands read kNear products
// ahead (registers are few here); keys(pair) reads one.
constexpr int kNear = 3;
template <typename T, int KS, typename K, typename Q>
__device__ __forceinline__ void scores_ahead(K keys, Q q, f32x16 &s) {
    u32x4 k[kNear];
#pragma unroll
    for (int c = 0; c < kNear; ++c) k[c] = keys(c);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < KS; ++c) {
        s = AttnMma<T>::chunk(k[c % kNear], q(c), c ? s : f32x16(0.f));
        if (c + kNear < KS) k[c % kNear] = keys(c + kNear);
        __builtin_amdgcn_sched_barrier(0);
    }
}
// Probabilities of 32 tokens and their products with the values; the second sixteen tokens'
// exponentials stand beside the products of the first.
template <typename T, int DT, typename V>
__device__ __forceinline__ void values_ahead(lds_char *vt, const V &values, f32x16 &s, float m,
                                             float &l, f32x16 (&o)[DT], float sl) {
    typedef AttnMma<T> M;
    const float ms = usable(m) * sl;
    auto soften1 = [&](int e) {
        s[e] = fast_exp2(s[e] * sl - ms);
        l += s[e];
    };
    typename M::Value v[kNear];
#pragma unroll
    for (int i = 0; i < kNear; ++i) v[i] = values.read(vt, i / DT, i % DT);
#pragma unroll
    for (int e = 0; e < 8; ++e) soften1(e);
    typename M::Prob p = M::prob(s, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) {
        const int to = i + kNear;
        if (i == DT) p = M::prob(s, 1);
        o[i % DT] = M::mma(v[i % kNear], p, o[i % DT]);
        if (to < 2 * DT) v[i % kNear] = values.read(vt, to / DT, to % DT);
        if (i < DT) {
#pragma unroll
            for (int e = 8 + i * 8 / DT; e < 8 + (i + 1) * 8 / DT; ++e) soften1(e);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

}  // namespace kda
