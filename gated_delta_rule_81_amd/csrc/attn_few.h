// attn_few.h -- attention of few query rows (at most 32: one token's heads of a group, or a
// few tokens') over a long cache.
//
// Every key and value is read once and meets few rows, so memory bounds it: what counts is bytes
// on their way.  The rows are one operand of 32 columns (empty ones repeat the last row: the
// matrix unit has room).  A wave streams tiles of 32 tokens of its own through LDS, without
// barriers; four waves share a workgroup, each taking every fourth tile, and join their
// (maximum, sum, output) at the end; two workgroups a CU.  With keys and values each in a place
// of their own, one comes while the other is read.
//
// Measured: bf16, one token of 128 sessions of 500 to 7900 own tokens, 8 heads of 128, 2.2 GB:
// 386 us and 6 for the join, 5.6 TB/s (through the tile walk of many rows, whose waves share
// a tile: 458).  fp32, 24 sessions of up to 700 tokens behind 2001 shared, 16 heads of 128, with the
// prefix in the tile walk: 49 and 6 us; 124 with both there.
#pragma once

#include "attn_device.h"

namespace kda {

constexpr int kFewTile = 32;  // tokens of a wave's tile

// What a part (its maximum in units of log 2, its sum) counts beside others: nothing where its
// maximum is -inf, unless its scores were no numbers, which its sum then is not either.
__device__ __forceinline__ float part_weight(const float2 &part, float top) {
    return part.x > -__builtin_inff() ? fast_exp2(part.x - top) : (part.y == 0.f ? 0.f : part.y);
}

template <typename T, int D, int NW, int PLACES> struct FewShape {
    static constexpr int C = D * (int)sizeof(T) / 16;   // 16-byte chunks of a row
    static constexpr int BUF = kFewTile * C * 16;       // keys or values of a tile
    static constexpr int LOADS = kFewTile * C / 64;
    static constexpr int LD = D + 4;                    // floats between rows of the joined output
    static constexpr int RING = NW * PLACES * BUF, JOIN = NW * 32 * LD * 4;
    static constexpr int LDS = (RING > JOIN ? RING : JOIN) + NW * 32 * 8;
};

// One workgroup per (session, kv head, split), or per (kv head, split) of the prefix.
template <typename T, int D, int NW, int PLACES, bool NEAR>
__device__ __forceinline__ void few_walk(const AttnArgs &a, int own_blocks, int block, char *smem) {
    typedef FewShape<T, D, NW, PLACES> S;
    constexpr int DT = D / 32, KS = S::C / 2;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, G = a.group;
    const bool pre = block >= own_blocks;
    const int b = pre ? block - own_blocks : block;
    const int splits = pre ? a.plan.prefix_splits : a.plan.own_splits;
    const int split = b % splits, hk = b / splits % a.kv_heads, session = b / splits / a.kv_heads;
    int tok0 = 0, n = a.seqs.tokens, len;
    if (pre) {
        len = prefix_tokens(a);
    } else {
        tok0 = session_first(a.seqs, session);
        n = session_first(a.seqs, session + 1) - tok0;
        len = own_tokens(a.seqs, a.pages, session);
    }
    if (n <= 0 || (int64_t)n * G > 32) return;
    const int rows = n * G;
    const int units = units_of(len), per = split_units(units, splits);
    if (split * per >= units && (split > 0 || a.part)) return;
    auto seen = [&](int row) { return pre ? len : len - n + row / G + 1; };
    const int64_t to = (int64_t)(split + 1) * per * kSplitTokens;
    const int beg = split * per * kSplitTokens, end = to < len ? (int)to : len;
    const int32_t *table = pre ? a.prefix_pages : a.seqs.table + (int64_t)session * a.seqs.width;

    const int row = (lane & 31) < rows ? lane & 31 : rows - 1;
    const int lim = seen(row), lim_min = seen(0);
    u32x4 q[KS];
    {
        const T *src = static_cast<const T *>(a.q) + (int64_t)(tok0 + row / G) * a.q_stride +
                       ((int64_t)hk * G + row % G) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[s] = *reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(src) +
                                                    16 * (2 * s + half));
    }
    const char *kc = static_cast<const char *>(a.k_cache) + (int64_t)hk * a.pages.head;
    const char *vc = static_cast<const char *>(a.v_cache) + (int64_t)hk * a.pages.head;
    // This wave's tiles are its own, every NW-th, in places of LDS that no other wave reads, so
    // that only its own loads are waited for: keys in one place and values in the other, each
    // loaded again as soon as it has been read (PLACES 1: both in one, in turn).
    lds_char *kt = (lds_char *)smem + wave * (PLACES * S::BUF), *vt = kt + (PLACES - 1) * S::BUF;
    const int tiles = a.pages.count > 0 ? (end - beg + kFewTile - 1) / kFewTile : 0;
    const int count = tiles > wave ? (tiles - wave + NW - 1) / NW : 0;
    auto base_of = [&](int k) { return beg + (k * NW + wave) * kFewTile; };
    // Where this lane's token of tile k lies; a window of 64 entries of the page table is held in
    // the lanes.
    int first = 0, entries = -1;
    bool held = false;
    auto where = [&](int k, uint32_t *valid) -> uint32_t {
        const int base = base_of(k), tok = base + lane;
        const int stop = base + kFewTile < end ? base + kFewTile : end;
        const int lo = a.pages.by_size(base), hi = a.pages.by_size(stop - 1);
        if (!held || hi - first >= 64) {
            const int most = a.pages.by_size(end - 1);
            held = true, first = lo;
            entries = table[lo + lane < most ? lo + lane : most];
        }
        const int idx = a.pages.by_size(tok < stop ? tok : base);
        int entry = __builtin_amdgcn_ds_bpermute(4 * (idx - first), entries);
        entry = tok < stop ? entry : -1;
        bool there;
        const uint32_t place = token_place(a.pages, entry, tok, &there);
        *valid = (uint32_t)__ballot(there);
        return place;
    };
    TileLoads<S::C, kFewTile, 1, NEAR> loads;
    auto load = [&](const char *cache, lds_char *to) { loads.load(a.pages, cache, to, 0, lane); };

    f32x16 o[DT];
    float m = -__builtin_inff(), l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16(0.f);
    const float sl = a.scale * kLog2e;
    const Keys<S::C> keys(0, lane);
    const typename AttnMma<T>::template Values<S::C> values(0, lane);
    uint32_t valid = 0, next_valid = 0;
    if (count > 0) loads.set(a.pages, where(0, &valid), 0, lane);
    wait_loads<0>();  // the queries, which have come with the entries: not waited for again
    if (count > 0) {
        load(kc, kt);
        if (PLACES == 2) load(vc, vt);
    }
    bool odd = false;  // a value that is no number in a tile that not all rows see whole
    // One tile; LATER: some row may not see some token of it.
    auto step = [&](int k, auto LATER) {
        constexpr bool later = decltype(LATER)::value;
        const bool more = k + 1 < count;
        const int base = base_of(k);
        wait_loads<PLACES == 2 ? S::LOADS : 0>();  // the keys; the values are behind them
        f32x16 s[1];
        scores<T, KS>(kt, keys, [&](int c) { return q[c]; }, s);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read, before they are loaded again
        if (PLACES == 1) load(vc, vt);
        if (more) loads.set(a.pages, where(k + 1, &next_valid), 0, lane);
        if (PLACES == 2 && more) load(kc, kt);
        if (later || valid != ~0u) hide_scores<1>(s, valid, later ? lim - base : kFewTile, lane);
        move_maximum<1, DT>(s, m, l, o, sl);
        soften<1>(s, m, l, sl);
        if (PLACES == 2 && more)
            wait_loads<S::LOADS>();
        else
            wait_loads<0>();
        if (valid != ~0u) {
            clear_rows<S::C, kFewTile, 1>(vt, valid, 0, lane);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        if (later && any_odd<T>(vt, kFewTile * S::C, lane)) odd = true;
        add_values<T, later>(s, vt, values, o);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (more) load(PLACES == 2 ? vc : kc, vt);
        valid = next_valid;
    };
    // tiles that all rows see whole first: those that end at the first row's last token or before
    const int whole = lim_min >= end ? tiles : (lim_min > beg ? (lim_min - beg) / kFewTile : 0);
    const int plain = whole > wave ? (whole - wave + NW - 1) / NW : 0;
    int k = 0;
    for (; k < plain && k < count; ++k) step(k, std::false_type{});
    for (; k < count; ++k) step(k, std::true_type{});
    // Of this wave's tiles alone: for a row that sees nothing of them its part counts nothing, and
    // an infinity of another wave's tile times that would be no number.
    if (odd)
        for (k = plain; k < count; ++k) {
            const int base = base_of(k);
            add_others<T>(a.pages, table, vc, base, base + kFewTile < end ? base + kFewTile : end, 0, lim,
                          lane, o);
        }

    // the waves' parts are joined through LDS, in wave order
    l = half_sum(l);
    __syncthreads();
    float *join = reinterpret_cast<float *>(smem);
    float2 *stat = reinterpret_cast<float2 *>(smem + (S::RING > S::JOIN ? S::RING : S::JOIN));
    if ((lane & 31) < rows) {
        float *dst = join + (wave * 32 + (lane & 31)) * S::LD + 4 * half;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                store4(dst + 32 * d + 8 * e, o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2],
                       o[d][4 * e + 3]);
        if (half == 0) stat[wave * 32 + lane] = float2{m * sl, l};
    }
    __syncthreads();
    uint32_t nothing = 0;  // rows that see nothing
    if (!a.part) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) sum += stat[w * 32 + row].y;
        if (__ballot(sum == 0.f)) {
            const int first = first_there(a.pages, table, len, lane);
            nothing = (uint32_t)__ballot(sum == 0.f && first >= lim);
        }
    }
    for (int i = threadIdx.x; i < rows * (D / 4); i += 64 * NW) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        float top = -__builtin_inff(), sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = __builtin_fmaxf(top, stat[w * 32 + r].x);
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float2 v = stat[w * 32 + r];
            const float f = part_weight(v, top);
            sum += v.y * f;
            y += *reinterpret_cast<const f32x4 *>(join + (w * 32 + r) * S::LD + c) * f;
        }
        const int64_t token = tok0 + r / G, h = (int64_t)hk * G + r % G;
        const int64_t at = token * a.heads + h;
        if (a.part) {
            const int64_t slot = (pre ? 0 : a.plan.prefix_splits) + split;
            const int64_t to = slot * a.seqs.tokens * a.heads + at;
            *reinterpret_cast<f32x4 *>(a.part + to * D + c) = y;
            if (c == 0) a.stat[to] = float2{top, sum};
        } else {
            const bool any = !((nothing >> r) & 1);
            const float inv = any ? 1.f / sum : 0.f;
            T *out = static_cast<T *>(a.out) + token * a.out_stride + h * D + c;
            store4(out, y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
            if (a.lse && c == 0)
                a.lse[at] = any ? (usable(top) + __builtin_log2f(sum)) * kLn2 : -__builtin_inff();
        }
    }
}

}  // namespace kda
