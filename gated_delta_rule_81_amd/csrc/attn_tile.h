// attn_tile.h -- attention of many query rows over a shared prefix, over a
// session's own tokens, or over both: matrix products fed from LDS.
#pragma once

#include "attn_device.h"

namespace kda {

template <typename T, int D, int DV, bool LATENT, int SPLIT, int NW, int TK> struct TileShape {
    static constexpr int E = sizeof(T), C = D * E / 16, CV = DV * E / 16;
    static constexpr int BM = 32 * NW / SPLIT;          // rows of a workgroup
    static constexpr int KB = TK * C * 16, VB = LATENT ? 0 : TK * CV * 16, BUF = KB + VB;
    static constexpr int LDS = 2 * BUF + (SPLIT == 2 ? 4096 * NW : 0);
    static constexpr int CHV = LATENT ? C : CV;         // chunks of a row that holds values
    static_assert(TK * C % 64 == 0 && TK * CV % 64 == 0, "whole loads");
};

// Ranges (kv heads x splits) and row tiles of the prefix and of the sessions' own tokens (or
// both), and the blocks of each, a multiple of the 8 XCDs.
struct TileGrid {
    int prefix_ranges, prefix_tiles, prefix_blocks;
    int own_ranges, own_tiles, own_blocks;
};

template <typename T, int D, int DV, bool LATENT, int SPLIT, int NW, int TK>
__device__ __forceinline__ void tile_walk(const AttnArgs &a, const TileGrid &g, int block, char *smem) {
    typedef TileShape<T, D, DV, LATENT, SPLIT, NW, TK> S;
    // A wave's share: 32 rows, KS chunk pairs of their channels, DT * 32 of their values.
    constexpr int TT = TK / 32, DT = DV / 32 / SPLIT, KS = S::C / 2 / SPLIT;
    constexpr uint64_t kAll = ~0ull >> (64 - TK);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, group = wave / SPLIT, part = wave % SPLIT;

    // Blocks in the order of their ranges (kv head, split), an eighth of them on each XCD:
    // those that read the same tokens share an L2.
    const bool pre = block < g.prefix_blocks;
    const int b = pre ? block : block - g.prefix_blocks;
    const int tiles = pre ? g.prefix_tiles : g.own_tiles;
    const int unit = b % 8 * (pre ? g.prefix_blocks / 8 : g.own_blocks / 8) + b / 8;
    const int range = unit / tiles;
    int tile = unit % tiles;
    if (range >= (pre ? g.prefix_ranges : g.own_ranges)) return;
    const bool joint = a.plan.joint;
    const int splits = pre || joint ? a.plan.prefix_splits : a.plan.own_splits;
    const int hk = range / splits, split = range % splits, G = a.group;

    // rows [row0, row0 + rows) of the tokens from tok0 on, G rows a token
    const int P = pre || joint ? prefix_tokens(a) : 0;
    int tok0 = 0, n = a.seqs.tokens, L = 0, session = 0;
    if (!pre) {
        const int64_t bm = S::BM;
        session = session_search(a.seqs, tile, lane,
                                 [&](int first, int s) { return (int64_t)first * G / bm + s; });
        tok0 = session_first(a.seqs, session);
        n = session_first(a.seqs, session + 1) - tok0;
        tile -= (int)((int64_t)tok0 * G / bm) + session;
        L = own_tokens(a.seqs, a.pages, session);
        if (tile < 0 || (int64_t)n * G <= a.plan.few_rows) return;
    }
    const int64_t rows = (int64_t)n * G - (int64_t)tile * S::BM;
    if (rows <= 0) return;
    const int64_t row0 = (int64_t)tile * S::BM;
    const int last = (int)(rows < S::BM ? rows : S::BM) - 1;

    // the tokens of this split: of the prefix, then of the session's own
    const int pu = units_of(P), units = pu + units_of(L), per = split_units(units, splits);
    const int u0 = split * per, u1 = u0 + per < units ? u0 + per : units;
    if (u0 >= units && (split > 0 || a.part)) return;
    auto seen = [&](int64_t row) { return L - n + (int)((row0 + row) / G) + 1; };  // own tokens
    int base0 = 0, end0 = 0, base1 = 0, end1 = 0;
    if (u0 < pu) {
        base0 = u0 * kSplitTokens;
        end0 = u1 < pu ? u1 * kSplitTokens : P;
    }
    if (u1 > pu) {
        const int64_t to = (int64_t)(u1 - pu) * kSplitTokens;
        base1 = u0 > pu ? (u0 - pu) * kSplitTokens : 0;
        end1 = to < L ? (int)to : L;
        const int most = seen(last);
        end1 = end1 < most ? end1 : most;
        end1 = end1 > base1 ? end1 : base1;
    }
    if (a.pages.count == 0) end0 = base0, end1 = base1;  // no page to read in place of one
    const int n0 = (end0 - base0 + TK - 1) / TK, nt = n0 + (end1 - base1 + TK - 1) / TK;
    const int32_t *own_table = pre ? nullptr : a.seqs.table + (int64_t)session * a.seqs.width;

    // this wave's queries; rows behind the last one are computed as the last one's
    u32x4 q[KS];
    const bool active = 32 * group <= last;
    int lim = 0, wave_max = 0;  // own tokens that a row sees, and the wave's last
    {
        int r = 32 * group + (lane & 31);
        r = r < last ? r : last;
        const int64_t row = row0 + r;
        const T *src = static_cast<const T *>(a.q) + (tok0 + row / G) * a.q_stride +
                       ((int64_t)hk * G + row % G) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[s] = *reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(src) +
                                                    16 * (2 * (part * KS + s) + half));
        if (!pre) {
            lim = seen(r);
            wave_max = seen(32 * group + 31 < last ? 32 * group + 31 : last);
        }
    }

    const int64_t head = (int64_t)hk * a.pages.head;
    const char *kc = static_cast<const char *>(a.k_cache) + head;
    const char *vc = LATENT ? nullptr : static_cast<const char *>(a.v_cache) + head;
    lds_char *lds = (lds_char *)smem;
    auto base_of = [&](int t) { return t < n0 ? base0 + t * TK : base1 + (t - n0) * TK; };
    // This lane's token of tile t: the entry of its page, -1 where there is none.
    auto entry_of = [&](int t) {
        const int tok = base_of(t) + lane;
        if (t >= nt || lane >= TK || tok >= (t < n0 ? end0 : end1)) return -1;
        return (t < n0 ? a.prefix_pages : own_table)[a.pages.by_size(tok)];
    };
    auto issue = [&](int t, int entry) -> uint64_t {
        bool there;
        const uint32_t place = token_place(a.pages, entry, base_of(t) + lane, &there);
        load_tile<S::C, TK, NW, !LATENT>(kc, vc, place, a.pages.shift, lds + (t & 1) * S::BUF, wave, lane);
        return __ballot(there);
    };

    f32x16 o[DT];
    float m = -__builtin_inff(), l = 0.f;  // running maximum of q k; this lane's half of the sum
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16(0.f);
    const float sl = a.scale * kLog2e;  // scores in units of log 2

    const Keys<S::C> keys(part * KS, lane);
    const typename AttnMma<T>::template Values<S::CHV> values(part * DT, lane);

    bool odd = false;  // a value that is no number in a tile that not all rows see whole
    uint64_t valid = 0, next_valid = 0;
    int entry = -1;
    if (nt > 0) {
        valid = issue(0, entry_of(0));
        entry = entry_of(1);
    }
    // One tile; LATER: some row may not see some token of it.
    auto step = [&](int t, auto LATER) {
        constexpr bool later_tiles = decltype(LATER)::value;
        lds_char *kt = lds + (t & 1) * S::BUF, *vt = LATENT ? kt : kt + S::KB;
        wait_loads<0>();
        if (valid != kAll) clear_rows<S::CHV, TK, NW>(vt, valid, wave, lane);
        __syncthreads();
        if (t + 1 < nt) {
            next_valid = issue(t + 1, entry);
            entry = entry_of(t + 2);
        }
        const int base = base_of(t);
        const bool look = active && !(later_tiles && base >= wave_max);
        f32x16 s[TT];
        if (SPLIT == 2 || look) scores<T, S::C, TT, KS>(kt, keys, q, s);
        if constexpr (SPLIT == 2) {  // the sum over the other half of the channels
            lds_char *mine = lds + 2 * S::BUF + wave * 4096 + lane * 16;
            lds_char *other = lds + 2 * S::BUF + (wave ^ 1) * 4096 + lane * 16;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *(lds_f32x4 *)(mine + 1024 * e) =
                    f32x4{s[0][4 * e], s[0][4 * e + 1], s[0][4 * e + 2], s[0][4 * e + 3]};
            lds_barrier();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4 w = *(lds_f32x4 *)(other + 1024 * e);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[0][4 * e + i] += w[i];
            }
        }
        if (look) {
            if (later_tiles || valid != kAll)
                hide_scores<TT>(s, valid, later_tiles ? lim - base : TK, lane);
            soften<TT, DT>(s, m, l, o, sl);
            if (later_tiles && any_odd<T>(vt, TK * S::CHV, lane)) odd = true;
            add_values<T, later_tiles>(s, vt, values, o);
        }
        valid = next_valid;
    };
    wait_loads<0>();  // the queries among them
    // tiles that all rows see whole first: of the prefix, and of own tokens up to the first row's
    int t = 0, plain = nt;
    if (!pre && end1 > base1) {
        const int whole = seen(0) > base1 ? (seen(0) - base1) / TK : 0;
        plain = n0 + whole < nt ? n0 + whole : nt;
    }
    for (; t < plain; ++t) step(t, std::false_type{});
    for (; t < nt; ++t) step(t, std::true_type{});
    if (odd) add_others<T>(a.pages, own_table, LATENT ? kc : vc, base_of(plain), end1, part * DT, lim, lane, o);

    if (!active) return;
    const int r = 32 * group + (lane & 31);
    if (r > last) return;
    l = half_sum(l);
    const int64_t row = row0 + r, token = tok0 + row / G, h = (int64_t)hk * G + row % G;
    const int64_t at = token * a.heads + h;
    const int c0 = 32 * part * DT + 4 * half;  // first channel of this lane
    const bool first = half == 0 && part == 0;
    if (a.part) {
        const int64_t slot = (pre || joint ? 0 : a.plan.prefix_splits) + split;
        const int64_t place = slot * a.seqs.tokens * a.heads + at;
        if (first) a.stat[place] = float2{m * sl, l};
        float *dst = a.part + place * DV + c0;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                store4(dst + 32 * d + 8 * e, o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2],
                       o[d][4 * e + 3]);
    } else {
        const bool any = P > 0 || lim > 0;
        const float inv = any ? 1.f / l : 0.f;
        T *dst = static_cast<T *>(a.out) + token * a.out_stride + h * DV + c0;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                store4(dst + 32 * d + 8 * e, o[d][4 * e] * inv, o[d][4 * e + 1] * inv,
                       o[d][4 * e + 2] * inv, o[d][4 * e + 3] * inv);
        if (a.lse && first)
            a.lse[at] = any ? (usable(m) * sl + __builtin_log2f(l)) * kLn2 : -__builtin_inff();
    }
}

}  // namespace kda
