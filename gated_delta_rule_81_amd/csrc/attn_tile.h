// attn_tile.h -- attention of many query rows over a shared prefix, over a
// session's own tokens, or over both: matrix products fed from LDS.
//
// A row is (token, head of the group), so the heads of a group and the tokens of all sessions
// (of one, over its own tokens) share what is read.  A workgroup takes 128 rows, 32 a wave with
// queries, maximum, sum and output in registers, and walks the tokens of its split in tiles of TK
// that all of its waves read; two workgroups a CU.  Keys and values take two places each: while
// tile t is worked on, the keys of t + 2 and the values of t + 1 come.  One barrier a tile.
// What bounds it is issue: for a tile of 64 tokens a wave issues 32 products (32 cycles each)
// beside 32 exponentials of a lane, their scaling, sum and rounding, and the maximum of as many scores.
// The scores of tile t + 1 are formed before the values of tile t are added, so that
// exponentials stand beside products that do not wait for them (turn_over): 675 us to 640 for the
// prompts below.
//
// A latent row (576 channels, the first 512 of them the values) has one place for both.  Its
// queries and outputs are too many for a wave: two waves share 32 rows, each with half of the channels
// of both products (SPLIT 2), whose partial scores meet in LDS behind a second barrier; 6 of 18
// pieces of the queries stay in LDS.  One workgroup of eight waves a CU, whose halves take turns at
// scores and values.
//
// Tiles that some row does not see whole (the own tokens' last ones, and the last of all) go through a
// loop of their own: there a value that is no number is left out of the product, where a
// probability of zero would not hide it, and added behind the walk for the rows that see it.
//
// Measured, bf16: six prompts of up to 1500 tokens x 32 heads (8 of keys) of 128 behind 6000
// shared ones, 0.56 TFLOP: 631 us, 890 TFLOP/s; the matrix unit is busy in 42% of the cycles, the
// vector unit in 45%, at 1.96 GHz.  Four drafts of 64 sessions behind 32K, 0.14 TFLOP: 159 us
// and 13 for the join (870 TFLOP/s).  Latent, 64 sessions x 96 heads behind 8192, 0.12 TFLOP:
// 166 us and 16 (matrix unit 29%: two barriers a tile, and the quarter of the CUs that takes own
// tokens ends early).
#pragma once

#include "attn_device.h"

namespace kda {

template <typename T, int D, int DV, bool LATENT, int SPLIT, int NW, int TK> struct TileShape {
    // Chunks of a row in LDS; of a latent row, its values alone: the channels behind them are a
    // tile of their own, of REST chunks a row.
    static constexpr int E = sizeof(T), C = (LATENT ? DV : D) * E / 16, CV = DV * E / 16;
    static constexpr int REST = LATENT ? (D - DV) * E / 16 : 0;
    static constexpr int BM = 32 * NW / SPLIT;          // rows of a workgroup
    static constexpr int KB = TK * (C + REST) * 16, VB = LATENT ? 0 : TK * CV * 16;
    // tiles of keys t + 1 and values t are read while keys t + 2 and values t + 1 come
    static constexpr int SUMS = 2 * (KB + VB);
    // SPLIT 2: scores on their way to the other half, and what of the queries has no registers
    static constexpr int PARKED = SPLIT == 2 ? 6 : 0, PARK = SUMS + (SPLIT == 2 ? 4096 * NW : 0);
    static constexpr int LDS = PARK + PARKED * 1024 * NW;
    static constexpr int CHV = LATENT ? C : CV;         // chunks of a row that holds values
    static_assert(TK * C % 64 == 0 && TK * CV % 64 == 0, "whole loads");
};

// Ranges (kv heads x splits) and row tiles of the prefix and of the sessions' own tokens (or
// both), and the blocks of each, a multiple of the 8 XCDs.
struct TileGrid {
    int prefix_ranges, prefix_tiles, prefix_blocks;
    int own_ranges, own_tiles, own_blocks;
};

template <typename T, int D, int DV, bool LATENT, int SPLIT, int NW, int TK, bool NEAR>
__device__ __forceinline__ void tile_walk(const AttnArgs &a, const TileGrid &g, int block, char *smem) {
    typedef TileShape<T, D, DV, LATENT, SPLIT, NW, TK> S;
    // A wave's share: 32 rows, KS chunk pairs of their channels, DT * 32 of their values.
    constexpr int TT = TK / 32, DT = DV / 32 / SPLIT, KS = D * S::E / 32 / SPLIT;
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
    constexpr int KR = KS - S::PARKED;  // chunk pairs in registers; the others in LDS
    u32x4 q[KR];
    lds_char *park = (lds_char *)smem + S::PARK + wave * (S::PARKED * 1024) + lane * 16;
    auto query = [&](int c) -> u32x4 {
        return c < KR ? q[c < KR ? c : 0] : *(lds_u32x4 *)(park + 1024 * (c - KR));
    };
    const bool active = 32 * group <= last;
    int lim = 0, wave_max = 0;  // own tokens that a row sees, and the wave's last
    {
        int r = 32 * group + (lane & 31);
        r = r < last ? r : last;
        const int64_t row = row0 + r;
        const T *src = static_cast<const T *>(a.q) + (tok0 + row / G) * a.q_stride +
                       ((int64_t)hk * G + row % G) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            // with SPLIT 2 a half of the values' channels and a half of those behind them
            constexpr int KV = KS - S::REST / 2 / SPLIT;
            const int pair = s < KV ? part * KV + s : S::C / 2 + part * (KS - KV) + s - KV;
            const u32x4 x = *reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(src) +
                                                             16 * (2 * pair + half));
            if (s < KR)
                q[s < KR ? s : 0] = x;
            else
                *(lds_u32x4 *)(park + 1024 * (s - KR)) = x;
        }
        if (!pre) {
            lim = seen(r);
            wave_max = seen(32 * group + 31 < last ? 32 * group + 31 : last);
        }
    }

    const int64_t head = (int64_t)hk * a.pages.head;
    const char *kc = static_cast<const char *>(a.k_cache) + head;
    const char *vc = LATENT ? nullptr : static_cast<const char *>(a.v_cache) + head;
    lds_char *lds = (lds_char *)smem;
    auto keys_of = [&](int t) { return lds + (t & 1) * S::KB; };
    auto values_of = [&](int t) { return LATENT ? keys_of(t) : lds + 2 * S::KB + (t & 1) * S::VB; };
    auto base_of = [&](int t) { return t < n0 ? base0 + t * TK : base1 + (t - n0) * TK; };

    // The tile that is placed next and the entry of its page for this lane's token (one of the
    // table's whether the token is there or not) and the token's number in the page; the same of
    // the tile behind it, whose entry is on its way.  No branches: this stands in the stream of
    // products.
    int ahead = 0, in = 0, entry = 0, in2 = 0, entry2 = 0;
    const int last0 = end0 > base0 ? a.pages.by_size(end0 - 1) : 0;
    const int last1 = end1 > base1 ? a.pages.by_size(end1 - 1) : 0;
    auto owned = [&](int t) { return n0 < nt && t >= n0; };
    auto look_up = [&](int t) {
        const int tok = base_of(t) + lane, idx = a.pages.by_size(tok);
        const int last = owned(t) ? last1 : last0;
        in = in2, entry = entry2;
        in2 = tok - idx * a.pages.size;
        entry2 = (owned(t) ? own_table : a.prefix_pages)[idx < last ? idx : last];
    };
    // That tile's place of this lane's token (0 where there is none: the first page's first, which
    // is there), and which of its tokens there are.
    auto place_token = [&](uint64_t *valid) -> uint32_t {
        const int end = ahead >= nt ? 0 : (owned(ahead) ? end1 : end0);
        const bool there = (lane < TK) & (base_of(ahead) + lane < end) &
                           ((unsigned)entry < (unsigned)a.pages.count);
        const uint32_t place = (uint32_t)entry * a.pages.page_units + (uint32_t)in * a.pages.token_units;
        *valid = __ballot(there);
        ++ahead;
        return there ? place : 0;
    };
    auto place_tile = [&](TileLoads<S::C, TK, NW, NEAR> &loads, uint64_t *valid) {
        loads.set(a.pages, place_token(valid), wave, lane);
    };
    auto load_keys = [&](int t, const TileLoads<S::C, TK, NW, NEAR> &loads) {
        if (t < nt) loads.load(a.pages, kc, keys_of(t), wave, lane);
    };
    auto load_values = [&](int t, const TileLoads<S::C, TK, NW, NEAR> &loads) {
        if (!LATENT && t < nt) loads.load(a.pages, vc, values_of(t), wave, lane);
    };

    f32x16 o[DT], s[TT];
    float m = -__builtin_inff(), l = 0.f;  // running maximum of q k; this lane's half of the sum
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16(0.f);
    const float sl = a.scale * kLog2e;  // scores in units of log 2
    bool odd = false;  // a value that is no number in a tile that not all rows see whole

    // SPLIT 2: the sums over the two halves of the channels meet in LDS.
    lds_char *mine = lds + S::SUMS + wave * 4096 + lane * 16;
    lds_char *other = lds + S::SUMS + (wave ^ 1) * 4096 + lane * 16;
    auto give = [&](const f32x16 &x) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *(lds_f32x4 *)(mine + 1024 * e) = f32x4{x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]};
    };
    auto take = [&](f32x16 &x) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f32x4 w = *(lds_f32x4 *)(other + 1024 * e);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * e + i] += w[i];
        }
    };

    // tiles under `plain` are seen whole by all rows: of the prefix, and own ones up to the first row's
    int plain = nt;
    if (!pre && end1 > base1) {
        const int whole = seen(0) > base1 ? (seen(0) - base1) / TK : 0;
        plain = n0 + whole < nt ? n0 + whole : nt;
    }
    // valid: which tokens of tile t there are; valid1, valid2: of the two behind it.
    uint64_t valid = 0, valid1 = 0, valid2 = 0;
    int t = 0, from = 0;  // from: the first tile of the loop that leaves out what is no number
    if (nt == 0) {
        wait_loads<0>();
    } else if constexpr (SPLIT == 1) {
        const Keys<S::C> keys(0, lane);
        const typename AttnMma<T>::template Values<S::CHV> values(0, lane);
        TileLoads<S::C, TK, NW, NEAR> loads, loads2;  // of tiles t + 1 and t + 2
        look_up(0), look_up(1);
        place_tile(loads, &valid);
        load_keys(0, loads);
        load_values(0, loads);
        look_up(2);
        place_tile(loads, &valid1);
        load_keys(1, loads);
        look_up(3);
        place_tile(loads2, &valid2);
        wait_loads<0>();  // the queries among them
        __syncthreads();
        if (nt > 0 && active) scores<T, KS>(keys_of(0), keys, query, s);
        // Tile t, whose scores are in x: probabilities and values, and beside them the scores of
        // tile t + 1, to y.  LATER: some row may not see some token of it, or it is the last.
        auto step = [&](f32x16 (&x)[TT], f32x16 (&y)[TT], auto LATER) {
            constexpr bool later = decltype(LATER)::value;
            lds_char *vt = values_of(t), *kt = keys_of(t + 1);
            wait_loads<0>();
            if (valid != kAll) clear_rows<S::CHV, TK, NW>(vt, valid, wave, lane);
            __syncthreads();
            load_values(t + 1, loads);
            load_keys(t + 2, loads2);
            look_up(t + 4);
            const int base = base_of(t);
            const bool own = t >= n0, look = active && !(later && own && base >= wave_max);
            if (look && (later || valid != kAll))
                hide_scores<TT>(x, valid, later && own ? lim - base : TK, lane);
            if (later && look && any_odd<T>(vt, TK * S::CHV, lane)) odd = true;
            valid = valid1, valid1 = valid2;
            auto place_next = [&]() {
                loads = loads2;
                place_tile(loads2, &valid2);
            };
            if constexpr (!later) {
                if (active) {
                    move_maximum<TT, DT>(x, m, l, o, sl);
                    turn_over<T>(kt, vt, keys, values, q, x, y, m, l, o, sl, [&](int i) {
                        if (i == 2) place_next();
                    });
                } else {
                    place_next();
                }
            } else {
                place_next();
                if (active && t + 1 < nt) scores<T, KS>(kt, keys, query, y);
                if (look) {
                    move_maximum<TT, DT>(x, m, l, o, sl);
                    soften<TT>(x, m, l, sl);
                    add_values<T, true>(x, vt, values, o);
                }
            }
            ++t;
        };
        f32x16 s2[TT];
        while (t + 1 < plain && t + 2 < nt) {
            step(s, s2, std::false_type{});
            step(s2, s, std::false_type{});
        }
        from = t;
        while (t < nt) {
            step(s, s2, std::true_type{});
#pragma unroll
            for (int j = 0; j < TT; ++j) s[j] = s2[j];
        }
    } else {
        // Few registers are left beside a wave's share of the queries and the outputs: a tile is
        // placed when it is loaded, its scores are formed when it is there, and where its operands
        // lie is formed again for each.  The 64 chunks of a row's values are one load, whose row
        // is the wave's; the channels behind them are four loads of eight rows each.
        static_assert(LATENT && S::C == 64 && S::REST == 8 && TK == 32 && NW == 8, "a latent row");
        auto issue = [&](int t, uint64_t *valid) {
            const uint32_t place = place_token(valid);
            if (t >= nt) return;
            lds_char *tile = keys_of(t);
            const int ln = here(lane);
#pragma unroll
            for (int i = 0; i < TK / NW; ++i) {
                const int row = NW * i + wave;
                const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)place, row)
                                    << a.pages.shift;
                load_lds16(kc + at, (uint32_t)((ln ^ tile_turn<S::C>(row)) * 16),
                           (uint32_t)(uintptr_t)tile + 1024 * row);
            }
            if (wave < 4) {
                const int row = 8 * wave + (ln >> 3);
                const uint64_t at =
                    (uint64_t)(uint32_t)__builtin_amdgcn_ds_bpermute(4 * row, (int)place) << a.pages.shift;
                load_lds16(kc + at + 1024 + ((ln & 7) ^ tile_turn<8>(row)) * 16,
                           (uint32_t)(uintptr_t)tile + TK * S::C * 16 + 1024 * wave);
            }
        };
        auto both_scores = [&](lds_char *tile) {
            constexpr int KV = KS - 2;
            const Keys<S::C> keys(part * KV, here(lane));
            const Keys<8> rest(part * 2, here(lane));
            scores_ahead<T, KS>(
                [&](int c) {
                    return c < KV ? keys.read(tile, 0, c) : rest.read(tile + TK * S::C * 16, 0, c - KV);
                },
                query, s[0]);
        };
        const bool second = wave >= NW / 2;
        look_up(0), look_up(1);
        issue(0, &valid);
        // Tile u is there and what is no token of it cleared; its place before is read to the end.
        auto arrive = [&](int u, uint64_t there) {
            wait_loads<0>();
            if (u < nt && there != kAll) clear_rows<S::CHV, TK, NW>(keys_of(u), there, wave, lane);
            lds_barrier();
        };
        auto follow = [&](int u) {  // the tile behind u, in the place of the one before it
            lds_barrier();
            look_up(u + 2);
            issue(u + 1, &valid1);
        };
        // Between two barriers one half of the waves forms scores and the other adds values, so
        // that every SIMD has a wave of each: the first half is at tile t's values when the
        // second is at its scores.  Scores, which are products alone, go first: what stands beside
        // the products of the values fills their gaps (latent, 64 sessions x 96 heads behind 8192,
        // on one card: 212 us to 201; either without the other 208 to 215).
        auto step = [&](auto LATER) {
            constexpr bool later = decltype(LATER)::value;
            lds_char *kt = keys_of(t);
            const int base = base_of(t);
            const bool own = t >= n0, look = active && !(later && own && base >= wave_max);
            if (active) {
                __builtin_amdgcn_s_setprio(1);
                both_scores(kt);
                __builtin_amdgcn_s_setprio(0);
                give(s[0]);
            }
            const uint64_t there = valid;
            if (second)
                arrive(t + 1, valid1);
            else
                follow(t);
            valid = valid1;
            if (look) {
                take(s[0]);
                if (later || there != kAll)
                    hide_scores<TT>(s, there, later && own ? lim - base : TK, lane);
                if (later && any_odd<T>(kt, TK * S::CHV, lane)) odd = true;
                move_maximum<TT, DT>(s, m, l, o, sl);
                const typename AttnMma<T>::template Values<S::CHV> values(part * DT, here(lane));
                if constexpr (later) {
                    soften<TT>(s, m, l, sl);
                    add_values<T, true>(s, kt, values, o);
                } else {
                    values_ahead<T>(kt, values, s[0], m, l, o, sl);
                }
            }
            if (!second)
                arrive(t + 1, valid1);
            else if (t + 1 < nt)
                follow(t + 1);
            ++t;
        };
        arrive(0, valid);  // the queries have come, too
        if (second) follow(0);
        while (t < plain) step(std::false_type{});
        from = t;
        while (t < nt) step(std::true_type{});
    }
    if (odd) {  // in the tiles from `from` on: the prefix's last ones, which all rows see, own ones
        const char *values = LATENT ? kc : vc;
        if (from < n0)
            add_others<T>(a.pages, a.prefix_pages, values, base_of(from), end0, part * DT, end0, lane, o);
        if (n0 < nt)
            add_others<T>(a.pages, own_table, values, base_of(from > n0 ? from : n0), end1, part * DT,
                          lim, lane, o);
    }

    if (!active) return;
    l = half_sum(l);
    bool any = true;  // whether this lane's row sees a token
    if (!a.part && __ballot(l == 0.f)) {
        const bool shared = first_there(a.pages, a.prefix_pages, P, lane) < P;
        const int first = first_there(a.pages, own_table, L, lane);
        any = l != 0.f || shared || first < lim;
    }
    const int r = 32 * group + (lane & 31);
    if (r > last) return;
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
