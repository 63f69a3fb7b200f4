// attn_few.hip -- attention of few query rows (at most 32: one token's heads of a group, or a
// few tokens') over a long cache, and the join of the parts of every row.
#include "attn_device.h"

namespace kda {
namespace {

constexpr int kTile = 32;  // tokens of a wave's tile

// What a part (its maximum in units of log 2, its sum) counts beside others: nothing where its
// maximum is -inf, unless its scores were no numbers, which its sum then is not either.
__device__ __forceinline__ float part_weight(const float2 &part, float top) {
    return part.x > -__builtin_inff() ? fast_exp2(part.x - top) : (part.y == 0.f ? 0.f : part.y);
}

template <typename T, int D, int NW, int ST> struct FewShape {
    static constexpr int C = D * (int)sizeof(T) / 16;   // 16-byte chunks of a row
    static constexpr int HALF = kTile * C * 16, BUF = 2 * HALF;
    static constexpr int LOADS = 2 * kTile * C / 64;    // of a tile, keys and values
    static constexpr int LD = D + 4;                    // floats between rows of the joined output
    static constexpr int RING = NW * ST * BUF, JOIN = NW * 32 * LD * 4;
    static constexpr int LDS = (RING > JOIN ? RING : JOIN) + NW * 32 * 8;
    static_assert((ST - 1) * LOADS < 64, "the counter of loads on their way");
};

// One workgroup per (session, kv head, split), or per (kv head, split) of the prefix.
template <typename T, int D, int NW, int ST>
__global__ __launch_bounds__(64 * NW) void attn_few_kernel(AttnArgs a, int own_blocks) {
    typedef FewShape<T, D, NW, ST> S;
    constexpr int DT = D / 32, KS = S::C / 2;
    __shared__ __attribute__((aligned(1024))) char smem[S::LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, G = a.group;
    const bool pre = (int)blockIdx.x >= own_blocks;
    const int b = pre ? blockIdx.x - own_blocks : blockIdx.x;
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
    lds_char *ring = (lds_char *)smem + wave * (ST * S::BUF);

    // This wave's tiles are its own: every NW-th, in a ring of ST places that no other wave
    // reads, so that only its own loads are waited for.  A window of 64 entries of the page
    // table is held in the lanes.
    const int tiles = a.pages.count > 0 ? (end - beg + kTile - 1) / kTile : 0;
    const int count = tiles > wave ? (tiles - wave + NW - 1) / NW : 0;
    int first = 0, entries = -1;
    bool held = false;
    auto base_of = [&](int k) { return beg + (k * NW + wave) * kTile; };
    auto issue = [&](int k, int place) -> uint32_t {
        const int base = base_of(k), tok = base + lane;
        const int stop = base + kTile < end ? base + kTile : end;
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
        const uint32_t at = token_place(a.pages, entry, tok, &there);
        load_tile<S::C, kTile, 1, true>(kc, vc, at, a.pages.shift, ring + place * S::BUF, 0, lane);
        return (uint32_t)__ballot(there);
    };

    f32x16 o[DT];
    float m = -__builtin_inff(), l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16(0.f);
    const float sl = a.scale * kLog2e;
    const Keys<S::C> keys(0, lane);
    const typename AttnMma<T>::template Values<S::C> values(0, lane);
    uint32_t valid[ST];
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) valid[i] = i < count ? issue(i, i) : 0;
    int place = 0, ahead = ST - 1;
    bool odd = false;  // a value that is no number in a tile that not all rows see whole
    // One tile; LATER: some row may not see some token of it.
    auto step = [&](int k, auto LATER) {
        constexpr bool later = decltype(LATER)::value;
        if (k + ST - 1 < count) {
            valid[ST - 1] = issue(k + ST - 1, ahead);
            wait_loads<(ST - 1) * S::LOADS>();
        } else {
            wait_loads<0>();
        }
        const int base = base_of(k);
        lds_char *kt = ring + place * S::BUF, *vt = kt + S::HALF;
        if (valid[0] != ~0u) {
            clear_rows<S::C, kTile, 1>(vt, valid[0], 0, lane);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        f32x16 s[1];
        scores<T, S::C, 1, KS>(kt, keys, q, s);
        if (later || valid[0] != ~0u) hide_scores<1>(s, valid[0], later ? lim - base : kTile, lane);
        soften<1, DT>(s, m, l, o, sl);
        if (later && any_odd<T>(vt, kTile * S::C, lane)) odd = true;
        add_values<T, later>(s, vt, values, o);
        // the tile is read before its place is filled again
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) valid[i] = valid[i + 1];
        place = place + 1 == ST ? 0 : place + 1;
        ahead = ahead + 1 == ST ? 0 : ahead + 1;
    };
    // tiles that all rows see whole first: those that end at the first row's last token or before
    const int whole = lim_min >= end ? tiles : (lim_min > beg ? (lim_min - beg) / kTile : 0);
    const int plain = whole > wave ? (whole - wave + NW - 1) / NW : 0;
    int k = 0;
    for (; k < plain; ++k) step(k, std::false_type{});
    for (; k < count; ++k) step(k, std::true_type{});
    if (odd) add_others<T>(a.pages, table, vc, beg + whole * kTile, end, 0, lim, lane, o);

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
            const bool any = seen(r) > 0;
            const float inv = any ? 1.f / sum : 0.f;
            T *out = static_cast<T *>(a.out) + token * a.out_stride + h * D + c;
            store4(out, y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
            if (a.lse && c == 0)
                a.lse[at] = any ? (usable(top) + __builtin_log2f(sum)) * kLn2 : -__builtin_inff();
        }
    }
}

int64_t few_blocks(const AttnArgs &a, int64_t *own) {
    const AttnPlan &p = a.plan;
    *own = p.few_rows > 0 && !p.joint ? (int64_t)a.seqs.num * a.kv_heads * p.own_splits : 0;
    return *own + (p.prefix_few ? (int64_t)a.kv_heads * p.prefix_splits : 0);
}

template <typename T, int D, int NW, int ST> int few(const AttnArgs &a, hipStream_t stream) {
    int64_t own;
    const int64_t n = few_blocks(a, &own);
    if (n > 0)
        hipLaunchKernelGGL((attn_few_kernel<T, D, NW, ST>), dim3((unsigned)n), dim3(64 * NW),
                           0, stream, a, (int)own);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

// One workgroup per row (token, head): DV / 4 lanes hold a row's values, the 1024 / DV groups
// of them take every so many-th part, and are added up in their order.  Its time is one chain
// of loads (lengths, statistics, parts), so everything that does not depend on another load is
// read at once.
template <typename T, int DV> __global__ __launch_bounds__(256) void attn_merge_kernel(AttnArgs a) {
    constexpr int LANES = DV / 4, GROUPS = 256 / LANES, SLOTS = 128;
    __shared__ float2 stat[SLOTS];
    __shared__ f32x4 sums[GROUPS][LANES];
    const int64_t at = blockIdx.x, rows = (int64_t)a.seqs.tokens * a.heads;
    const int token = (int)(at / a.heads), h = (int)(at % a.heads);
    const int tid = threadIdx.x, lane = tid & 63, group = tid / LANES, c = 4 * (tid % LANES);
    const AttnPlan &p = a.plan;
    // statistics of every slot, whether a part was written or not
    const int slots = p.prefix_splits + p.own_splits;
    float2 mine = {0.f, 0.f};
    if (tid < slots) mine = a.stat[tid * rows + at];
    const int s = a.seqs.cu ? session_search(a.seqs, token, lane, [](int first, int) { return first; })
                            : token / a.seqs.each;
    const int first = session_first(a.seqs, s), last = session_first(a.seqs, s + 1);
    if (token < first || token >= last) return;  // in no session
    const int L = own_tokens(a.seqs, a.pages, s), P = prefix_tokens(a);
    const bool any = P > 0 || L - (last - token) + 1 > 0;

    // which slots hold a part: the first n0 of the prefix's, the first n1 of the own ones
    const int pu = units_of(P), lu = units_of(L);
    const int u0 = p.joint ? pu + lu : pu, per0 = split_units(u0, p.prefix_splits);
    const int n0 = per0 > 0 ? (u0 + per0 - 1) / per0 : 0;
    const int per1 = p.joint ? 0 : split_units(lu, p.own_splits);
    const int n1 = per1 > 0 ? (lu + per1 - 1) / per1 : 0, n = n0 + n1;
    const int slot = tid < p.prefix_splits ? tid : tid - p.prefix_splits + n0;
    if (tid < slots && (tid < p.prefix_splits ? tid < n0 : slot < n)) stat[slot] = mine;
    __syncthreads();
    float top = -__builtin_inff();
    for (int k = 0; k < n; ++k) top = __builtin_fmaxf(top, stat[k].x);
    float sum = 0.f;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < n; ++k) sum += stat[k].y * part_weight(stat[k], top);
#pragma unroll 4
    for (int k = group; k < n; k += GROUPS) {
        const int64_t from = k < n0 ? k : p.prefix_splits + k - n0;
        const f32x4 w = *reinterpret_cast<const f32x4 *>(a.part + (from * rows + at) * DV + c);
        const float f = part_weight(stat[k], top);
        if (f != 0.f) y += w * f;  // a part of which nothing was seen holds anything
    }
    sums[group][tid % LANES] = y;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) y += sums[g][tid];
    const float inv = any ? 1.f / sum : 0.f;
    T *out = static_cast<T *>(a.out) + token * a.out_stride + (int64_t)h * DV + c;
    store4(out, y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    if (a.lse && c == 0)
        a.lse[at] = any ? (usable(top) + __builtin_log2f(sum)) * kLn2 : -__builtin_inff();
}

}  // namespace

int64_t attn_few_threads(const AttnArgs &a) {
    int64_t own;
    return few_blocks(a, &own) * 256;
}
int64_t attn_merge_threads(const AttnArgs &a) {
    return (int64_t)a.seqs.tokens * a.heads * 256;
}

int launch_attn_few(const AttnArgs &a, hipStream_t stream) {
    if (a.dtype == kDtypeF32)
        return a.d == 64 ? few<float, 64, 4, 2>(a, stream) : few<float, 128, 2, 2>(a, stream);
    return a.d == 64 ? few<bf16, 64, 4, 2>(a, stream) : few<bf16, 128, 4, 2>(a, stream);
}

int launch_attn_merge(const AttnArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(attn_merge_threads(a) / 256));
    if (a.dv == 512)
        hipLaunchKernelGGL((attn_merge_kernel<bf16, 512>), grid, dim3(256), 0, stream, a);
    else if (a.dtype == kDtypeF32 && a.dv == 64)
        hipLaunchKernelGGL((attn_merge_kernel<float, 64>), grid, dim3(256), 0, stream, a);
    else if (a.dtype == kDtypeF32)
        hipLaunchKernelGGL((attn_merge_kernel<float, 128>), grid, dim3(256), 0, stream, a);
    else if (a.dv == 64)
        hipLaunchKernelGGL((attn_merge_kernel<bf16, 64>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((attn_merge_kernel<bf16, 128>), grid, dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace kda
