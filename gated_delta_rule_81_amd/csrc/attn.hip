// attn.hip -- the launches of the attention over a shared prefix and each session's
// own tokens, and the join of what its splits leave.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(scale log2(e) q k_j - m)
//
// A part holds its maximum m, its sum and its unscaled output; parts are joined by 2^(m - max m).
// Measured with one token of 256 sessions, 32 heads (8 of keys) of 128, behind 16K shared tokens and up to
// 2000 own ones (1.1 GB and 0.07 TFLOP): 272 us and 15 for the join; in two launches,
// prefix then own tokens, 386 in all.
#include "attn_few.h"
#include "attn_tile.h"

namespace kda {
namespace {

// Tile blocks of a turn (see attn_kernel): as many as there are CUs.
constexpr int kTurn = 256;

// What a launch is made of: `few` blocks for few rows (own_few of them own tokens, the others
// prefix), and those of the tile grid.
struct MixGrid {
    int few, own_few;
    TileGrid tile;
};

// Per-head caches: both walks in one launch, so that the one bound by memory and the one bound
// by the matrix units share each CU.
template <typename T, int D, int TK, int PLACES> struct MixShape {
    static constexpr int A = TileShape<T, D, D, false, 1, 4, TK>::LDS;
    static constexpr int B = FewShape<T, D, 4, PLACES>::LDS;
    static constexpr int LDS = A > B ? A : B;
};
template <typename T, int D, int TK, int PLACES, bool NEAR>
__global__ __launch_bounds__(256, 2) void attn_kernel(AttnArgs a, MixGrid g) {
    __shared__ __attribute__((aligned(1024))) char smem[MixShape<T, D, TK, PLACES>::LDS];
    // Turns of kTurn tile blocks, one for each CU, with an equal share of the others behind each:
    // those are short, and take up the second place of every CU while the tiles last.  (256
    // tokens behind 16K: 300 us; all tiles first, two of them on every CU, 312.)
    const int tiles = g.tile.prefix_blocks + g.tile.own_blocks, turns = tiles / kTurn;
    const int share = turns > 0 ? g.few / turns / 8 * 8 : 0, turn = kTurn + share;
    int b = blockIdx.x;
    bool few;
    if (b < turns * turn) {
        const int r = b % turn;
        few = r >= kTurn;
        b = b / turn * (few ? share : kTurn) + (few ? r - kTurn : r);
    } else {  // what is left of the tiles, then of the others
        b -= turns * turn;
        const int left = tiles - turns * kTurn;
        few = b >= left;
        b += few ? turns * share - left : turns * kTurn;
    }
    if (few)
        few_walk<T, D, 4, PLACES, NEAR>(a, g.own_few, b, smem);
    else
        tile_walk<T, D, D, false, 1, 4, TK, NEAR>(a, g.tile, b, smem);
}

__global__ __launch_bounds__(512, 2) void attn_latent_kernel(AttnArgs a, TileGrid g) {
    typedef TileShape<bf16, 576, 512, true, 2, 8, 32> S;
    __shared__ __attribute__((aligned(1024))) char smem[S::LDS];
    tile_walk<bf16, 576, 512, true, 2, 8, 32, true>(a, g, blockIdx.x, smem);
}

// Row (token, head): the parts of its splits.  W waves a row; DV / 4 lanes hold its values, the
// groups of them take every so many-th part and are added up in their order.  Its time is one
// chain of loads (lengths, statistics, parts), so what does not depend on another load is read at
// once, and rows are many at once: 8192 rows of 10 parts of 128 take 15 us with one wave a row
// and 26 with four; 64 rows of 67 parts 10 with four.
template <typename T, int DV, int W> __global__ __launch_bounds__(256) void attn_merge_kernel(AttnArgs a) {
    constexpr int LANES = DV / 4, GROUPS = 64 * W / LANES, SLOTS = 128, ROWS = 4 / W;
    static_assert(GROUPS >= 1 && 64 * W * GROUPS % LANES == 0, "whole groups");
    __shared__ float2 stat_all[ROWS][SLOTS];
    __shared__ f32x4 sums_all[ROWS][GROUPS][LANES];
    const int tid = threadIdx.x % (64 * W), mine = threadIdx.x / (64 * W);
    const int64_t rows = (int64_t)a.seqs.tokens * a.heads, at = (int64_t)blockIdx.x * ROWS + mine;
    float2 *stat = stat_all[mine];
    const bool row = at < rows;
    const int token = row ? (int)(at / a.heads) : 0, h = row ? (int)(at % a.heads) : 0;
    const int group = tid / LANES, c = 4 * (tid % LANES);
    const AttnPlan &p = a.plan;
    // statistics of every slot, whether a part was written or not
    const int slots = p.prefix_splits + p.own_splits;
    float2 got[SLOTS / 64 / W > 0 ? SLOTS / 64 / W : 1];
#pragma unroll
    for (int i = 0; i * 64 * W < SLOTS; ++i) {
        const int k = tid + i * 64 * W;
        got[i] = row && k < slots ? a.stat[k * rows + at] : float2{0.f, 0.f};
    }
    const int s = a.seqs.cu ? session_search(a.seqs, token, threadIdx.x & 63,
                                             [](int first, int) { return first; })
                            : token / a.seqs.each;
    const int first = session_first(a.seqs, s), last = session_first(a.seqs, s + 1);
    const bool held = row && token >= first && token < last;  // in a session
    const int L = own_tokens(a.seqs, a.pages, s), P = prefix_tokens(a);
    const int lim = L - (last - token) + 1;  // own tokens that the row sees

    // which slots hold a part: the first n0 of the prefix's, the first n1 of the own ones
    const int pu = units_of(P), lu = units_of(L);
    const int u0 = p.joint ? pu + lu : pu, per0 = split_units(u0, p.prefix_splits);
    const int n0 = per0 > 0 ? (u0 + per0 - 1) / per0 : 0;
    const int per1 = p.joint ? 0 : split_units(lu, p.own_splits);
    const int n1 = per1 > 0 ? (lu + per1 - 1) / per1 : 0, n = n0 + n1;
#pragma unroll
    for (int i = 0; i * 64 * W < SLOTS; ++i) {
        const int k = tid + i * 64 * W, to = k < p.prefix_splits ? k : k - p.prefix_splits + n0;
        if (k < slots && (k < p.prefix_splits ? k < n0 : to < n)) stat[to] = got[i];
    }
    __syncthreads();
    float top = -__builtin_inff(), sum = 0.f;
    bool any = true;  // whether the row sees a token
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    if (held) {
        for (int k = 0; k < n; ++k) top = __builtin_fmaxf(top, stat[k].x);
        for (int k = 0; k < n; ++k) sum += stat[k].y * part_weight(stat[k], top);
        if (sum == 0.f) {  // the same in all lanes
            const int lane = threadIdx.x & 63;
            const int32_t *table = a.seqs.table + (int64_t)s * a.seqs.width;
            const bool shared = first_there(a.pages, a.prefix_pages, P, lane) < P;
            any = shared || first_there(a.pages, table, L, lane) < lim;
        }
#pragma unroll 4
        for (int k = group; k < n; k += GROUPS) {
            const int64_t from = k < n0 ? k : p.prefix_splits + k - n0;
            const f32x4 w = *reinterpret_cast<const f32x4 *>(a.part + (from * rows + at) * DV + c);
            const float f = part_weight(stat[k], top);
            if (f != 0.f) y += w * f;  // a part of which nothing was seen holds anything
        }
    }
    sums_all[mine][group][tid % LANES] = y;
    __syncthreads();
    if (group > 0 || !held) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) y += sums_all[mine][g][tid];
    const float inv = any ? 1.f / sum : 0.f;
    T *out = static_cast<T *>(a.out) + token * a.out_stride + (int64_t)h * DV + c;
    store4(out, y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    if (a.lse && c == 0)
        a.lse[at] = any ? (usable(top) + __builtin_log2f(sum)) * kLn2 : -__builtin_inff();
}

// Blocks of the launch; -1 where they are too many for one.
int64_t tile_grid(const AttnArgs &a, TileGrid *g) {
    const AttnPlan &p = a.plan;
    const int64_t rows = (int64_t)a.seqs.tokens * a.group;
    int64_t r0 = 0, t0 = 0, r1 = 0, t1 = 0;
    if (p.prefix_splits > 0 && !p.joint && !p.prefix_few) {
        r0 = (int64_t)a.kv_heads * p.prefix_splits;
        t0 = (rows + p.tile_rows - 1) / p.tile_rows;
    }
    if (p.joint || (p.own_splits > 0 && p.own_tiles)) {
        r1 = (int64_t)a.kv_heads * (p.joint ? p.prefix_splits : p.own_splits);
        // a session's first one: its first row's / tile_rows + its number
        t1 = rows / p.tile_rows + a.seqs.num;
    }
    constexpr int64_t kMost = (int64_t)1 << 22;  // 512 threads each
    if (r0 > kMost || t0 > kMost || r1 > kMost || t1 > kMost) return -1;
    const int64_t b0 = (r0 * t0 + 7) / 8 * 8, b1 = (r1 * t1 + 7) / 8 * 8;
    if (b0 + b1 > kMost) return -1;
    *g = {(int)r0, (int)t0, (int)b0, (int)r1, (int)t1, (int)b1};
    return b0 + b1;
}

int64_t few_blocks(const AttnArgs &a, int64_t *own) {
    const AttnPlan &p = a.plan;
    *own = p.few_rows > 0 && !p.joint ? (int64_t)a.seqs.num * a.kv_heads * p.own_splits : 0;
    return *own + (p.prefix_few ? (int64_t)a.kv_heads * p.prefix_splits : 0);
}

// NEAR: places of a head's values in 32 bits, drafts over 32K 173 us against 181 with 64 bits,
// prompts 624 against 666.
template <typename T, int D, int TK, int PLACES>
int mixed(const AttnArgs &a, const MixGrid &g, int64_t blocks, hipStream_t stream) {
    if (a.pages.near)
        hipLaunchKernelGGL((attn_kernel<T, D, TK, PLACES, true>), dim3((unsigned)blocks), dim3(256), 0,
                           stream, a, g);
    else
        hipLaunchKernelGGL((attn_kernel<T, D, TK, PLACES, false>), dim3((unsigned)blocks), dim3(256), 0,
                           stream, a, g);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

// Blocks of the launch in all, -1 where they are too many for one.
int64_t mix_grid(const AttnArgs &a, MixGrid *g) {
    int64_t own;
    const int64_t few = few_blocks(a, &own), tile = tile_grid(a, &g->tile);
    if (tile < 0 || few + tile > (1 << 23)) return -1;
    g->few = (int)few, g->own_few = (int)own;
    return few + tile;
}

}  // namespace

int64_t attn_threads(const AttnArgs &a) {
    MixGrid g;
    const int64_t n = mix_grid(a, &g);
    return n < 0 ? kMostThreads + 1 : n * 512;
}
// Workgroups of the join, and waves a row: all four of a workgroup, or where rows are more than
// workgroups run at once (8 a CU) as many as hold a row.
static int64_t merge_grid(const AttnArgs &a, int *waves) {
    const int64_t rows = (int64_t)a.seqs.tokens * a.heads;
    *waves = rows <= 2048 ? 4 : (a.dv == 512 ? 2 : 1);
    return (rows * *waves + 3) / 4;
}
int64_t attn_merge_threads(const AttnArgs &a) {
    int waves;
    return merge_grid(a, &waves) * 256;
}

int launch_attn(const AttnArgs &a, hipStream_t stream) {
    MixGrid g;
    const int64_t n = mix_grid(a, &g);
    if (n <= 0) return (int)n;
    if (a.d == 576) {
        hipLaunchKernelGGL(attn_latent_kernel, dim3((unsigned)n), dim3(512), 0, stream, a, g.tile);
        return hipGetLastError() == hipSuccess ? 0 : -1;
    }
    if (a.dtype == kDtypeF32)
        return a.d == 64 ? mixed<float, 64, 32, 2>(a, g, n, stream)
                         : mixed<float, 128, 32, 1>(a, g, n, stream);
    return a.d == 64 ? mixed<bf16, 64, 64, 2>(a, g, n, stream)
                     : mixed<bf16, 128, 64, 2>(a, g, n, stream);
}

namespace {

template <typename T, int DV> int merge(const AttnArgs &a, hipStream_t stream) {
    constexpr int FEW = DV == 512 ? 2 : 1;
    int waves;
    const dim3 grid((unsigned)merge_grid(a, &waves));
    if (waves == FEW)
        hipLaunchKernelGGL((attn_merge_kernel<T, DV, FEW>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((attn_merge_kernel<T, DV, 4>), grid, dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_attn_merge(const AttnArgs &a, hipStream_t stream) {
    if (a.dv == 512) return merge<bf16, 512>(a, stream);
    if (a.dtype == kDtypeF32)
        return a.dv == 64 ? merge<float, 64>(a, stream) : merge<float, 128>(a, stream);
    return a.dv == 64 ? merge<bf16, 64>(a, stream) : merge<bf16, 128>(a, stream);
}

}  // namespace kda
