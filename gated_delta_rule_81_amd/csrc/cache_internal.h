// cache_internal.h -- host-side launch functions of the operators on a paged
// cache (not part of the public ABI; see include/kda_cache.h).  Arguments are
// already validated.  Each returns 0, or -1 if a launch failed.
#pragma once

#include "kda_internal.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// New tokens of the sessions: packed offsets cu, or each = tokens / num of every one.
struct Sessions {
    const int32_t *cu, *lens, *table;
    int32_t num, each, tokens, width;  // width: columns of the page table
};

// x / d for 0 <= x < 2^31 as a product's upper half and two shifts (division by an invariant
// integer, Granlund and Montgomery 1994).
struct Divisor {
    uint32_t mul, sh1, sh2;
    Divisor() = default;
    explicit Divisor(uint32_t d) {
        uint32_t l = 0;
        while (l < 32 && ((uint64_t)1 << l) < d) ++l;
        mul = (uint32_t)((((((uint64_t)1 << l) - d) << 32) / d) + 1);
        sh1 = l < 1 ? l : 1, sh2 = l < 1 ? 0 : l - 1;
    }
#ifdef __HIPCC__
    __device__ uint32_t operator()(uint32_t x) const {
        const uint32_t t = __umulhi(mul, x);
        return (t + ((x - t) >> sh1)) >> sh2;
    }
#endif
};

// Places in a paged cache, in bytes.
struct Pages {
    int32_t count, size;
    Divisor by_size;
    int64_t page, token, head;  // distance between pages, tokens, heads
    // the first two in units of 2^shift bytes: every token's place of a head fits 32 bits
    uint32_t page_units, token_units;
    int32_t shift;
    int32_t near;  // every value of a head lies under 2^32 bytes behind its first: places in bytes
};

struct AppendArgs {
    const void *q, *k, *v;
    const float *table;
    const int32_t *positions;
    void *out_q, *k_cache, *v_cache;
    Sessions seqs;
    Pages pages;
    int32_t q_heads, kv_heads, head_dim, rot, rot_at, table_rows, interleaved, dtype;
    int64_t q_stride, k_stride, v_stride, out_q_stride;  // elements
};
int launch_cache_append(const AppendArgs &a, hipStream_t stream);

// How a call's work is cut.  Lengths are split in units of kSplitTokens tokens.
constexpr int kSplitTokens = 128;
constexpr int64_t kMostThreads = UINT32_MAX;  // of a launch
constexpr float kLn2 = 0.6931471805599453f;
struct AttnPlan {
    int32_t tile_rows;    // rows (tokens x heads of a group) of a workgroup of the tile kernel
    int32_t few_rows;     // sessions of at most so many rows go to the row kernel (0: none)
    int32_t prefix_few;   // the prefix goes to the row kernel
    int32_t joint;        // one walk over prefix and own tokens, in prefix_splits parts
    int32_t own_tiles;    // whether a session may have more than few_rows rows
    int32_t prefix_splits, own_splits;
};

struct AttnArgs {
    const void *q, *k_cache, *v_cache;
    const int32_t *prefix_pages, *prefix_len;
    void *out;
    float *lse;
    float *part;   // [slot][token][head][v_dim], slots: the prefix's splits, then the own ones
    float2 *stat;  // [slot][token][head]: maximum (in units of log 2), sum
    Sessions seqs;
    Pages pages;
    int32_t heads, kv_heads, group, d, dv, prefix_width, dtype;
    int64_t q_stride, out_stride;  // elements
    float scale;
    AttnPlan plan;
};
AttnPlan attn_plan(int64_t tokens, int64_t num_seqs, bool packed, int64_t q_heads,
                   int64_t kv_heads, int head_dim, int64_t own_tokens, int64_t prefix_tokens,
                   int dtype);
// Threads of the launches that a call is made of, and those.
int64_t attn_threads(const AttnArgs &a);
int64_t attn_merge_threads(const AttnArgs &a);
int launch_attn(const AttnArgs &a, hipStream_t stream);
int launch_attn_merge(const AttnArgs &a, hipStream_t stream);

}  // namespace kda
