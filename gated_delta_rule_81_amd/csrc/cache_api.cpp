// cache_api.cpp -- the C ABI declared in include/kda_cache.h: argument validation
// on the host, then the launches on the caller's stream.
//
// Validation order as in kda_api.cpp: sizes, NULL pointers, supported
// configurations, alignment, aliasing (host checks only), then the device,
// then (debug mode) the offsets, then the launch.
#include "cache_internal.h"
#include "kda_api_common.h"
#include "kda_cache.h"

namespace {

int elem_size(int32_t dtype) {
    return dtype == kda::kDtypeBf16 ? 2 : (dtype == kda::kDtypeF32 ? 4 : 0);
}

// Token numbers a little past the last one still fit 32 bits.
constexpr int64_t kMostTokens = INT32_MAX - 4095;

// Bytes from the first to the last of a tensor of rows.
Range rows_range(const void *p, int64_t rows, int64_t len, int64_t stride, int esz) {
    if (rows <= 0 || len <= 0) return {p, 0};
    return {p, (uint64_t)((rows - 1) * stride + len) * esz};
}

// Sizes of the sessions and their tables; *s receives them.
int check_sessions(const int32_t *cu, const int32_t *lens, const int32_t *table, int32_t tokens,
                   int32_t num_seqs, int32_t page_size, int32_t width, kda::Sessions *s) {
    if (tokens < 0 || num_seqs < 0 || page_size < 1 || width < 0) return KDA_ERR_SHAPE;
    if (tokens > kMostTokens || (int64_t)page_size * width > kMostTokens) return KDA_ERR_SHAPE;
    if (!cu && (num_seqs ? tokens % num_seqs != 0 : tokens != 0)) return KDA_ERR_SHAPE;
    *s = {cu, lens, table, num_seqs, cu || !num_seqs ? 0 : tokens / num_seqs, tokens, width};
    return KDA_OK;
}

// The cache's layout; strides in elements, places of two (page, token, head) apart.
int check_pages(int32_t num_pages, int32_t page_size, int32_t heads, int32_t d, int64_t page_stride,
                int64_t token_stride, int64_t head_stride, int esz, kda::Pages *p) {
    if (num_pages < 0 || heads < 0) return KDA_ERR_SHAPE;
    const int64_t limit = (int64_t)1 << 45;  // elements: sums and products stay in 64 bits
    if (page_stride < 0 || token_stride < 0 || head_stride < 0 || page_stride > limit ||
        token_stride > limit || head_stride > limit)
        return KDA_ERR_SHAPE;
    // an axis of one place may have any stride
    if (num_pages > 0 && heads > 0) {
        const int64_t n[2] = {page_size, heads}, s[2] = {token_stride, head_stride};
        const int in = page_size == 1 ? 1 : (heads == 1 ? 0 : (s[0] < s[1] ? 0 : 1)), out = 1 - in;
        int64_t span = d;
        const int order[2] = {in, out};
        for (int i = 0; i < 2; ++i) {
            const int k = order[i];
            if (n[k] == 1) continue;
            if (s[k] < span) return KDA_ERR_SHAPE;
            if (s[k] > ((int64_t)1 << 62) / n[k]) return KDA_ERR_SHAPE;
            span = (n[k] - 1) * s[k] + span;
        }
        if (num_pages > 1 && page_stride < span) return KDA_ERR_SHAPE;
        if (span > ((int64_t)1 << 58) || page_stride > ((int64_t)1 << 58) / num_pages)
            return KDA_ERR_SHAPE;
    }
    *p = {num_pages, page_size, kda::Divisor((uint32_t)page_size), page_stride * esz,
          token_stride * esz, head_stride * esz, 0, 0, 4, 0};
    // the largest power of two that divides both (16 bytes at least: checked with the alignment)
    const uint64_t page = num_pages > 1 ? (uint64_t)p->page : 0;
    const uint64_t token = page_size > 1 ? (uint64_t)p->token : 0, bits = page | token;
    while (p->shift < 32 && bits && ((bits >> p->shift) & 1) == 0) ++p->shift;
    const uint64_t most = (page >> p->shift) * (num_pages > 1 ? num_pages - 1 : 0) +
                          (token >> p->shift) * (page_size - 1);
    if (most > UINT32_MAX) return KDA_ERR_UNSUPPORTED;
    p->page_units = (uint32_t)(page >> p->shift), p->token_units = (uint32_t)(token >> p->shift);
    p->near = ((most << p->shift) + (uint64_t)d * esz) >> 32 == 0;
    return KDA_OK;
}

// One cache: its pages, each of `len` bytes, `stride` bytes apart.
struct CacheSpan {
    const void *p;
    uint64_t bytes, stride, len;
};
CacheSpan cache_span(const void *p, const kda::Pages &g, int32_t heads, int32_t d, int esz) {
    if (!p || g.count == 0 || heads == 0) return {p, 0, 0, 0};
    const uint64_t len = (uint64_t)(g.size > 1 ? (g.size - 1) * g.token : 0) +
                         (uint64_t)(heads > 1 ? (heads - 1) * g.head : 0) + (uint64_t)d * esz;
    return {p, (uint64_t)(g.count > 1 ? (g.count - 1) * g.page : 0) + len,
            g.count > 1 ? (uint64_t)g.page : 0, len};
}
Range whole(const CacheSpan &c) { return {c.p, c.bytes}; }

// Halves of each page of one tensor (or of each token's or head's place) share no byte.
bool caches_overlap(const void *k, const void *v, const kda::Pages &g, int32_t heads, int32_t d,
                    int esz) {
    if (!overlap(whole(cache_span(k, g, heads, d, esz)), whole(cache_span(v, g, heads, d, esz))))
        return false;
    int64_t apart = (int64_t)reinterpret_cast<uintptr_t>(v) - (int64_t)reinterpret_cast<uintptr_t>(k);
    if (apart < 0) apart = -apart;
    // v's places are k's moved by `apart`: they meet k's only where a difference of two places is
    // within a row's length of it.  From the widest axis inwards, such a difference is fixed
    // but for the two neighbours of a quotient.
    const int64_t n[3] = {g.count, g.size, heads}, s[3] = {g.page, g.token, g.head};
    int order[3] = {0, 1, 2};
    if (s[1] < s[2]) order[1] = 2, order[2] = 1;
    const int64_t len = (int64_t)d * esz;
    for (int a = -1; a <= 1; ++a)
        for (int b = -1; b <= 1; ++b)
            for (int c = -1; c <= 1; ++c) {
                const int near[3] = {a, b, c};
                int64_t left = apart;
                bool in = true;
                for (int i = 0; i < 3; ++i) {
                    const int64_t stride = s[order[i]], most = n[order[i]] - 1;
                    int64_t q = stride > 0 && most > 0 ? left / stride + near[i] : 0;
                    if (q > most || q < -most) in = false;
                    left -= q * stride;
                }
                if (in && left < len && left > -len) return true;
            }
    return false;
}

bool multiple16(int64_t stride, int esz) { return stride * esz % 16 == 0; }

}  // namespace

extern "C" {

int kda_cache_append(const void *q, const void *k, const void *v, const float *table,
                     const int32_t *positions, const int32_t *page_table, const int32_t *lens,
                     const int32_t *cu_seqlens, void *out_q, void *k_cache, void *v_cache,
                     int32_t tokens, int32_t num_seqs, int32_t q_heads, int32_t kv_heads,
                     int32_t head_dim, int32_t rotary_dim, int32_t rotary_offset,
                     int32_t table_rows, int32_t num_pages, int32_t page_size,
                     int32_t table_width, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                     int64_t out_q_stride, int64_t page_stride, int64_t token_stride,
                     int64_t head_stride, int32_t interleaved, int32_t dtype,
                     hipStream_t stream) {
    kda::Sessions seqs;
    kda::Pages pages;
    int st = check_sessions(cu_seqlens, lens, page_table, tokens, num_seqs, page_size, table_width,
                            &seqs);
    if (st != KDA_OK) return st;
    if (q_heads < 0 || kv_heads < 0 || head_dim <= 0 || rotary_dim < 0 || rotary_offset < 0 ||
        (int64_t)rotary_offset + rotary_dim > head_dim)
        return KDA_ERR_SHAPE;
    const int esz = elem_size(dtype);
    if (!esz) return KDA_ERR_UNSUPPORTED;
    if (((int64_t)q_heads + 2 * (int64_t)kv_heads) * head_dim > INT32_MAX / 4)
        return KDA_ERR_UNSUPPORTED;  // a token's pieces are counted in 32 bits
    if ((st = check_pages(num_pages, page_size, kv_heads, head_dim, page_stride, token_stride,
                          head_stride, esz, &pages)) != KDA_OK)
        return st;
    const int64_t ql = (int64_t)q_heads * head_dim, kl = (int64_t)kv_heads * head_dim;
    const bool some = tokens > 0 && num_seqs > 0, any_q = some && q_heads > 0;
    const bool any_k = some && kv_heads > 0;
    if ((any_q && (q_stride < ql || out_q_stride < ql)) || (any_k && k_stride < kl) ||
        (any_k && v && v_stride < kl))
        return KDA_ERR_SHAPE;
    if ((any_q && (!q || !out_q)) || (any_k && (!k || (!v) != (!v_cache)))) return KDA_ERR_NULL;
    if (any_k && num_pages > 0 && (!k_cache || (v && !v_cache))) return KDA_ERR_NULL;
    if ((any_q || any_k) && (!lens || (table_width > 0 && !page_table))) return KDA_ERR_NULL;
    if (rotary_dim > 0 && (any_q || any_k)) {
        if (!table || !positions) return KDA_ERR_NULL;
        if (table_rows < 1) return KDA_ERR_SHAPE;
    }
    if (head_dim != 64 && head_dim != 128 && head_dim != 576) return KDA_ERR_UNSUPPORTED;
    if (rotary_dim % 16 != 0 || rotary_offset % 16 != 0) return KDA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out_q) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned16(table) || !aligned4(positions) || !aligned4(page_table) ||
        !aligned4(lens) || !aligned4(cu_seqlens) ||
        (any_q && (!multiple16(q_stride, esz) || !multiple16(out_q_stride, esz))) ||
        (any_k && (!multiple16(k_stride, esz) || (v && !multiple16(v_stride, esz)) ||
                   !multiple16(page_stride, esz) || !multiple16(token_stride, esz) ||
                   !multiple16(head_stride, esz))))
        return KDA_ERR_ALIGN;
    const bool rot = rotary_dim > 0;
    const Range kc = whole(cache_span(k_cache, pages, kv_heads, head_dim, esz));
    const Range vc = whole(cache_span(v_cache, pages, kv_heads, head_dim, esz));
    const Range rq = rows_range(q, any_q ? tokens : 0, ql, q_stride, esz);
    const Range ro = rows_range(out_q, any_q ? tokens : 0, ql, out_q_stride, esz);
    const Range ins[] = {rows_range(k, any_k ? tokens : 0, kl, k_stride, esz),
                         rows_range(v, any_k ? tokens : 0, kl, v_stride, esz),
                         {rot ? table : nullptr, (uint64_t)table_rows * rotary_dim * 4},
                         {rot ? positions : nullptr, (uint64_t)tokens * 4},
                         {page_table, (uint64_t)num_seqs * table_width * 4},
                         {lens, (uint64_t)num_seqs * 4},
                         {cu_seqlens, ((uint64_t)num_seqs + 1) * 4}};
    // rotated in place: beside k and v in the same rows
    const bool in_place = q == out_q && q_stride == out_q_stride;
    if (!in_place && overlap(ro, rq)) return KDA_ERR_ALIAS;
    for (int i = 0; i < 7; ++i) {
        if (overlap(kc, ins[i]) || overlap(vc, ins[i])) return KDA_ERR_ALIAS;
        if (!overlap(ro, ins[i])) continue;
        const int64_t stride = i == 0 ? k_stride : v_stride;
        if (i > 1 || stride != out_q_stride) return KDA_ERR_ALIAS;
        const int64_t row = stride * esz;
        const int64_t apart = (int64_t)reinterpret_cast<uintptr_t>(ins[i].p) -
                              (int64_t)reinterpret_cast<uintptr_t>(out_q);
        const int64_t col = (apart % row + row) % row;
        if (col < ql * esz || col + kl * esz > row) return KDA_ERR_ALIAS;
    }
    if (overlap(ro, kc) || overlap(ro, vc) || overlap(rq, kc) || overlap(rq, vc))
        return KDA_ERR_ALIAS;
    if (k_cache && v_cache && any_k && num_pages > 0 &&
        caches_overlap(k_cache, v_cache, pages, kv_heads, head_dim, esz))
        return KDA_ERR_ALIAS;
    if (!any_q && !any_k) return KDA_OK;
    if ((st = check_device()) != KDA_OK) return st;
    const char *where = "kda_cache_append";
    if (debug_mode() &&
        (st = debug_check_offsets(cu_seqlens, num_seqs, tokens, stream, where)) != KDA_OK)
        return st;
    const kda::AppendArgs a = {q,       k,        v,        table,    positions,     out_q,
                               k_cache, v_cache,  seqs,     pages,    q_heads,       kv_heads,
                               head_dim, rotary_dim, rotary_offset, table_rows, interleaved != 0, dtype,
                               q_stride, k_stride, v_stride, out_q_stride};
    return launch_status(kda::launch_cache_append(a, stream), stream, where);
}

}  // extern "C"

namespace kda {

// How a call is cut: see AttnPlan.  Rows are the tokens times the heads of a group.  Lengths are on the
// device and sizes alone decide: the widths of the tables stand for them, so a table far wider than
// the lengths may be cut more often than they need (256 single tokens behind 16K with up to 2000 of
// their own, a table of 128K 303 us, of 2000 289).
AttnPlan attn_plan(int64_t tokens, int64_t num_seqs, bool packed, int64_t q_heads,
                   int64_t kv_heads, int head_dim, int64_t own_tokens, int64_t prefix_tokens,
                   int dtype) {
    AttnPlan p = {};
    const bool latent = head_dim == 576;
    const int64_t rows = tokens * (q_heads / kv_heads);
    const int64_t most = packed ? rows : rows / num_seqs;  // of a session
    const int64_t own_units = (own_tokens + kSplitTokens - 1) / kSplitTokens;
    const int64_t pre_units = (prefix_tokens + kSplitTokens - 1) / kSplitTokens;
    p.tile_rows = 128;
    // 128 sessions of up to 7900 own tokens 388 us with the walk of few rows, 458 without; fp32, 24
    // sessions behind 2001 56 and 124; four drafts of 64 sessions behind 32K 173 and 170
    p.few_rows = latent ? 0 : 32;
    p.prefix_few = !latent && pre_units > 0 && rows <= 32;
    p.own_tiles = most > p.few_rows;
    // Sessions of a tile's rows each, on average: one walk over both leaves no parts to join (six
    // prompts behind 6000 tokens 624 us, in two walks 1117).  With fewer rows a session's tiles
    // are not full (latent 96 heads: 305 against 198; 32 rows of drafts: 421 against 173).  The average
    // stands for all: single tokens beside a long prompt walk the prefix on their own (4096 tokens
    // and 100 single ones behind 16K 1854 us; the two apart 1204 + 93).
    p.joint = p.own_tiles && own_units > 0 && pre_units > 0 && rows >= num_seqs * p.tile_rows;
    // At most 64 parts of each kind: the join holds the statistics of 128.  (One or two key heads over a
    // long length leave places empty: one token behind 256K, one key head, 49 us for 134 MB.)
    auto cut = [](int64_t want, int64_t units) {
        const int64_t n = want < units ? want : units;
        return (int32_t)(n < 1 ? 1 : (n > 64 ? 64 : n));
    };
    const int64_t slots = latent ? 256 : 512;  // workgroups that run at once on the card's 256 CUs
    const int64_t tiles = (rows + p.tile_rows - 1) / p.tile_rows;
    if (p.joint) {
        p.few_rows = 0;
        p.prefix_splits = cut(slots / (kv_heads * tiles), pre_units + own_units);
        return p;
    }
    // workgroups of the sessions' own tokens, where those go tile by tile
    const int64_t own_tiles =
        own_units > 0 && !p.few_rows ? kv_heads * num_seqs * ((most + p.tile_rows - 1) / p.tile_rows) : 0;
    if (pre_units > 0) {
        // as many parts as fill the places that those leave, if they leave enough (latent, 64 sessions
        // behind 8192: 4 parts 216 us, 5 263, 6 280, 8 235, on one card)
        const int64_t one = p.prefix_few ? kv_heads : kv_heads * tiles, left = slots - own_tiles;
        p.prefix_splits = cut((left >= one ? left : slots) / one, pre_units);
    }
    if (own_units > 0 && p.few_rows > 0 && rows >= num_seqs * p.tile_rows) {
        // Prompts without a prefix: a part holds all of their rows, so no more than fill the places
        // that their tiles leave.  (Cut as the lengths of few rows are: one prompt of 8K, 32 heads,
        // 4818 us and 8.1 GiB of parts, this 673 and none; 512 tokens behind 32K 643 and 418.)
        p.own_splits = cut(slots / (kv_heads * tiles), own_units);
    } else if (own_units > 0 && p.few_rows > 0) {
        // twice as many as run at once (four times: fp32, 24 sessions 62 us against 56), and lengths
        // over 2048 tokens cut so that ragged ones even out (128 sessions of 500 to 7900: 427 to 388 us)
        const int64_t base = kv_heads * num_seqs, even = own_units / 16 < 4 ? own_units / 16 : 4;
        const int64_t want = (2 * slots + base - 1) / base;
        p.own_splits = cut(want < even ? even : want, own_units);
    } else if (own_units > 0) {
        // a part of many rows is large beside the tokens it stands for: only where workgroups lack
        p.own_splits = cut((slots - kv_heads * tiles * p.prefix_splits) / own_tiles, own_units);
    }
    return p;
}

}  // namespace kda

namespace {

// Bytes of the parts of a plan (values, then maxima and sums), 0 where there is one part.
int64_t part_bytes(const kda::AttnPlan &p, bool packed, int64_t tokens, int64_t q_heads,
                   int64_t v_dim, int64_t *values) {
    const int64_t slots = (int64_t)p.prefix_splits + p.own_splits;
    *values = slots * tokens * q_heads * v_dim * 4;
    if (slots == 0) return 0;
    // one part, whose kernel knows the sessions' tokens, is the output
    if (slots == 1 && (!packed || p.joint || p.own_splits)) return 0;
    return *values + slots * tokens * q_heads * 8;
}

bool attn_dims(int32_t d, int32_t dv, int32_t dtype) {
    return (d == 64 && dv == 64) || (d == 128 && dv == 128) ||
           (d == 576 && dv == 512 && dtype == kda::kDtypeBf16);
}

}  // namespace

extern "C" {

int64_t kda_prefix_attn_workspace_size(int32_t tokens, int32_t num_seqs, int32_t q_heads,
                                       int32_t kv_heads, int32_t head_dim, int32_t v_dim,
                                       int32_t page_size, int32_t table_width,
                                       int32_t prefix_width, int32_t dtype) {
    if (tokens < 0 || num_seqs < 0 || q_heads < 0 || kv_heads < 0 || page_size < 1 ||
        table_width < 0 || prefix_width < 0 || !attn_dims(head_dim, v_dim, dtype) || !elem_size(dtype))
        return -1;
    if (tokens > kMostTokens || (int64_t)page_size * table_width > kMostTokens ||
        (int64_t)page_size * prefix_width > kMostTokens)
        return -1;
    if (tokens == 0 || num_seqs == 0 || q_heads == 0) return 0;
    if (kv_heads == 0 || q_heads % kv_heads != 0) return -1;
    // the larger of packed and equal sessions
    int64_t need = 0;
    for (int packed = tokens % num_seqs != 0; packed < 2; ++packed) {
        int64_t values;
        const kda::AttnPlan p = kda::attn_plan(tokens, num_seqs, packed, q_heads, kv_heads, head_dim,
                                               (int64_t)page_size * table_width,
                                               (int64_t)page_size * prefix_width, dtype);
        const int64_t n = part_bytes(p, packed, tokens, q_heads, v_dim, &values);
        need = n > need ? n : need;
    }
    return need;
}

int kda_prefix_attn_fwd(const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *page_table, const int32_t *lens,
                        const int32_t *prefix_pages, const int32_t *prefix_len,
                        const int32_t *cu_seqlens, void *out, float *lse, int32_t tokens,
                        int32_t num_seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                        int32_t v_dim, int32_t num_pages, int32_t page_size,
                        int32_t table_width, int32_t prefix_width, int64_t q_stride,
                        int64_t out_stride, int64_t page_stride, int64_t token_stride,
                        int64_t head_stride, float scale, int32_t dtype, void *workspace,
                        int64_t workspace_bytes, hipStream_t stream) {
    kda::Sessions seqs;
    kda::Pages pages;
    int st = check_sessions(cu_seqlens, lens, page_table, tokens, num_seqs, page_size, table_width,
                            &seqs);
    if (st != KDA_OK) return st;
    if (q_heads < 0 || kv_heads < 0 || head_dim <= 0 || v_dim <= 0 || prefix_width < 0 ||
        (int64_t)page_size * prefix_width > kMostTokens)
        return KDA_ERR_SHAPE;
    if (q_heads > 0 && (kv_heads == 0 || q_heads % kv_heads != 0)) return KDA_ERR_SHAPE;
    if (!(scale > 0.f) || scale > 3.4e38f) return KDA_ERR_SHAPE;
    const int esz = elem_size(dtype);
    if (!esz) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)q_heads * head_dim > INT32_MAX / 4) return KDA_ERR_UNSUPPORTED;
    if ((st = check_pages(num_pages, page_size, kv_heads, head_dim, page_stride, token_stride,
                          head_stride, esz, &pages)) != KDA_OK)
        return st;
    const bool work = tokens > 0 && num_seqs > 0 && q_heads > 0;
    const int64_t ql = (int64_t)q_heads * head_dim, ol = (int64_t)q_heads * v_dim;
    if (work && (q_stride < ql || out_stride < ol)) return KDA_ERR_SHAPE;
    if (work && (!q || !out || !lens || (table_width > 0 && !page_table) ||
                 (prefix_width > 0 && (!prefix_pages || !prefix_len)) || (num_pages > 0 && !k_cache)))
        return KDA_ERR_NULL;
    if (!attn_dims(head_dim, v_dim, dtype)) return KDA_ERR_UNSUPPORTED;
    if (work && num_pages > 0 && head_dim != 576 && !v_cache) return KDA_ERR_NULL;
    if (head_dim == 576 && v_cache) return KDA_ERR_UNSUPPORTED;
    kda::AttnArgs a = {};
    int64_t values = 0, need = 0;
    if (work) {
        a.plan = kda::attn_plan(tokens, num_seqs, cu_seqlens != nullptr, q_heads, kv_heads, head_dim,
                                (int64_t)page_size * table_width, (int64_t)page_size * prefix_width,
                                dtype);
        need = part_bytes(a.plan, cu_seqlens != nullptr, tokens, q_heads, v_dim, &values);
    }
    if (need > 0 && !workspace) return KDA_ERR_NULL;
    if (workspace_bytes < need) return KDA_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        !aligned16(workspace) || !aligned4(lse) || !aligned4(page_table) || !aligned4(lens) ||
        !aligned4(prefix_pages) || !aligned4(prefix_len) || !aligned4(cu_seqlens) ||
        (work && (!multiple16(q_stride, esz) || !multiple16(out_stride, esz) ||
                  !multiple16(page_stride, esz) || !multiple16(token_stride, esz) ||
                  !multiple16(head_stride, esz))))
        return KDA_ERR_ALIGN;
    if (work) {
        const Range outs[] = {rows_range(out, tokens, ol, out_stride, esz),
                              {lse, (uint64_t)tokens * q_heads * 4},
                              {workspace, (uint64_t)need}};
        const Range ins[] = {rows_range(q, tokens, ql, q_stride, esz),
                             whole(cache_span(k_cache, pages, kv_heads, head_dim, esz)),
                             whole(cache_span(v_cache, pages, kv_heads, head_dim, esz)),
                             {page_table, (uint64_t)num_seqs * table_width * 4},
                             {lens, (uint64_t)num_seqs * 4},
                             {prefix_width ? prefix_pages : nullptr, (uint64_t)prefix_width * 4},
                             {prefix_width ? prefix_len : nullptr, 4},
                             {cu_seqlens, ((uint64_t)num_seqs + 1) * 4}};
        for (int i = 0; i < 3; ++i) {
            for (int j = i + 1; j < 3; ++j)
                if (overlap(outs[i], outs[j])) return KDA_ERR_ALIAS;
            for (const Range &r : ins)
                if (overlap(outs[i], r)) return KDA_ERR_ALIAS;
        }
    }
    if (!work) return KDA_OK;
    a.q = q, a.k_cache = k_cache, a.v_cache = v_cache;
    a.prefix_pages = prefix_pages, a.prefix_len = prefix_len, a.out = out, a.lse = lse;
    a.seqs = seqs, a.pages = pages, a.heads = q_heads, a.kv_heads = kv_heads;
    a.group = q_heads / kv_heads, a.d = head_dim, a.dv = v_dim, a.prefix_width = prefix_width;
    a.dtype = dtype, a.q_stride = q_stride, a.out_stride = out_stride, a.scale = scale;
    const bool parts = need > 0 || a.plan.prefix_splits + a.plan.own_splits == 0;
    if (need > 0) {
        a.part = static_cast<float *>(workspace);
        a.stat = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + values);
    }
    if (kda::attn_threads(a) > kda::kMostThreads ||
        (parts && kda::attn_merge_threads(a) > kda::kMostThreads))
        return KDA_ERR_UNSUPPORTED;
    if ((st = check_device()) != KDA_OK) return st;
    const char *where = "kda_prefix_attn_fwd";
    if (debug_mode() &&
        (st = debug_check_offsets(cu_seqlens, num_seqs, tokens, stream, where)) != KDA_OK)
        return st;
    int rc = kda::launch_attn(a, stream);
    if (rc == 0 && parts) rc = kda::launch_attn_merge(a, stream);
    return launch_status(rc, stream, where);
}

}  // extern "C"
