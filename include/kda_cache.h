/*
 * kda_cache.h -- C ABI of libkda, the operators of a full attention layer beside
 * the recurrent ones of a hybrid model, as it is served from a paged cache (AMD
 * Instinct MI355X, gfx950, hand-written HIP):
 *
 *   - new keys and values appended to the cache, rotated by position on the way
 *     (kda_cache_append);
 *   - attention of a batch of sessions over a prefix that all of them share and
 *     each session's own tokens (kda_prefix_attn_*): single tokens, a few at a
 *     time, or prompts.  The prefix is read once for every 128 rows (tokens x heads
 *     of a group): of all sessions together, or, where a session has that many on
 *     average, of each.
 *
 * Conventions shared by both (those of kda_layer.h otherwise):
 *   - Cache: num_pages pages of page_size tokens of kv_heads heads of head_dim
 *     values.  The value at (page, token, head, channel) lies page * page_stride +
 *     token * token_stride + head * head_stride + channel elements behind the
 *     start, the same in k_cache and v_cache; strides are multiples of 16 bytes
 *     and two places never share a byte.  A head's places are counted in units of
 *     the largest power of two that divides page_stride and token_stride (in
 *     bytes): 2^32 of them are the most (1 TB where it is 256 bytes), a cache that
 *     holds more is refused (KDA_ERR_UNSUPPORTED).  A page may hold its tokens' heads
 *     together or its heads' tokens; the caches may be two tensors or halves of
 *     each page of one.
 *   - Latent cache: v_cache NULL.  A token's values are then the first v_dim
 *     channels of its keys.
 *   - New tokens: `tokens` rows, packed by cu_seqlens (a DEVICE int32 array of
 *     num_seqs + 1 offsets, 0 first, not decreasing, tokens last); NULL = tokens /
 *     num_seqs rows of each session.  Tokens behind the last offset are in no
 *     session: their outputs are left as they were.
 *   - lens [num_seqs] int32: how many tokens of its own each session has, the
 *     new ones (its last) among them.  New token i of n is own token lens - n + i;
 *     one that comes out under 0 has no place and sees no own token.
 *   - page_table [num_seqs, table_width] int32: the pages of each session's own
 *     tokens in order; lens over table_width * page_size count as that much.
 *   - lens, tables, offsets and prefix_len are read on the device: a captured
 *     call follows what they hold at each replay, within the widths of its tables.
 *   - An entry of a table that is read and is no page (under 0, or num_pages and
 *     more) is never followed: append leaves its tokens out, attention does not
 *     see them.  Pages that two sessions append to at the same place receive
 *     either's values.
 */
#ifndef KDA_CACHE_H_
#define KDA_CACHE_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kda_cache_append -- for every new token at own place p of its session, with
 * page = page_table[session][p / page_size] and slot = p % page_size,
 *     k_cache[page][slot] = R k,  v_cache[page][slot] = v,  out_q = R q,
 * where R rotates channels rotary_offset .. rotary_offset + rotary_dim of each
 * head: (a, b) <- (a cos - b sin, b cos + a sin) for pairs (i, i + rotary_dim / 2),
 * or (2 i, 2 i + 1) when interleaved != 0, i < rotary_dim / 2, with cos | sin from
 * row positions[token] of the table, in fp32, rounded once:
 *   q, out_q   [tokens, q_heads, head_dim]   dtype (rows *_stride apart), or q_heads 0
 *   k, v       [tokens, kv_heads, head_dim]  dtype (rows *_stride apart); v NULL with
 *                                            v_cache NULL
 *   table      [table_rows, rotary_dim]: cos, then sin           fp32
 *   positions  [tokens]  int32; values outside the table are moved into it
 * out_q may be q itself (the same rows).  A token without a place has its q
 * rotated all the same.  head_dim is 64, 128 or 576; rotary_dim and rotary_offset
 * multiples of 16, rotary_dim 0 = no rotation (table and positions are then not
 * read).  Row starts, caches and the table are 16-byte aligned.
 */
int kda_cache_append(const void *q, const void *k, const void *v, const float *table,
                     const int32_t *positions, const int32_t *page_table, const int32_t *lens,
                     const int32_t *cu_seqlens, void *out_q, void *k_cache, void *v_cache,
                     int32_t tokens, int32_t num_seqs, int32_t q_heads, int32_t kv_heads,
                     int32_t head_dim, int32_t rotary_dim, int32_t rotary_offset,
                     int32_t table_rows, int32_t num_pages, int32_t page_size,
                     int32_t table_width, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                     int64_t out_q_stride, int64_t page_stride, int64_t token_stride,
                     int64_t head_stride, int32_t interleaved, int32_t dtype,
                     hipStream_t stream);

/*
 * kda_prefix_attn_fwd -- softmax attention of every new token over the first
 * prefix_len[0] tokens of the pages prefix_pages, which every session shares, and
 * its session's own tokens up to itself:
 *     out = sum_j p_j v_j,  p_j = exp(scale q k_j - lse),  lse = log sum_j exp(scale q k_j)
 * with query head h reading key head h / (q_heads / kv_heads):
 *   q            [tokens, q_heads, head_dim]  dtype (rows q_stride apart)
 *   out          [tokens, q_heads, v_dim]     dtype (rows out_stride apart)
 *   lse          [tokens, q_heads] or NULL    fp32
 *   prefix_pages [prefix_width] int32, prefix_len [1] int32 (prefix_width 0: no
 *                prefix, neither is read); a prefix_len over the pages counts as theirs
 * A token that sees nothing, because no length or no page shows it anything, gets
 * out = 0 and lse = -inf; one whose scores are all -inf gets NaN and -inf, as the
 * formula has it.  What a token does not see never reaches it, NaN and infinities
 * included.  Scores, sums and the output
 * are held in fp32; bf16: each exp(..) enters its product with v rounded to bf16
 * once, the sum of them does not.
 *
 * (head_dim, v_dim): (64, 64), (128, 128) with v_cache, bf16 or fp32, or (576, 512)
 * with v_cache NULL, bf16.  scale > 0 and finite.  Row starts and caches are
 * 16-byte aligned.  A call of more than 2^22 workgroups of 128 rows, or of 2^23 with
 * those of the sessions of few rows (key heads x parts of each), is refused
 * (KDA_ERR_UNSUPPORTED), and where parts are joined one of 2^26 tokens x q_heads or
 * more (2^25 with v_dim 512).
 */
int64_t kda_prefix_attn_workspace_size(int32_t tokens, int32_t num_seqs, int32_t q_heads,
                                       int32_t kv_heads, int32_t head_dim, int32_t v_dim,
                                       int32_t page_size, int32_t table_width,
                                       int32_t prefix_width, int32_t dtype);
int kda_prefix_attn_fwd(const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *page_table, const int32_t *lens,
                        const int32_t *prefix_pages, const int32_t *prefix_len,
                        const int32_t *cu_seqlens, void *out, float *lse, int32_t tokens,
                        int32_t num_seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                        int32_t v_dim, int32_t num_pages, int32_t page_size,
                        int32_t table_width, int32_t prefix_width, int64_t q_stride,
                        int64_t out_stride, int64_t page_stride, int64_t token_stride,
                        int64_t head_stride, float scale, int32_t dtype, void *workspace,
                        int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* KDA_CACHE_H_ */
