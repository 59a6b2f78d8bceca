/*
 * gdn_cache.h - C ABI of the operators around a paged key/value cache held in 8 bits, for the
 * attention layers of a hybrid model: queries and keys prepared (norm of each head and position
 * rotation), keys and values appended, attention over the pages, and the upkeep of the pages
 * (forks of a prefix, growth with copy on write, freeing, compaction).
 *
 * They stand beside gdn_prefix_attention of gdn_hybrid.h and keep the library's conventions:
 * packed token streams, caller-owned buffers, a 256-byte workspace with the sticky device status
 * word (gdn_read_status), work enqueued on `stream`, invalid arguments rejected on the host
 * before anything is enqueued.  Page tables, lengths and row numbers live on the device and are
 * read there alone, so every call can be captured into a graph, a decode loop with the growth of
 * its rows included.  (The pages that gdn_scan.h cites name the attention layers and their prefix
 * cache without defining them: these operators have no counterpart there.)
 */
#ifndef GDN_CACHE_H
#define GDN_CACHE_H

#include "gdn_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Norm of each head of queries and keys, and the rotation by their positions, in one pass:
 *
 *     y = x * rsqrt(mean(x^2) + eps) * w                        (normalize != 0; w may be NULL: 1)
 *     (y_a, y_b) -> mscale * (y_a cos t - y_b sin t, y_b cos t + y_a sin t),   t = position * inv_freq[i]
 *
 * for the pairs i < rotary_dim / 2: a = i, b = i + rotary_dim / 2 (GDN_ROPE_HALF) or a = 2 i,
 * b = 2 i + 1 (GDN_ROPE_INTERLEAVED); elements from rotary_dim on are not rotated (nor scaled by
 * mscale).  Everything in fp32, rounded once.  The angle is the product of the position and inv_freq
 * as given, held as a 64-bit fraction of a turn: off by 2^-64 of a turn times the position, 2^-33 at
 * the farthest, whatever the frequency (up to 2^40 radians a token).
 *
 *  q, k           device [T, num_q_heads, D], [T, num_k_heads, D], dtype; k may be NULL
 *                 (num_k_heads 0)
 *  positions      device int32 [T] (any value); may be NULL when rotary_dim = 0
 *  inv_freq       device double [rotary_dim / 2], radians a token; may be NULL when rotary_dim = 0
 *  q_weight, k_weight   device [D], dtype, or NULL
 *  q_out, k_out   device, shapes of q and k; may be q and k themselves (with the same stride).
 *                 Any other overlap is not allowed.
 *  *_stride       elements between tokens (0: packed), heads and widths contiguous inside a row;
 *                 base addresses and strides multiples of 16 bytes
 *  head_dim       32, 64 or 128;  rotary_dim  a multiple of 16, 0 .. head_dim
 */
typedef enum gdn_rope_layout { GDN_ROPE_HALF = 0, GDN_ROPE_INTERLEAVED = 1 } gdn_rope_layout;

typedef struct gdn_rope_problem {
    int64_t num_tokens;          /* T >= 0 */
    int32_t num_q_heads;         /* >= 1 */
    int32_t num_k_heads;         /* >= 0 */
    int32_t head_dim;
    int32_t rotary_dim;
    gdn_dtype dtype;             /* of q, k, the weights and the outputs */
    gdn_rope_layout layout;
    int32_t normalize;
    float eps;                   /* >= 0 */
    float mscale;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;
} gdn_rope_problem;

gdn_status gdn_qk_norm_rope(const gdn_rope_problem* p, const void* q, const void* k, const int32_t* positions,
                            const double* inv_freq, const void* q_weight, const void* k_weight, void* q_out,
                            void* k_out, gdn_stream_t stream);

/*
 * A paged cache.  Page j of layer i holds page_size tokens of every key/value head, keys and
 * values, in e4m3 with one scale for each block (the tokens of a page for one head):
 *
 *     k of token t, head h = pages[i][j][0][h][t] * scales[i][j][0][h]     (values: [1])
 *
 * Row r holds lens[r] tokens in the pages table[r][0], table[r][1], ..; refs[j] rows hold page j
 * (0: free).  Rows may share pages: forks of one prefix.  All three are changed by
 * gdn_cache_update and gdn_cache_compact alone.  No call takes tokens back from a row, and freeing
 * gives up the pages that its lens count: a lens lowered by hand past the end of a page leaves that
 * page held for nobody.
 *
 * Scales are powers of two: the least with which the block's largest value is at most 448 times
 * its scale (2^-126 .. 2^120).  A block's scale can so grow when a token is appended without a
 * second rounding of what it holds (but for values below 2^-14 of the block's largest): what a
 * row's cache holds does not depend on how its tokens were cut into calls, which keeps a cache
 * hit equal to a recompute.  Infinities and NaN are held as NaN and do not count for the scale.
 */
typedef struct gdn_cache {
    int32_t num_layers;          /* L >= 1 */
    int32_t num_pages;           /* N >= 1, of each layer */
    int32_t page_size;           /* 16, 32, 64 or 128 tokens */
    int32_t num_kv_heads;        /* Hkv >= 1 */
    int32_t head_dim;            /* D: 32, 64 or 128 */
    int32_t num_rows;            /* R >= 1 */
    int32_t row_pages;           /* W >= 1: pages that a row may hold; W * page_size < 2^31 - 512 */
    void* pages;                 /* device [L, N, 2, Hkv, page_size, D] e4m3, 16-byte aligned */
    float* scales;               /* device [L, N, 2, Hkv] */
    int32_t* table;              /* device [R, W] */
    int32_t* lens;               /* device [R] */
    int32_t* refs;               /* device [N] (NULL will do for append and attention) */
} gdn_cache;

/*
 * A batch of requests, each with new tokens of one row: request b's are tokens cu_new[b] ..
 * cu_new[b + 1] of the packed streams, and the last ones of row rows[b], whose lens[rows[b]]
 * counts them already (gdn_cache_update grows it).
 *
 *  cu_new       device int32 [B + 1], never falling, from 0 to at most num_tokens; what lies
 *               behind cu_new[B] is neither read nor written
 *  rows         device int32 [B], or NULL for row b (then B <= R).  A negative or out-of-range
 *               row marks padding: nothing is appended, its queries get zeros and lse -infinity.
 *  max_new      host bound of a request's new tokens.  It decides the plan alone (results differ in
 *               their last roundings at most); a close one makes the better plan: decode batches of 8 to 256 requests whose bound is all of T take
 *               8 us more in bf16 (64 rows of 500 tokens 27 -> 35, of 4000 99 -> 107), in fp32 up
 *               to 1.7 times as long (84 -> 146), their append 7 us for 3.
 *  max_len      host bound of a row's tokens for attention, 0: W * page_size.  A close one makes
 *               the better plan, too (64 rows of 500 in a table for 500 without either: 46 us).
 *               Attention counts its work in units of 64 tokens, or of 128 where a head has more
 *               than 16 query rows in bf16 (head_dim 64 or 128): for each tile of 16 or 32 rows, or
 *               of 256, of each request and key/value head, those of max_len and 4 more.  Calls
 *               whose bounds allow more than 2^31 - 2^20 of them are GDN_ERR_UNSUPPORTED.
 *
 * A request with more new tokens or a longer row than these bounds is refused on the device:
 * GDN_ERR_INVALID_ARG in the status word, its results undefined (nothing is appended).
 *
 * A page number outside the pool among a row's pages is never followed: the status word takes
 * GDN_ERR_INVALID_ARG, and the request's results are undefined.
 */
typedef struct gdn_batch {
    int32_t num_requests;        /* B, 1 .. 4096 */
    int32_t max_new;             /* >= 1 */
    int64_t num_tokens;          /* T: tokens of the packed streams */
    int64_t max_len;
    const int32_t* cu_new;
    const int32_t* rows;
} gdn_batch;

/*
 * Appends keys and values: token t of a row goes to its page t / page_size, which has to be the
 * row's own (refs 1).  k, v: device [T, Hkv, D], dtype, strides as above.  Two requests of one
 * call must not share a row.
 */
gdn_status gdn_cache_append(const gdn_cache* c, int32_t layer, const gdn_batch* b, const void* k, const void* v,
                            gdn_dtype dtype, int64_t k_stride, int64_t v_stride, void* workspace, size_t ws_bytes,
                            gdn_stream_t stream);

/*
 * Causal attention of each request's new tokens over its row (their own keys and values, appended
 * before, included): new token i of n sees the tokens 0 .. lens - n + i,
 *
 *     x_j = softmax_scale (q_i . k_j),  o_i = sum_j e^{x_j} v_j / sum_j e^{x_j},  lse_i = log sum_j e^{x_j}
 *
 * A query that sees nothing gives o = 0 and lse = -infinity.  One token a request is a decode
 * step.  Scores, statistics and sums are fp32; bf16 queries meet the cache's values exactly, fp32
 * ones to 2^-22 of a row's largest.  A weight is rounded to half a step of 11 bits (bf16) or 22
 * (fp32), or by 2^-32 (bf16) or 2^-36 (fp32) of the row's largest weight where that is more.  In bf16
 * a block of values whose scale is r times the largest that the row sees has 2^-32 / r in that
 * place: 11 bits of its weights down to r = 2^-21, and a bit less for each power of two below.  In
 * fp32 it keeps them down to r = 2^-100.
 * All values are expected to be finite; a NaN spreads to every query of its own request.  What a
 * page holds behind a row's tokens is never taken into a result.
 *
 *  q            device [T, Hq, D], dtype (token stride q_stride); Hkv divides Hq, head h reads
 *               key/value head h / (Hq / Hkv), at most 128 query heads to one
 *  softmax_scale  any sign; softmax_scale * log2 e finite in fp32
 *  o            device [T, Hq, D], dtype, packed;  lse  device [T, Hq] fp32, or NULL.  Neither may
 *               overlap q, the cache or one another (not checked)
 *  scratch      device, 32-byte aligned, gdn_paged_scratch_bytes(...) bytes
 */
size_t gdn_paged_scratch_bytes(const gdn_cache* c, const gdn_batch* b, gdn_dtype dtype, int32_t num_q_heads);

gdn_status gdn_paged_attention(const gdn_cache* c, int32_t layer, const gdn_batch* b, const void* q, gdn_dtype dtype,
                               int32_t num_q_heads, int64_t q_stride, float softmax_scale, void* o, float* lse,
                               void* scratch, size_t scratch_bytes, void* workspace, size_t ws_bytes,
                               gdn_stream_t stream);

/*
 * One turn of upkeep, in this order (each part may be absent: count 0 or NULL):
 *
 *  1. free: the rows drop[0 ..] and fork_to[0 ..] give up their pages (lens 0);
 *  2. fork: row fork_to[i] becomes a fork of row fork_from[i]: the same pages, held once more (a
 *     source that was just freed leaves an empty row);
 *  3. grow: row r gets room for grow[r] more tokens (lens grows by it).  A last page that other
 *     rows hold too is copied first, in every layer, if the row has tokens in part of it: whether
 *     they do is seen before any row grows, so the last holders of a page that grow in one call all
 *     take a copy, and the page itself comes free.  New
 *     pages are the free ones with the lowest numbers, in the order of the rows and of their
 *     tokens.  Rows are served in order until one finds too few pages: it and the rows after it
 *     that need some are refused, as are rows that would pass W pages.
 *
 *  drop, fork_from, fork_to   device int32; row numbers out of range are passed over, a pair with
 *               from = to as well; a row that is named twice is freed once, and forked as the
 *               first of its pairs says
 *  grow         device int32 [R], or NULL; negative ones count as 0
 *  granted      device int32 [R], or NULL: grow[r], or -1 where row r was refused (and left as it is)
 *  scratch      device, 16-byte aligned, gdn_cache_scratch_bytes(c) bytes
 *
 * R <= 16384.
 */
size_t gdn_cache_scratch_bytes(const gdn_cache* c);

gdn_status gdn_cache_update(const gdn_cache* c, int32_t num_drop, const int32_t* drop, int32_t num_fork,
                            const int32_t* fork_from, const int32_t* fork_to, const int32_t* grow, int32_t* granted,
                            void* scratch, size_t scratch_bytes, void* workspace, size_t ws_bytes,
                            gdn_stream_t stream);

/*
 * Moves the pages in use together: with n of them, those at numbers from n on take the places that
 * are free below n, both in rising order; tables and refs follow.  live: device int32 [1], n.
 */
gdn_status gdn_cache_compact(const gdn_cache* c, int32_t* live, void* scratch, size_t scratch_bytes, void* workspace,
                             size_t ws_bytes, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_CACHE_H */
