/*
 * spec_cache.h -- C ABI of libspecverify's paged 4-bit KV cache: the cache
 * that a target model's verification pass over drafted rows reads, writes and
 * cuts back, on one NVIDIA GB300 (sm_103a).
 *
 * Conventions (arrays, streams, errors, workspaces) are those of
 * spec_verify.h.  `status` arrays here are optional (NULL) and accumulate:
 * bits are OR-ed in, so that one array cleared once can follow a request
 * through a whole step.
 *
 * The cache.  One layer's pool is num_pages x kv_heads blocks.  A block holds
 * one page of P tokens of one kv head, D values a key and D a value:
 *
 *     K codes [P][D/2] | K scales bf16 [P][D/32] | V codes [P][D/2] | V scales bf16 [P][D/32]
 *
 * P is 16, 32 or 64 and D is 64 or 128: P * D * 9/8 bytes a block, 4.5 bits a
 * value.  Element d of a row is the low (even d) or high (odd d) half of byte
 * d/2 and stands for (code - 8) * scale[d / 32].  Codes lie in 1..15 and
 * scales carry five significant bits, so that every value the cache stands
 * for is exact in bfloat16.  Block (page, head) starts at pool +
 * page * page_stride + head * head_stride (bytes, multiples of 16; pool
 * 16-byte aligned, device memory).
 *
 * Position t of request b lies in page page_table[b * table_stride + t / P],
 * slot t % P.  Entries outside [0, num_pages) hold no page; a position whose
 * entry is needed and holds none, or that lies past table_width pages, is
 * skipped (SPEC_ST_BAD_PAGE).
 *
 * Source page: [SD-survey], "大模型投机解码：Medusa、MTP、EAGLE、DFlash、DDTree 与
 * DSpark", §5 "DDTree" (position ids by depth, ancestor-only visibility; only
 * the accepted path's KV is kept).  The 4-bit format, the pages and the
 * sliding window have no counterpart there.
 */
#ifndef SPEC_CACHE_H
#define SPEC_CACHE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_ST_BAD_PAGE 128   /* a needed position has no page (or a page id / request id out of range) */
#define SPEC_ST_NO_PAGE  256   /* the free pages did not suffice: the request got none */
#define SPEC_ST_SHARED_PAGE 512 /* a request ends inside a page that others hold too: rows must not be written there */

/* bytes at the start of spec_cache_attend's workspace that begin zeroed */
#define SPEC_CACHE_WS_CONTROL 16384

/* bytes of one block (one page of one kv head); 0 if the shape is not supported */
size_t spec_cache_block_bytes(int head_dim, int page_size);

/* ------------------------------------------------------------------------
 * spec_cache_append -- write rows into the cache in 4 bits
 *   k, v     bf16; row (b, i, head) at b*bs + i*rs + head*hs (strides in
 *            elements, unit element stride).
 *   start    [B]: row (b, i) goes to position start[b] + i.
 *   count    NULL (n rows each) or [B] in [0, n] (values outside are cut).
 * Per group of 32 values: scale = amax / 7 rounded to five significant bits
 * (ties to even; 0 below 2^-120), code = 8 + round(x / scale) (ties to even).
 * A NaN is stored as 0, an infinity as +-7 steps of the group's largest
 * finite value, and SPEC_ST_BAD_ROW is set.
 * ---------------------------------------------------------------------- */
spec_status spec_cache_append(
    const void* k, int64_t k_bs, int64_t k_rs, int64_t k_hs,
    const void* v, int64_t v_bs, int64_t v_rs, int64_t v_hs,
    void* pool, int64_t page_stride, int64_t head_stride, int num_pages,
    const int32_t* page_table, int64_t table_stride, int table_width,
    const int32_t* start, const int32_t* count,
    int B, int n, int kv_heads, int head_dim, int page_size, int32_t* status, void* stream);

/* ------------------------------------------------------------------------
 * spec_cache_read -- rows of the cache as bf16 values (exact)
 *   k, v     outputs [B, n, kv_heads, D] contiguous; rows i >= count[b] and
 *            skipped positions are 0.
 * ---------------------------------------------------------------------- */
spec_status spec_cache_read(
    const void* pool, int64_t page_stride, int64_t head_stride, int num_pages,
    const int32_t* page_table, int64_t table_stride, int table_width,
    const int32_t* start, const int32_t* count,
    int B, int n, int kv_heads, int head_dim, int page_size,
    void* k, void* v, int32_t* status, void* stream);

/* ------------------------------------------------------------------------
 * spec_cache_attend -- attention of drafted rows over the cache
 * [SD-survey] §5 "DDTree": drafted nodes take position id = depth and see
 * only their ancestors.
 *
 * Request b's cache holds ctx_len[b] context positions and, behind them, the
 * K and V of its num_rows[b] drafted rows (spec_cache_append at ctx_len).
 * Row i < num_rows[b] has position p_i = ctx_len[b] + depth[b, i] (depth NULL:
 * i) and sees every context position, and drafted row j iff bit j of its
 * ancestor mask is set (mask NULL: j <= i).  With window > 0 it sees of these
 * only keys of position p with p_i - p < window or p < sinks.
 *
 *   q        bf16; row (b, i, h) at b*q_bs + i*q_rs + h*q_hs, h < q_heads; head
 *            h reads kv head h / (q_heads / kv_heads).
 *   num_rows NULL (n each) or [B] (cut to [0, n]); ctx_len is cut to what the
 *            table can hold.
 *   anc_mask NULL or [B, n, ceil(n/64)] uint64, as spec_tree_build writes it;
 *            depth NULL or [B, n] int32, cut to [0, n] (both, or a mask
 *            alone: depth = i).
 *   scale    multiplies q . k (> 0, < 1.4e37).
 * Outputs: out bf16 [B, n, q_heads, D] contiguous: softmax over the seen keys
 *   times V (sums in fp32; the weights meet V in bf16 and are divided by the sum
 *   of what they were rounded to); lse NULL or fp32 [B, n, q_heads]: natural log
 *   of the softmax's denominator, of weights before that rounding.  Rows that
 *   see nothing, and rows i >= num_rows[b], are 0 with lse = -inf.  Positions past the last drafted row, and context that lies
 *   outside every row's window, contribute nothing whatever the cache holds
 *   there.  Scales of all other positions must be finite, as spec_cache_append
 *   writes them.
 *   ws       sized by the query for the same shape, 16-byte aligned; its first
 *            SPEC_CACHE_WS_CONTROL bytes must be zero before the first call
 *            and are zero again after every call (except the error word that
 *            spec_workspace_error reads).  One workspace serves calls of any
 *            shape that fits it, one after another.  A captured graph keeps its
 *            address: it has to outlive the graph, and nothing else may use it
 *            while a replay runs.
 * 1 <= n <= 1024.  Deterministic: the same inputs give the same bits.
 * ---------------------------------------------------------------------- */
size_t spec_cache_attend_workspace_size(int B, int n, int q_heads, int kv_heads, int head_dim);
spec_status spec_cache_attend(
    const void* q, int64_t q_bs, int64_t q_rs, int64_t q_hs,
    const void* pool, int64_t page_stride, int64_t head_stride, int num_pages,
    const int32_t* page_table, int64_t table_stride, int table_width,
    const int32_t* ctx_len, const int32_t* num_rows,
    const uint64_t* anc_mask, const int32_t* depth, int window, int sinks, float scale,
    int B, int n, int q_heads, int kv_heads, int head_dim, int page_size,
    void* out, float* lse, int32_t* status, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * spec_cache_compact -- keep the accepted path's rows, in place
 * [SD-survey] §5 "DDTree": only the accepted path's KV is kept.  For j = 0 ..
 * num_accepted[b] the row at position ctx_len[b] + path[b, j] moves to
 * ctx_len[b] + j, in every layer and head, K and V.  path ([B, path_width], as
 * the tree walks write it) ascends, so path[b, j] >= j; an entry below j is
 * skipped (SPEC_ST_BAD_NODE).
 *   pool     layers pools, layer_stride bytes apart.
 * ---------------------------------------------------------------------- */
spec_status spec_cache_compact(
    void* pool, int layers, int64_t layer_stride, int64_t page_stride, int64_t head_stride, int num_pages,
    const int32_t* page_table, int64_t table_stride, int table_width,
    const int32_t* ctx_len, const int32_t* path, int path_width, const int32_t* num_accepted,
    int B, int kv_heads, int head_dim, int page_size, int32_t* status, void* stream);

/* ------------------------------------------------------------------------
 * Pages.  The state of a pool's pages (caller-owned, device memory):
 *   page_table [R, table_width] (row stride table_stride), num_held [R]: the
 *            pages of each request, in order; entries past num_held are -1.
 *   ref      [num_pages]: how many requests hold a page.
 *   free_list [num_pages], num_free [1]: a stack of the free pages.
 * All three calls are deterministic.  num_pages <= 2^20.
 *
 * spec_cache_reserve: request r gets the pages it lacks for length[r] tokens,
 *   off the top of the stack, requests in order: the i-th page taken is
 *   free_list[num_free - 1 - i].  A request whose pages, with those of all
 *   requests before it, exceed num_free gets none (SPEC_ST_NO_PAGE); one that
 *   needs more than table_width pages gets none (SPEC_ST_BAD_PAGE).
 * spec_cache_release: request r keeps the pages of length[r] tokens (0 frees
 *   the request); the others lose a reference, and those that nothing holds
 *   any more are pushed on the stack in ascending order.
 *   A page that a fork made shared is for reading: spec_cache_append and
 *   spec_cache_compact write where they are told to and would change the other
 *   holders' rows.  A request only comes to write there when it is cut back to
 *   a length inside a shared page; release says so (SPEC_ST_SHARED_PAGE, after
 *   all of the call's references are dropped).  To go on from such a length,
 *   fork the request at it, which gives the copy a page of its own for the
 *   rest, and release the request itself.
 * spec_cache_fork: request dst[f] becomes a copy of request src[f] at
 *   length[src[f]] tokens: it shares the full pages and gets one of its own
 *   for the rest, taken as in reserve, into which the rest's rows are copied
 *   in every layer and head.  new_page [F] receives that page, or -1.  dst[f]
 *   holds no page before and src[f] at least length's (else SPEC_ST_BAD_PAGE,
 *   and nothing is done for f); the dst are distinct and none is a src.
 *   status [F].
 * ---------------------------------------------------------------------- */
spec_status spec_cache_reserve(
    int32_t* page_table, int64_t table_stride, int table_width, int32_t* num_held,
    int32_t* ref, int32_t* free_list, int32_t* num_free, int num_pages,
    const int32_t* length, int R, int page_size, int32_t* status, void* stream);
spec_status spec_cache_release(
    int32_t* page_table, int64_t table_stride, int table_width, int32_t* num_held,
    int32_t* ref, int32_t* free_list, int32_t* num_free, int num_pages,
    const int32_t* length, int R, int page_size, int32_t* status, void* stream);
spec_status spec_cache_fork(
    void* pool, int layers, int64_t layer_stride, int64_t page_stride, int64_t head_stride,
    int32_t* page_table, int64_t table_stride, int table_width, int32_t* num_held,
    int32_t* ref, int32_t* free_list, int32_t* num_free, int num_pages,
    const int32_t* src, const int32_t* dst, const int32_t* length, int R, int F,
    int kv_heads, int head_dim, int page_size, int32_t* new_page, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_CACHE_H */
