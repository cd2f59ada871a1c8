/*
 * wall_paged.h -- C ABI of the paged Wall cache (libwall.so): the page plan of
 * a serving step, the append of its tokens and their attention over the pages.
 * Conventions, status codes and dtypes are those of wall.h.
 */
#ifndef WALL_PAGED_H
#define WALL_PAGED_H

#include "wall.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The paged cache: requests of different lengths share pools of pages of
 * page_size positions (32, 64 or 128).  No counterpart on the pages, whose
 * decode cache has one length for all batch rows; the key rows are the same
 * pre-rescaled ones (README "Decode"), with a page as the anchor chunk.
 *
 * Packed batch: n_req requests, request i owning rows [cu_q[i], cu_q[i+1])
 * of the n_tokens packed rows (cu_q int32 [n_req + 1]); its block_table row
 * (int32 [max_pages]) gives its pages in order.  One layer's pools:
 *   k_pages [num_pages, HQ, page_size, K], v_pages [num_pages, H, page_size, V]
 *   in `dtype`, r_pages [num_pages, HQ, K] int32 (each page's anchors).
 * Gate prefix, in fixed point with 24 fraction bits, in powers of two:
 *   e_t = rint(g_t * 2^24 / ln 2)   (fp32 product; clamped to 32 signed bits,
 *                                    so a step beyond -128 counts as -128)
 *   P_t = P_{t-1} + e_t             (64-bit; exact whatever the order)
 *   R_c = floor(P / 2^24 + 1/2) at page c's first position
 *   p_t = P_t / 2^24 - R_{page(t)}  (fp32)
 *   k_pages row of t = k_t * 2^(-p_t), rounded to `dtype`
 * so that for cached position j of page c and query t
 *   2^(P_t - P_j) k_j = 2^(p_t + R_{page(t)} - R_c) * (k_pages row of j).
 * |p_t| > 100 on some channel (a page whose gates sum past 100 powers of two)
 * cannot be stored and records WALL_ERR_RANGE; smaller pages reach further.
 * Gates may have either sign.  A query's factor 2^(p_t + R_{page(t)} - R_c) of
 * 2^127 and more counts as 2^127.
 * A row offset, slot or page id outside its array is never followed: it
 * records WALL_ERR_INVALID_ARG (wall_get_status) and what hangs on it is
 * unspecified.  r_pages, carry_in, carry_out and the arrays of `dtype` and fp32
 * values are aligned to 16 bytes (sink_bias and lse to 4), the other int32 and
 * int64 arrays to their element.  Limits: n_req <= 2^20, HQ <= 4096, num_pages *
 * page_size * HQ < 2^31.
 */

/*
 * wall_paged_plan -- a serving step's row offsets, pages and slots, from the
 * requests' lengths, on the device.  Request i has lens[i] cached tokens and
 * brings new_lens[i] more.  In: new_lens, lens [n_req], free_list [num_pages]
 * whose first *free_count entries are the free pages (a stack).  In/out:
 * block_table [n_req, max_pages], entries of the pages opened now written.
 * Out: cu_q [n_req + 1]; kv_lens [n_req] = lens + new_lens, or 0 for a
 * refused request; admitted [n_req]; slot_map [n_tokens] = page * page_size +
 * offset of each packed row, -1 for rows of refused requests and past
 * cu_q[n_req]; lens_out [n_req] and free_count_out, which may be lens and
 * free_count.  Pages come off the top of the stack in request order.  A
 * request is refused, and changes nothing, when its pages would not fit its
 * table row, when its rows would pass n_tokens (offsets are clamped there),
 * or when it needs a page and the pages needed up to and with it exceed the
 * stack.
 */
int wall_paged_plan(const int32_t* new_lens, const int32_t* lens, int32_t* block_table,
                    const int32_t* free_list, const int32_t* free_count, int n_req, int max_pages,
                    int num_pages, int page_size, int n_tokens, int32_t* cu_q, int32_t* kv_lens,
                    int64_t* slot_map, int32_t* admitted, int32_t* lens_out,
                    int32_t* free_count_out, wall_stream_t stream);

/* wall_paged_release -- pages of the requests with finished[i] != 0 back onto
 * the stack (request order, each in table order); their table entries become
 * -1 and their lens 0.  All arrays in place.  A table entry outside the pool is
 * no page: it records WALL_ERR_INVALID_ARG and is dropped. */
int wall_paged_release(const int32_t* finished, int32_t* lens, int32_t* block_table,
                       int32_t* free_list, int32_t* free_count, int n_req, int max_pages,
                       int num_pages, int page_size, wall_stream_t stream);

/* wall_paged_append_workspace -- bytes of workspace wall_paged_append needs
 * (0 is possible). */
size_t wall_paged_append_workspace(int n_req, int n_tokens, int max_new, int HQ, int K,
                                   int page_size);

/*
 * wall_paged_append -- packed new tokens into one layer's pools.  In: k
 * [n_tokens, H, K], v [n_tokens, H, V], g [n_tokens, HQ, K]; cu_q, kv_lens and
 * slot_map of a plan; max_new a bound on a request's new tokens (0: none
 * known); carry_in int64 [n_req, HQ, K], each request's P at its last cached
 * token (not read where nothing is cached).  Out: the tokens' rows of k_pages
 * and v_pages, r_pages of the pages that begin among them, carry_out (may be
 * carry_in; a request without new tokens keeps its carry), p [n_tokens, HQ, K]
 * fp32.  Rows of requests with kv_lens < rows (refused) and rows past
 * cu_q[n_req] are skipped.  A NaN gate makes its token's p and key row NaN.
 */
int wall_paged_append(const void* k, const void* v, const void* g, int dtype, const int32_t* cu_q,
                      const int32_t* kv_lens, const int64_t* slot_map, int n_req, int n_tokens,
                      int max_new, int H, int HQ, int K, int V, int page_size, int num_pages,
                      void* k_pages, void* v_pages, int32_t* r_pages, const int64_t* carry_in,
                      int64_t* carry_out, float* p, void* workspace, size_t workspace_bytes,
                      wall_stream_t stream);

/* wall_paged_attn_workspace -- bytes of workspace wall_paged_attn needs. */
size_t wall_paged_attn_workspace(int dtype, int n_req, int n_tokens, int max_new, int H, int HQ,
                                 int K, int V);

/*
 * wall_paged_attn -- attention of packed query rows over the paged cache.
 * Row r of request i's n rows sits at position t = kv_lens[i] - n + r and sees
 * cached positions j <= t (with a window, t - j < window_size):
 *   s_j = scale * sum_n q_n 2^(p_n + R_{page(t),n} - R_{page(j),n}) * k_pages_jn
 *   o = sum_j softmax(s, sink)_j v_j,   lse = log-sum-exp (natural)
 * In: q [n_tokens, HQ, K]; p of the same rows from wall_paged_append;
 * max_new a bound on a request's rows (0: none known; a request beyond it
 * records WALL_ERR_INVALID_ARG; 1 and up to 8 have kernels of their own, for
 * plain steps and for drafts); sink_bias [HQ] fp32 or NULL.  Out:
 * o [n_tokens, HQ, V]; lse [n_tokens, HQ] fp32 (may be NULL).  A request with
 * kv_lens < n sees nothing: o = 0, lse = -inf (the sink's bias with a sink).
 * One with kv_lens beyond max_pages * page_size is taken for such a one, and
 * records WALL_ERR_INVALID_ARG.
 * Rows past cu_q[n_req] are left as they are.  Table entries of pages that no
 * row sees (before the window) may be anything.
 */
int wall_paged_attn(const void* q, const float* p, int dtype, const int32_t* cu_q,
                    const int32_t* kv_lens, const int32_t* block_table, int n_req, int n_tokens,
                    int max_new, int max_pages, int H, int HQ, int K, int V, int page_size,
                    int num_pages, const void* k_pages, const void* v_pages,
                    const int32_t* r_pages, const float* sink_bias, float scale, int window_size,
                    void* o, float* lse, void* workspace, size_t workspace_bytes,
                    wall_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif
