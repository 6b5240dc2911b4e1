/*
 * kmeans_cache.h -- the paged key/value cache that K-Means compresses, on one
 * MI355X (gfx950): tables, append and attention (libkm_cache.so).
 *
 * Citations name the page "Flash-KMeans: Fast and Memory-Efficient Exact
 * K-Means" (gist.science summary of paper 2603.09229): "tech §n" is a section
 * of its technical summary.  The page names key/value-cache compression and
 * longer contexts as users of K-Means as an online primitive (tech §1, §5);
 * it describes no cache.  The rules below are this library's.
 *
 * The cache.  Keys and values of `heads` heads of `dim` 16-bit elements live
 * in pages of `page_size` slots.  Slot s of the cache is entry s % page_size
 * of page s / page_size.  Row r of the block table lists the pages of request
 * r in order: its i-th slot is slot table[r][i / page_size] * page_size +
 * i % page_size.  A slot usually holds one token.  It may instead hold a
 * centroid of n tokens' keys beside the mean of their values, with the
 * logarithm of n as its weight: the attention adds that weight to the slot's
 * score, so the slot counts as n equal keys.
 *
 * Conventions are those of kmeans.h: device pointers, caller-owned memory, a
 * workspace of any content, asynchronous work on `stream` (NULL = the default
 * stream), no host synchronisation, no allocation, arguments checked before
 * any HIP call, and a km_status as result.  Calls can be captured in a HIP
 * graph.  kmeans_kv_last_error() describes the last failure of the calling
 * thread.  Strides count elements.  Data that only the device can see is
 * checked there: a page, slot or position out of range is never read or
 * written, with the outcome each call states.
 */
#ifndef MEANS_CLUSTERING_AMD_KMEANS_CACHE_H
#define MEANS_CLUSTERING_AMD_KMEANS_CACHE_H

#include "kmeans.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A key/value cache in device memory.  The element strides of page, slot and
 * head are free (pages x slots x heads x dim and pages x heads x slots x dim
 * are both usual), elements of a row are adjacent.  Rows must be 16-byte
 * aligned: k and v 16-byte aligned, strides multiples of 8.
 * Limits: dim a multiple of 16 up to 256; heads up to 65,536; page_size a power
 * of two from 16 to 2^20; pages * page_size < 2^31; strides < 2^40.
 */
typedef struct km_kv_cache {
  void* k;
  void* v;
  int64_t pages, page_size, heads, dim;
  int64_t k_page, k_slot, k_head;
  int64_t v_page, v_slot, v_head;
} km_kv_cache;

/*
 * kmeans_kv_tables -- the tables of one serving step, from request lengths.
 * Request r holds ctx_lens[r] slots and gets new_lens[r] new tokens; negative
 * lengths count as 0.  Pages have = ceil(ctx / page_size) up to need =
 * ceil((ctx + new) / page_size) are taken from the free list in request
 * order.
 *   ctx_lens, new_lens  device int32[R]                      (read)
 *   pos_offset  device int32[R] or NULL: added to positions (tokens that a
 *               request has seen but no longer holds)        (read)
 *   block_table device int32, R rows `table_stride` apart, `width` columns:
 *               entries below have are read, entries have .. need-1 written,
 *               the others left as they are
 *   free_pages  device int32[num_free]: pages to take, in order (read)
 *   seq_lens    device int32[R]: ctx + new                   (written)
 *   query_start device int32[R+1]: first new token of each request, total
 *   page_start  device int32[R+1]: first entry of free_pages that each request
 *               takes; page_start[R] pages are taken in all
 *   positions   device int32[T]: ctx + i + pos_offset of token i of a request
 *   slots       device int32[T]: the token's slot in the cache
 * T is the capacity of positions and slots.  Tokens beyond the total get
 * position 0 and slot -1; tokens that find no room (free list or table row
 * exhausted: page_start[R] > num_free, or need > width) get slot -1 and their
 * table entries -1.  Tokens in a page that no cache can have (negative, or
 * 2^31 / page_size or more) get slot -1.  Outputs overlap neither each other nor
 * inputs (ctx_lens is not updated in place).  Sums of lengths must stay below
 * 2^31.  Limits: R < 2^24; width * page_size < 2^31.
 */
km_status kmeans_kv_tables(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* pos_offset, int64_t R,
                           int64_t page_size, int32_t* block_table, int64_t width, int64_t table_stride,
                           const int32_t* free_pages, int64_t num_free, int64_t T, int32_t* seq_lens,
                           int32_t* query_start, int32_t* page_start, int32_t* positions, int32_t* slots,
                           void* stream);

/*
 * kmeans_kv_append -- RMS norm of each head's query and key, rotation by
 * position, and the write of keys and values into the cache, in one pass.
 *   y = x / sqrt(mean(x^2) + eps) * weight        (if the weight is given)
 *   (a, b) -> (a cos - b sin, b cos + a sin)      (if rope is given)
 * for the pairs (i, i + rot/2), i < rot/2, or with `interleaved` the pairs
 * (2i, 2i+1); elements from rot on are not rotated.  All in fp32, rounded
 * once.  Values are copied.
 *   q, k, v    device, T tokens of q_heads / cache heads / cache heads rows of
 *              cache dim elements of type dt (KM_BF16 or KM_F16); strides of
 *              token and head are multiples of 8, pointers 16-byte aligned.
 *              q may be NULL with q_heads = 0; v may be NULL (keys only).
 *   q_weight, k_weight  device fp32[dim], 16-byte aligned, or NULL
 *   positions  device int32[T], rope device fp32[max_pos x rot]: cos in the
 *              first rot/2 columns, sin in the others (16-byte aligned, rot a
 *              multiple of 16 up to dim); both NULL with rot = 0: no rotation
 *   slots      device int32[T] or NULL (token t goes to slot t)
 *   q_out      device, as q; may be q itself (same strides)
 * A token whose slot is not in the cache or whose position is not in
 * [0, max_pos) is padding: its q_out row is zero and the cache is not written.
 * No two tokens of a call may share a slot.
 * Limits: q_heads up to 2^20; T * (q_heads + 2 * heads) <= 2^28 - 16 (beyond:
 * KM_ERR_UNSUPPORTED).
 */
km_status kmeans_kv_append(const km_kv_cache* cache, km_dtype dt, int64_t T, const void* q, int64_t q_heads,
                           int64_t q_token, int64_t q_head, const void* k, int64_t k_token, int64_t k_head,
                           const void* v, int64_t v_token, int64_t v_head, const float* q_weight,
                           const float* k_weight, float eps, const int32_t* positions, const float* rope,
                           int64_t max_pos, int64_t rot, int interleaved, const int32_t* slots, void* q_out,
                           int64_t o_token, int64_t o_head, void* stream);

/*
 * Workspace bytes of kmeans_kv_attend for T query tokens of q_heads heads in
 * R requests.  Returns 0 if the arguments are invalid.
 */
size_t kmeans_kv_attend_workspace(const km_kv_cache* cache, int64_t T, int64_t q_heads, int64_t R, int64_t max_new);

/*
 * kmeans_kv_attend -- attention of each request's new tokens over its pages.
 * Request r's queries are tokens query_start[r] .. query_start[r+1]-1, and
 * stand at slots seq_lens[r] - n .. seq_lens[r] - 1 of its cache (its last n;
 * their keys and values are in the cache already).  The query at slot p sees
 * slots j <= p, with window > 0 only those with j > p - window:
 *   s_j = scale * (q . k_j) + log_weight_j,  out = sum_j softmax(s)_j v_j,
 *   lse = log sum_j exp(s_j).
 * Query head h reads cache head h / (q_heads / heads).
 *   q, out      device, T x q_heads x dim of type dt, token and head strides
 *               multiples of 8, 16-byte aligned
 *   block_table device int32, R rows `table_stride` apart, `width` columns
 *   query_start device int32[R+1], ascending from 0; seq_lens device int32[R]
 *   log_weight  device fp32 or NULL: entry of slot o of page p and head h at
 *               p * lw_page + h * lw_head + o (16-byte aligned, strides
 *               multiples of 4); -inf removes a slot whatever it holds
 *   lse         device fp32[T x q_heads] or NULL
 *   max_new     no request has more new tokens (T always serves)
 * Slots beyond seq_lens[r] or width * page_size and slots of pages outside
 * [0, pages) are not seen.  Of a request whose tokens pass T the first ones
 * are answered, at the slots that they have among all of them.  Rows of a
 * request with more than max_new new tokens are left as they are or hold
 * anything.  A row that sees nothing is zero, its lse -inf.
 * What a row does not see never reaches it, whatever it holds (infinities and
 * NaN too).  Rows of tokens outside every request are not written.  Scores,
 * softmax and sums are fp32; the softmax terms are rounded to dt for the
 * product with the values: to 8 bits in KM_BF16; in KM_F16 to 11 bits, fewer
 * below 2^-28 and none below 2^-39 of the row's largest so far.  (So a visible
 * infinite value whose term is 0 can make its row NaN.)  Results do not depend
 * on scheduling.
 * Limits: q_heads a multiple of heads up to 2^17; T, R < 2^24; T * q_heads <
 * 2^31; width * page_size <= 2^30; (R + T * q_heads / heads / 128) * heads below
 * about 2^24 (beyond: KM_ERR_UNSUPPORTED).
 */
km_status kmeans_kv_attend(const km_kv_cache* cache, km_dtype dt, const void* q, int64_t T, int64_t q_heads,
                           int64_t q_token, int64_t q_head, const int32_t* block_table, int64_t R, int64_t width,
                           int64_t table_stride, const int32_t* query_start, const int32_t* seq_lens,
                           const float* log_weight, int64_t lw_page, int64_t lw_head, float scale, int64_t window,
                           int64_t max_new, void* out, int64_t o_token, int64_t o_head, float* lse, void* ws,
                           size_t ws_bytes, void* stream);

/* Message describing the last failed kmeans_kv_* call on this thread ("" if none). */
const char* kmeans_kv_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MEANS_CLUSTERING_AMD_KMEANS_CACHE_H */
