/*
 * kmeans_cache_forms.h -- further forms of the paged key/value cache of
 * kmeans_cache.h, on one MI355X (gfx950): a cache in 8 bits, rotation by
 * several position axes, and attention whose scores are capped or fall with
 * distance or whose queries all see a prefix (libkm_cache_forms.so).
 *
 * The page "Flash-KMeans: Fast and Memory-Efficient Exact K-Means" (gist.science
 * summary of paper 2603.09229) names key/value-cache compression and longer
 * contexts as users of K-Means (tech §1, §5); it describes no cache.  The rules
 * below are this library's.
 *
 * Conventions, the cache's layout and the checks on the device are those of
 * kmeans_cache.h; kmeans_kv_form_last_error() describes the last failure of
 * the calling thread.  Calls can be captured in a HIP graph.
 *
 * An 8-bit cache.  km_kv_cache describes it with codes in place of 16-bit
 * elements: e4m3 (finite up to 448, NaN 0x7f and 0xff, no infinities), one
 * byte each; k and v 16-byte aligned, strides multiples of 16.  A block is 16
 * slots of a page, from slot 16 b on, of one head; its byte s stands for the
 * scale 2^(s - 127) (255: NaN), and a code c for the value c * 2^(s - 127).
 * The attention and kmeans_kv_read take that value rounded to their 16-bit type
 * (exact in KM_BF16 but for values below 2^-126; in KM_F16 with its range).
 */
#ifndef MEANS_CLUSTERING_AMD_KMEANS_CACHE_FORMS_H
#define MEANS_CLUSTERING_AMD_KMEANS_CACHE_FORMS_H

#include "kmeans_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Scales of an 8-bit cache: the byte of block b of page p and head h is at
 * p * page + h * head + b.  k and v are different arrays; head strides at
 * least page_size / 16, page strides at least (heads - 1) * head stride +
 * page_size / 16, both below 2^40.
 */
typedef struct km_kv_scales {
  uint8_t* k;
  uint8_t* v;
  int64_t k_page, k_head, v_page, v_head;
} km_kv_scales;

/*
 * Rotation by position.  rope: device fp32[max_pos x rot], cos in the first
 * rot / 2 columns, sin in the others (16-byte aligned, rot a multiple of 16 from
 * 16 to the cache's dim).  positions: device int32, `axes` rows (1 to 4) of T,
 * `axis_stride` apart.  Pair i turns by the position on axis[i] (device
 * uint8[rot / 2], 8-byte aligned; NULL: axis 0); a pair whose axis is not below
 * `axes` is not turned.  Pairs are (i, i + rot / 2), or with `interleaved`
 * (2 i, 2 i + 1).
 */
typedef struct km_kv_turn {
  const float* rope;
  int64_t max_pos, rot;
  int interleaved;
  const int32_t* positions;
  int64_t axes, axis_stride;
  const uint8_t* axis;
} km_kv_turn;

/*
 * kmeans_kv_append_form -- kmeans_kv_append with the rotation of `turn` (NULL:
 * none), into a 16-bit cache (scales NULL) or an 8-bit one.  A token one of
 * whose positions is outside [0, max_pos) is padding.  q_out is of type dt.
 *   An 8-bit cache.  For each block that the call's tokens fall into, with A
 * the largest finite magnitude that they bring (keys normed and rotated, fp32)
 * and need the least exponent >= -126 with A <= 448 * 2^need:
 *   - where the block's first slot is among theirs the block begins anew: its
 *     scale is 2^need, and what its other slots held is gone;
 *   - otherwise the scale becomes the larger of its own and 2^need, and the
 *     codes of the block's other slots are brought to it, rounded to nearest.
 * New codes are rounded to nearest, ties to even; infinities become NaN.
 * (Scale bytes of 0 and 255 count as 1 and 254 here.)
 * The tokens of a block must stand within 15 places of one another in the call
 * (the tables of kmeans_kv_tables put them side by side); no two share a slot.
 * Nothing looks for others: the block that they share, no more, then holds
 * anything.
 * Without v values and their scales are not touched (scales->v may be NULL).
 * Limits as kmeans_kv_append.  With an 8-bit cache T * heads <= 2^26 - 4, k and v
 * are different arrays, and pages, slots and heads must not overlap: in the order
 * of their strides, each of which there are several steps over all of the smaller
 * ones.
 */
km_status kmeans_kv_append_form(const km_kv_cache* cache, const km_kv_scales* scales, km_dtype dt, int64_t T,
                                const void* q, int64_t q_heads, int64_t q_token, int64_t q_head, const void* k,
                                int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                                const float* q_weight, const float* k_weight, float eps, const km_kv_turn* turn,
                                const int32_t* slots, void* q_out, int64_t o_token, int64_t o_head, void* stream);

/*
 * kmeans_kv_read -- the values of n slots of an 8-bit cache, for all heads.
 *   slots      device int32[n], or NULL: slots 0 .. n-1.  A slot that is not in
 *              the cache gives zeros.
 *   k, v       device, n x heads x dim of type dt, strides of row and head
 *              multiples of 8, 16-byte aligned; either may be NULL (not read)
 * Limits: n * heads <= 2^28 - 16.
 */
km_status kmeans_kv_read(const km_kv_cache* cache, const km_kv_scales* scales, km_dtype dt, const int32_t* slots,
                         int64_t n, void* k, int64_t k_row, int64_t k_head, void* v, int64_t v_row, int64_t v_head,
                         void* stream);

/*
 * The scores of an attention.  A query at slot p and a key at slot j, with
 * x = scale * (q . k_j):
 *   s = cap * tanh(x / cap) (cap > 0; else x) + log_weight_j - slope_h * |p - j|
 * (a distance in fp32: beyond 2^24 slots rounded to 24 bits; a score that
 * overflows to -inf counts as one that is not seen).
 * Distances and windows count slots, whatever a slot stands for.
 * slopes: device fp32[q_heads] or NULL.  The query sees slot j of its request
 * (below seq_lens[r]) if j < prefix[r] (device int32[R] or NULL; wherever the
 * query stands), or if j <= p and, with window > 0, j > p - window.  So a prefix
 * is a part of the prompt whose tokens see one another, or with a window the
 * slots (sinks, centroids) that stay in sight.
 * Limits: cap 0 (none) or positive and finite, scale and cap finite times
 * log2(e) without weights, scale / cap finite times 2 log2(e) and 0 or at least
 * 2^-126.
 */
typedef struct km_kv_scores {
  float scale;
  int64_t window;
  float cap;
  const float* slopes;
  const int32_t* prefix;
} km_kv_scores;

/*
 * Workspace bytes of kmeans_kv_attend_form (scales NULL: a 16-bit cache).
 * Returns 0 if the arguments are invalid.
 */
size_t kmeans_kv_attend_form_workspace(const km_kv_cache* cache, const km_kv_scales* scales, int64_t T,
                                       int64_t q_heads, int64_t R, int64_t max_new);

/*
 * kmeans_kv_attend_form -- kmeans_kv_attend with these scores, over a 16-bit
 * cache (scales NULL) or an 8-bit one with queries and results of type dt.
 * Everything else is as there: rows that see nothing are zero with an lse of
 * -inf, slots of weight -inf are removed whatever they hold, and what a row
 * does not see never reaches it.
 */
km_status kmeans_kv_attend_form(const km_kv_cache* cache, const km_kv_scales* scales, km_dtype dt, const void* q,
                                int64_t T, int64_t q_heads, int64_t q_token, int64_t q_head,
                                const int32_t* block_table, int64_t R, int64_t width, int64_t table_stride,
                                const int32_t* query_start, const int32_t* seq_lens, const float* log_weight,
                                int64_t lw_page, int64_t lw_head, const km_kv_scores* scores, int64_t max_new,
                                void* out, int64_t o_token, int64_t o_head, float* lse, void* ws, size_t ws_bytes,
                                void* stream);

/* Message describing the last failed call of this header on this thread ("" if none). */
const char* kmeans_kv_form_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MEANS_CLUSTERING_AMD_KMEANS_CACHE_FORMS_H */
