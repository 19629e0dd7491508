/*
 * sdpa_cache.h -- C ABI of the bounded decode cache: a key/value cache held in 4 bits, the attention
 * that reads it, and eviction of the rows that the attention weighs least.
 *
 * The decode paths of sdpa.h stream a bf16 cache that only grows.  These entry points bound it twice:
 * a 4-bit row takes 9/32 of a bf16 row's bytes per channel, and eviction bounds the number of rows.
 * A serving loop runs sdpa_fwd on the prompt, sdpa_fwd_acc for the prompt's weights, sdpa_evict,
 * sdpa_kv4_append, then per token sdpa_kv4_append and sdpa_decode_kv4 (which keeps the weights up to
 * date), with sdpa_kv4_evict whenever the cache is full.  Before the next prompt, sdpa_kv4_load gives
 * the rows back as bf16 for sdpa_fwd.
 *
 * Conventions of sdpa.h hold: contiguous row-major caller-owned device memory, 16-byte aligned where
 * not said otherwise, asynchronous on `stream`, nothing allocated, argument checks before any launch,
 * device-side problems in the device error word (a length outside its range is clamped and recorded
 * as SDPA_ERR_DEVICE_BAD_LENGTH), batch == 0 or heads == 0 -> SDPA_OK and nothing is written.  d is 64 or 128,
 * else SDPA_ERR_UNSUPPORTED.  Unlike sdpa_decode, lengths may be 0 here (an empty slot of a padded batch).
 * int32 and float arrays (lengths, LSE, weights, kept rows) need 4-byte alignment only.
 * batch * heads * rows of every array is at most 2^31 - 8192, batch and heads are at most 65535.
 * Values may be of any finite size as long as scores, scale q . k, and for bf16 caches q . k itself are finite in 32 bits (scores
 * times log2 e).  A key whose score is -inf weighs 0; a NaN or +inf score makes its query NaN.  In the 4-bit decode, elements of q
 * below 2^-27 times their head's largest lose bits, and values are exact to bf16 beside rows up to 2^100 times as large.
 *
 * The 4-bit row.  The d channels form NG = d / 32 groups of 32.  Group g has a scale s and a minimum m,
 * both bf16, and a code c in 0 .. 15 for each channel, which stands for the number s c + m.
 *   scales [batch, heads, n_kv_cap, NG, 2] bf16: s, then m
 *   codes  [batch, heads, n_kv_cap, d / 2] bytes: byte 2 (r NG + g) + e (r in 0 .. 7, e in 0 .. 1)
 *          holds channel 32 g + 4 r + 2 e in its low four bits and the next channel in its high four
 * (a tensor-core lane finds its channels of every group side by side in this order).
 */
#ifndef SDPA_B200_CACHE_H
#define SDPA_B200_CACHE_H

#include "sdpa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * sdpa_kv4_append -- quantise new rows into the cache.
 *
 * K, V [batch, heads, n_rows, d] bf16.  Row t of sequence b becomes cache row kv_lens[b] + t, for
 * t < n_new[b] (n_new NULL: all n_rows); kv_lens, n_new: int32 [batch] in device memory, 0 <= kv_lens[b],
 * 0 <= n_new[b] <= n_rows, kv_lens[b] + n_new[b] <= n_kv_cap (rows past the capacity are not written
 * and SDPA_ERR_DEVICE_BAD_LENGTH is recorded).  The lengths are not changed; other cache rows are
 * left as they were.  Weights kept beside the cache are not touched: before rows are written where others were (a slot
 * that starts again at length 0), zero the weights there (an eviction zeroes them past the rows that it keeps).
 * Per group: m = the smallest value, s = the smallest bf16 number not below (largest - m) / 15, and
 * c = (x - m) / s rounded to the nearest whole number, halves to the even one, from the exact quotient
 * (c = 0 where s = 0), so |x - (s c + m)| <= s / 2.  A group with a NaN or an infinity gets
 * s = m = NaN and reads back as NaN.
 * k_read, v_read [batch, heads, n_rows, d] bf16, or both NULL: the values the cache now stands for,
 * s c + m rounded to bf16, for the attention of the rows' own step (rows t >= n_new[b] are left as
 * they were).  They may not overlap K, V or each other (SDPA_ERR_INVALID_ARG).
 */
SDPA_API int sdpa_kv4_append(const void* K, const void* V, const int* kv_lens, const int* n_new, void* k_codes,
                             void* k_scales, void* v_codes, void* v_scales, void* k_read, void* v_read, int batch,
                             int heads, int n_rows, int n_kv_cap, int d, void* stream);

/*
 * sdpa_kv4_load -- cache rows 0 .. min(kv_lens[b], n_rows) - 1 as bf16 (s c + m rounded to nearest even)
 * into K, V [batch, heads, n_rows, d]; other rows of K and V are left as they were.
 * 0 <= kv_lens[b] <= n_kv_cap.
 */
SDPA_API int sdpa_kv4_load(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                           const int* kv_lens, void* K, void* V, int batch, int heads, int n_rows, int n_kv_cap,
                           int d, void* stream);

/*
 * sdpa_decode_kv4 -- sdpa_decode_gqa over a 4-bit cache, optionally keeping the attention weights.
 *
 * Q [batch, heads_q, d], O [batch, heads_q, d] bf16; LSE [batch, heads_q] float or NULL.  Query head h reads
 * key/value head h / (heads_q / heads_kv).  Sequence b attends to cache rows 0 .. kv_lens[b] - 1
 * (0 <= kv_lens[b] <= n_kv_cap); other rows are never used.  kv_lens[b] == 0, or all scores -inf: O = 0, LSE = -inf,
 * weights 0.
 * Keys and values enter as the numbers s c + m they stand for (not rounded to bf16 first).
 * acc_out [batch, heads_kv, n_kv_cap] float or NULL:
 *     acc_out[b, g, j] = acc[b, g, j] + sum over the query heads h of group g of exp(scale q_h . k_j - LSE_h)
 * for j < kv_lens[b]; entries at or past kv_lens[b] are left as they were.  acc may be acc_out (the usual
 * running sum) or NULL (zeros); acc without acc_out, or overlapping it in part, is SDPA_ERR_INVALID_ARG.
 * workspace: sdpa_decode_kv4_workspace_size bytes (with_acc: whether acc_out is given), scratch: a few MB, and with weights 4
 * bytes for every query head and row of capacity (n_kv_cap, not the lengths: at d = 128 a cache row pair is 160 bytes, its group's
 * scores 32 for 8 query heads).  Calls that may run at the same time (other streams, graphs replayed side by side) need
 * one each.
 */
SDPA_API size_t sdpa_decode_kv4_workspace_size(int batch, int heads_q, int heads_kv, int n_kv_cap, int d, int with_acc);
SDPA_API int sdpa_decode_kv4(const void* Q, const void* k_codes, const void* k_scales, const void* v_codes,
                             const void* v_scales, const int* kv_lens, void* O, float* LSE, const float* acc,
                             float* acc_out, int batch, int heads_q, int heads_kv, int n_kv_cap, int d, float scale,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * sdpa_decode_acc -- sdpa_decode_gqa over a bf16 cache K, V [batch, heads_kv, n_kv_cap, d] that also keeps the
 * attention weights; acc and acc_out (required) as in sdpa_decode_kv4, lengths from 0.
 */
SDPA_API size_t sdpa_decode_acc_workspace_size(int batch, int heads_q, int heads_kv, int n_kv_cap, int d);
SDPA_API int sdpa_decode_acc(const void* Q, const void* K, const void* V, const int* kv_lens, void* O, float* LSE,
                             const float* acc, float* acc_out, int batch, int heads_q, int heads_kv, int n_kv_cap,
                             int d, float scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * sdpa_fwd_acc -- the attention weights of a prompt, summed over its queries:
 *     acc_out[b, g, j] = acc[b, g, j] + sum over the heads h of group g and the queries i that see key j of
 *                        exp(scale q_hi . k_j - LSE_hi)
 * for j < n_kv.  Q [batch, heads_q, n_q, d], K [batch, heads_kv, n_kv, d] bf16; LSE [batch, heads_q, n_q] as
 * sdpa_fwd wrote it for the same scale and mask (a query with LSE = -inf or +inf adds nothing where its scores are below
 * +inf; a weight is as exact as the LSE's rounding, 2^-24 of it, allows).  causal is
 * bottom-right aligned, so the last n_q queries of a longer prompt may be given alone.  acc, acc_out
 * [batch, heads_kv, n_acc], n_acc >= n_kv (the decode cache's capacity); entries at or past n_kv are left
 * as they were; acc may be acc_out (not overlap it in part) or NULL (zeros).  n_q == 0 copies acc.
 */
SDPA_API int sdpa_fwd_acc(const void* Q, const void* K, const float* LSE, const float* acc, float* acc_out, int batch,
                          int heads_q, int heads_kv, int n_q, int n_kv, int n_acc, int d, float scale, int causal,
                          void* stream);

/*
 * sdpa_evict, sdpa_kv4_evict -- keep the rows that attention weighs most, drop the others.
 *
 * Per (sequence, head): of the kv_lens[b] rows, new_lens[b] = min(kv_lens[b], budget) are kept: the last
 * min(recent, new_lens[b]) rows, and of the rows before them those with the largest acc (of equal ones the
 * lower row; NaN counts as lower than every number).  Kept rows keep their order and become rows
 * 0 .. new_lens[b] - 1 of the output cache (capacity n_out_cap); its other rows are left as they were.
 * keep [batch, heads, budget] int32: the old row of each kept one, -1 past new_lens[b].
 * acc [batch, heads, n_kv_cap]; acc_out [batch, heads, n_out_cap]: the kept rows' weights, 0 past
 * new_lens[b] (rows appended later start at 0).
 * Every output array (acc_out included) is either its input (in place; then n_out_cap == n_kv_cap) or does
 * not overlap any input.  1 <= budget <= n_out_cap, 0 <= recent <= budget, 0 <= kv_lens[b] <= n_kv_cap;
 * keep and new_lens overlap no other array.
 */
SDPA_API int sdpa_evict(const void* K, const void* V, const float* acc, const int* kv_lens, void* K_out, void* V_out,
                        float* acc_out, int* keep, int* new_lens, int batch, int heads, int n_kv_cap, int n_out_cap,
                        int d, int budget, int recent, void* stream);
SDPA_API int sdpa_kv4_evict(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                            const float* acc, const int* kv_lens, void* k_codes_out, void* k_scales_out,
                            void* v_codes_out, void* v_scales_out, float* acc_out, int* keep, int* new_lens,
                            int batch, int heads, int n_kv_cap, int n_out_cap, int d, int budget, int recent,
                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SDPA_B200_CACHE_H */
