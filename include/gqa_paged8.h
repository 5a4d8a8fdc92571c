/*
 * gqa_paged8.h -- C ABI of the paged key/value cache held in 8 bits: the calls of gqa_paged.h for a cache of half
 * the size (GB300, sm_103a).  Part of libmoe_gb300.so; shares its status codes and its workspace error word with
 * moe.h, and its shapes (gqa_paged_dims) and its plan (gqa_paged_plan) with gqa_paged.h.
 *
 *   gqa_paged8_append     new keys and values, quantised, into the cache (once per layer)
 *   gqa_paged8_attention  the new tokens' attention over the cache (once per layer)
 *   gqa_paged8_read       cached keys and values back in 16 bits
 *
 * The cache.  Position p of sequence b lives in page block_table[b][p / page_size] at offset p % page_size, as in
 * gqa_paged.h.  A key or value is an 8-bit code (e4m3: a sign, four bits of exponent, three of mantissa, largest 448,
 * no infinities, NaN 0x7F and 0xFF) times the fp32 scale of its block, the 16 positions p / 16 * 16 .. p / 16 * 16 + 15
 * of one key/value head:
 *     k_cache, v_cache  uint8 [num_pages, Hkv, page_size, D] with the strides of dims (elements are bytes here)
 *     k_scale, v_scale  fp32 [num_pages, Hkv, page_size / 16], packed
 * A scale is a power of two from 2^-60 to 2^60, as gqa_paged8_append writes it.  Any other number in the place of a
 * scale that a call needs counts as 2^-60 and sets bit 16.
 *
 * Rows.  In all three calls sequence b's rows are q_start[b] .. q_start[b+1] - 1 and stand for its positions
 * kv_len[b] - n .. kv_len[b] - 1, n = q_start[b+1] - q_start[b], as gqa_paged_plan writes them.
 *
 * Conventions, statuses, the limits of dims and the error word are those of gqa_paged.h, but: strides of the caches
 * are multiples of 16 bytes; the scales are 16-byte aligned; bit 8 is also set by gqa_paged8_append for an input that
 * is not finite (below).  Block-table entries, codes and scales of what no row needs are not read, or have no effect;
 * and as there, what a row does not see has no effect on that row (but for last bits), whatever its scales.
 */
#ifndef GQA_PAGED8_GB300_H_
#define GQA_PAGED8_GB300_H_

#include <stddef.h>
#include <stdint.h>

#include "gqa_paged.h"
#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GQA_PAGED8_BLOCK 16

/* Workspace bytes for these dims (one workspace serves the three calls and gqa_paged_plan).  0 for invalid dims. */
size_t gqa_paged8_workspace_bytes(const gqa_paged_dims* dims);

/* Keys and values of the new tokens, quantised, into their positions.
 *   k, v         [T, Hkv, D] of the dims' type with their token strides
 *   block_table  int32 [B, max_pages];  q_start int32 [B + 1];  kv_len int32 [B]
 * A block that gets positions o .. of its 16 holds what it held at offsets below o; what lay at o and past it counts
 * as never written.  Its scale becomes s = max(2^e, its scale before where o > 0), e the least number from -60 to 60
 * with |x| <= 448 * 2^e for every new x; new codes are x / s rounded to nearest even.  Where s has grown, the codes
 * below o are rounded once more, code * before / s (exact but for those that leave the type's range of 2^-9 and
 * more).  So the cache depends on how a sequence was cut into calls in these last bits, and never on what else is in
 * a call.  An x that is not finite or is past 448 * 2^60 is left out of e, its code is NaN, and it sets bit 8.
 * Codes past a sequence's last position are left as they were.  Rows before position 0 are skipped.  A sequence whose
 * pages others share must not get positions in a shared one.  A page number outside 0 .. num_pages - 1 sets bit 16,
 * and the positions in that page are skipped.  Otherwise as gqa_paged8_attention.  One launch. */
moe_status gqa_paged8_append(const gqa_paged_dims* dims, const uint16_t* k, const uint16_t* v, const int32_t* block_table,
                             const int32_t* q_start, const int32_t* kv_len, uint8_t* k_cache, uint8_t* v_cache,
                             float* k_scale, float* v_scale, void* workspace, size_t workspace_bytes, void* stream);

/* Cached keys and values of every sequence's last positions.
 *   k, v         [T, Hkv, D] of the dims' type with their token strides: code * scale, rounded once (fp16: values
 *                past 65504 become 65504); zeros in rows before position 0 and of a page number out of range (which
 *                sets bit 16)
 * window, sinks and max_new play no part but for max_new's check.  Rows of no sequence are left as they were.  k and v
 * have no element in common (one address for both is refused).  One launch. */
moe_status gqa_paged8_read(const gqa_paged_dims* dims, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                           const float* v_scale, const int32_t* block_table, const int32_t* q_start, const int32_t* kv_len,
                           uint16_t* k, uint16_t* v, void* workspace, size_t workspace_bytes, void* stream);

/* Attention of the new tokens over the cache: gqa_paged_attention with K and V the products code * scale, exact.
 * Products are fp16 on the tensor cores, with fp32 sums, and what enters them:
 *   queries     fp16 as they are; bf16 times a power of two of each row and head, off by at most 2^-39 of the row's
 *               largest number, or by 2^-105 if that is less than 2^-66 (one of 65520 * 2^60 or more counts as infinite)
 *   keys, values   exact
 *   numerators  as gqa_paged_attention states for fp16.  In single tokens, and in chunks from 128 positions on whose scales
 *               (those that some row of its block needs) differ by more than 2^15, or are that far below an earlier value
 *               scale: times their block's value scale over the largest that the token has met, and so each off by
 *               2^-40 (single tokens) or 2^-34 (chunks) of 448 times the largest value scale that the token sees
 * Bit 8 is set for an output that is not finite: visible NaN codes, or values past the dims' type.
 *   workspace  >= gqa_paged8_workspace_bytes(dims) */
moe_status gqa_paged8_attention(const gqa_paged_dims* dims, const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                const float* k_scale, const float* v_scale, const int32_t* block_table,
                                const int32_t* q_start, const int32_t* kv_len, uint16_t* o, void* workspace,
                                size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_PAGED8_GB300_H_ */
