/*
 * gqa_rotary.h -- C ABI of the rotary positions of queries and keys (GB300, sm_103a).  Part of
 * libmoe_gb300.so; shares its status codes with moe.h.
 *
 * The token at position p has the pairs of its query and key heads turned by angles that grow with p, so that
 * scores depend on distances alone.  Pair i of a head, i = 0 .. rot_dim / 2 - 1, is
 *     (x[i], x[i + rot_dim / 2])   GQA_ROTARY_HALF
 *     (x[2 i], x[2 i + 1])         GQA_ROTARY_INTERLEAVED
 * and (a, b) becomes amplitude * (a cos - b sin, a sin + b cos) of the angle p * w[i].  Dims at and past rot_dim
 * are copied.  The calls stand between gqa_paged_plan (gqa_paged.h), which gives the positions, and the append and
 * attention of a cache of either kind; the heads of gqa_decode_attention may be turned by them as well.
 *
 * Frequencies.  w[i] = base^(-2 i / rot_dim) radians a position, changed for contexts longer than a model was
 * trained at by one of
 *     GQA_ROTARY_PLAIN      nothing
 *     GQA_ROTARY_LINEAR     w / factor
 *     GQA_ROTARY_BASE       base * factor^(rot_dim / (rot_dim - 2)) in place of base: the lowest frequency becomes
 *                           that of GQA_ROTARY_LINEAR, the highest stays
 *     GQA_ROTARY_BY_PARTS   g w + (1 - g) w / factor with g = clamp((n - low) / (high - low), 0, 1), n = original
 *                           w / (2 pi): pairs that turn `high` times or more over the original length stay, those
 *                           that turn `low` times or less become those of GQA_ROTARY_LINEAR
 * gqa_rotary_table writes them as turns a position in 64-bit fixed point, a whole turn being 2^64: position times
 * frequency then wraps by itself, exactly, at every whole turn, however far the position, and what is left of a
 * turn goes to fp32 (off by at most 2^-23 radians beside p * 2^-54 of a turn from the table's own rounding).
 */
#ifndef GQA_ROTARY_GB300_H_
#define GQA_ROTARY_GB300_H_

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GQA_ROTARY_HALF 0
#define GQA_ROTARY_INTERLEAVED 1

#define GQA_ROTARY_PLAIN 0
#define GQA_ROTARY_LINEAR 1
#define GQA_ROTARY_BASE 2
#define GQA_ROTARY_BY_PARTS 3

/* rot_dim as in gqa_rotary_dims; base >= 1; factor >= 1 (1 for GQA_ROTARY_PLAIN); original > 0 and high > low >= 0
 * are used, and looked at, with GQA_ROTARY_BY_PARTS alone. */
typedef struct gqa_rotary_scaling {
  int32_t rot_dim, kind;
  double base, factor, original, low, high;
} gqa_rotary_scaling;

/* Frequencies into turns[0 .. rot_dim / 2 - 1], on the host, in host memory (copied once to the GPU by the caller).
 * Returns MOE_ERR_INVALID_ARG for a null pointer or a value outside its meaning, MOE_ERR_UNSUPPORTED for rot_dim
 * past 256 or GQA_ROTARY_BASE with rot_dim 2. */
moe_status gqa_rotary_table(const gqa_rotary_scaling* scaling, uint64_t* turns);

/* Shapes.  Strides are in elements, from one token to the next; 0 stands for the packed value.
 *   n_heads, n_kv_heads   heads of q and of k; one of them may be 0 (its pointers are then not used); (n_heads +
 *                n_kv_heads) * head_dim <= 2^26
 *   head_dim     a multiple of 8, at most 256
 *   rot_dim      even, 2 .. head_dim
 *   n_tokens     T, rows of q, k and positions; T * (n_heads + n_kv_heads) < 2^31
 *   pairs        GQA_ROTARY_HALF or GQA_ROTARY_INTERLEAVED
 *   dtype        GQA_PAGED_BF16 (0) or GQA_PAGED_FP16 (1)
 *   amplitude    finite
 *   q_stride, k_stride, q_out_stride, k_out_stride   multiples of 8, at least heads * head_dim, below 2^39 */
typedef struct gqa_rotary_dims {
  int32_t n_heads, n_kv_heads, head_dim, rot_dim;
  int32_t n_tokens, pairs, dtype;
  float amplitude;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
} gqa_rotary_dims;

/*   q, k              [T, heads, head_dim] with their token strides, 16-byte aligned
 *   positions         int32 [T], any numbers (negative ones turn the other way)
 *   turns             [rot_dim / 2], as gqa_rotary_table writes them (16-byte aligned)
 *   n_rows            int32 [1] or NULL: rows at or past it are not written, and what they hold has no effect (q_start +
 *                     n_seqs of a plan); NULL: all T
 *   q_out, k_out      [T, heads, head_dim]; may be q and k themselves with the same strides.  An output may not
 *                     overlap an input or the other output in any other way
 * Sums are fp32, rounded once to the 16-bit type.  Device pointers, streams and statuses as in gqa_paged.h; no
 * workspace.  n_tokens == 0 is a no-op.  One launch. */
moe_status gqa_rotary(const gqa_rotary_dims* dims, const uint16_t* q, const uint16_t* k, const int32_t* positions,
                      const uint64_t* turns, const int32_t* n_rows, uint16_t* q_out, uint16_t* k_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_ROTARY_GB300_H_ */
