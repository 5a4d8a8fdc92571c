/*
 * gqa_paged.h -- C ABI of the paged key/value cache for batches of sequences and of the grouped-query
 * attention that reads it (GB300, sm_103a).  Part of libmoe_gb300.so; shares its status codes and its
 * workspace error word with moe.h.
 *
 * gqa_decode_attention (gqa_attention.h) serves one sequence whose cache is one block of memory.  The
 * calls here serve the same layers (grouped-query heads, scores q . k / sqrt(D), softmax in fp32) for
 * many sequences at once, prompts in chunks and single tokens alike:
 *
 *   gqa_paged_plan       from the sequences' lengths, on the GPU: where each sequence's rows start, its
 *                        length after this step, the block table with fresh pages taken from a free
 *                        list, and each new token's position and cache slot (once per step)
 *   gqa_paged_append     new keys and values into their slots (once per layer)
 *   gqa_paged_attention  the new tokens' attention over the cache (once per layer)
 *
 * The cache is a pool of pages of page_size positions; position p of sequence b lives in page
 * block_table[b][p / page_size], at offset p % page_size, and its slot is
 * block_table[b][p / page_size] * page_size + p % page_size.
 *
 * Attention.  Sequence b has n = q_start[b+1] - q_start[b] new tokens (rows q_start[b] .. q_start[b+1]-1
 * of q and o) at positions kv_len[b] - n .. kv_len[b] - 1, their keys and values already in the cache.
 * The token at position p sees position j if
 *     j <= p   and   (window == 0  or  j > p - window  or  j < sinks),
 * that is, every earlier position, or the last `window` ones and the first `sinks` ones.  For query
 * head h with g = h / (Hq / Hkv):
 *     o[t, h, :] = sum_j softmax_j(q[t, h, :] . K[g, j, :] / sqrt(D)) V[g, j, :]  over the visible j.
 * A row that sees nothing (kv_len[b] < n puts rows before position 0) gets zeros.  What lies in the
 * cache at positions that a row does not see has no effect on it, non-finite values included.  Block-
 * table entries of pages that no row sees are not read, so a window's passed pages may be freed.
 * Sums and softmax statistics are fp32; o is rounded once to the 16-bit type.  In the chunk form the
 * softmax's numerators are rounded to the 16-bit type before the product with V (the tensor cores'
 * operand type: at most half a step each, relative to the numerator, or in fp16 2^-34 relative to the row's
 * largest one); the single-token form keeps their rounding remainders (fp16: 2^-40).  The form follows
 * max_new, so a sequence with one new token in a call that has room for more is rounded as a chunk.
 * Identical calls give identical results; the work of a whole call is cut and joined by one rule, so the
 * last bits of a sequence's outputs may differ with what else is in the call.
 *
 * Conventions are those of moe.h: device pointers owned by the caller, 16-byte aligned (the int32 arrays
 * 4-byte aligned, so they may be slices); work is
 * enqueued on `stream` (a cudaStream_t, NULL = legacy default stream) of the current device; argument
 * checks on the host before any launch; inputs never written, except that gqa_paged_plan's block
 * table is updated in place and n_free_out may be n_free.  Scratch and the error word live in the
 * caller's workspace (clear its first 4 bytes once with moe_clear_error_flags; read them with
 * moe_read_error_flags); calls that may run at the same time need workspaces of their own.  Bits these
 * calls may set: 1 (a bounded wait timed out; o invalid), 8 (an output is not finite, which only
 * non-finite visible inputs, scores past fp32's range or bf16 values of 2^84 and more cause) and 16 (a
 * length, page or slot out of range; what each call does then stands with it: no call reads or writes
 * out of bounds).
 */
#ifndef GQA_PAGED_GB300_H_
#define GQA_PAGED_GB300_H_

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GQA_PAGED_BF16 0
#define GQA_PAGED_FP16 1

/* Shapes of the calls.  Strides are in elements; 0 stands for the packed value given with each.
 *   n_heads, n_kv_heads, head_dim   Hq, Hkv, D: Hq % Hkv == 0, Hq / Hkv <= 8, D = 64 or 128
 *   page_size    positions per page: 16, 32, 64 or 128
 *   num_pages    pages of the pool, num_pages * page_size * Hkv < 2^31
 *   max_pages    entries of a block-table row, max_pages * page_size <= 2^30
 *   n_seqs       B, sequences, 0 .. 4096
 *   n_tokens     T, rows of q, k, v, o, positions and slots, T * Hq < 2^31.  May exceed the sum of the
 *                new tokens: the rows behind the last sequence are neither used nor written
 *   max_new      bound on the new tokens of any one sequence; 0 stands for n_tokens.  1 selects the
 *                single-token form of the attention
 *   window       0 (all earlier positions) or the number of latest positions a token sees, itself among
 *                them
 *   sinks        leading positions that stay visible beyond the window
 *   dtype        GQA_PAGED_BF16 or GQA_PAGED_FP16: type of q, k, v, the caches and o
 *   q_stride, o_stride, k_stride, v_stride   from one token to the next (packed: Hq * D, Hq * D,
 *                Hkv * D, Hkv * D); heads are D apart
 *   page_stride, head_stride, row_stride     of both caches, from page to page, key/value head to head,
 *                and position to position (packed: Hkv * page_size * D, page_size * D, D)
 * Strides are multiples of 8 elements (16 bytes), at least the extent they step over (for the cache's:
 * at least D, and no two elements at one address), below 2^39 elements. */
typedef struct gqa_paged_dims {
  int32_t n_heads, n_kv_heads, head_dim;
  int32_t page_size, num_pages, max_pages;
  int32_t n_seqs, n_tokens, max_new;
  int32_t window, sinks;
  int32_t dtype;
  int64_t q_stride, o_stride, k_stride, v_stride;
  int64_t page_stride, head_stride, row_stride;
} gqa_paged_dims;

/* Workspace bytes for these dims (one workspace serves all three calls).  0 for invalid dims. */
size_t gqa_paged_workspace_bytes(const gqa_paged_dims* dims);

/* Tables of one step.  All arrays int32.
 *   ctx_len      [B]             positions that each sequence has in the cache
 *   new_len      [B]             positions that this step adds, 0 allowed
 *   free_pages   [free_capacity] free pages; the first *n_free of them are valid (may be NULL if
 *                                free_capacity is 0)
 *   n_free       [1]             0 .. free_capacity
 *   block_table  [B, max_pages]  entries of held pages are kept; fresh ones are written
 *   q_start      [B + 1]         out: first row of each sequence; q_start[B] rows are in use
 *   kv_len       [B]             out: ctx_len + new_len
 *   positions    [T] or NULL     out: position of each new token in its sequence
 *   slots        [T]             out: cache slot of each new token (may be NULL if T is 0)
 *   n_free_out   [1]             out: *n_free less the pages taken; may be n_free itself
 * Sequence b holds ceil(ctx_len / page_size) pages and needs ceil(kv_len / page_size).  The fresh ones
 * are taken from the end of the free list: in order of (sequence, page), the m-th is
 * free_pages[*n_free - 1 - m].  Everything else in block_table, positions and slots (rows at or past
 * q_start[B]) is left as it was.
 * Bit 16 is set for: a negative length (taken as 0); lengths whose sum passes T (the rows past T have
 * no entries, q_start is cut at T) or a row of the block table (kv_len is cut at max_pages * page_size,
 * the slots past it are -1); *n_free outside its range (cut); a free list that runs out (the entries and
 * slots become -1), or that holds, or a held page that is, a number outside 0 .. num_pages - 1 (likewise).
 * Returns as gqa_paged_attention, and MOE_ERR_INVALID_ARG if an output overlaps an input or another output
 * (but n_free_out == n_free); n_seqs == 0 is a no-op.  One launch. */
moe_status gqa_paged_plan(const gqa_paged_dims* dims, const int32_t* ctx_len, const int32_t* new_len,
                          const int32_t* free_pages, int32_t free_capacity, const int32_t* n_free,
                          int32_t* block_table, int32_t* q_start, int32_t* kv_len, int32_t* positions, int32_t* slots,
                          int32_t* n_free_out, void* workspace, size_t workspace_bytes, void* stream);

/* Keys and values of the new tokens into their slots.
 *   k, v              [T, Hkv, D] with their token strides
 *   slots             int32 [T]
 *   q_start           int32 [B + 1]: rows at or past q_start[B] are skipped
 *   k_cache, v_cache  [num_pages, Hkv, page_size, D] with the strides of dims
 * A slot of -1 is skipped; any other slot outside 0 .. num_pages * page_size - 1 is skipped and sets bit
 * 16.  Two rows must not have the same slot (one of them would be stored, mixed 16 bytes by 16 bytes).
 * Returns as gqa_paged_attention; n_tokens == 0 or n_seqs == 0 is a no-op.  One launch. */
moe_status gqa_paged_append(const gqa_paged_dims* dims, const uint16_t* k, const uint16_t* v, const int32_t* slots,
                            const int32_t* q_start, uint16_t* k_cache, uint16_t* v_cache, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Attention of the new tokens over the cache.
 *   q                 [T, Hq, D] with its token stride
 *   k_cache, v_cache  [num_pages, Hkv, page_size, D] with the strides of dims
 *   block_table       int32 [B, max_pages]
 *   q_start           int32 [B + 1], kv_len int32 [B]: as gqa_paged_plan writes them
 *   o                 [T, Hq, D] with its token stride
 *   workspace         >= gqa_paged_workspace_bytes(dims)
 * Bit 16 is set for: rows of a sequence outside 0 .. T or falling (the sequence is skipped; sequences
 * that claim the same rows leave either's results there), kv_len outside 0 .. max_pages * page_size
 * (cut), more than max_new rows of a sequence (the first max_new are computed), a page number outside
 * 0 .. num_pages - 1 (its keys and values count as zeros), and work of 2^32 or more cache tiles over all
 * sequences and heads (128 positions for a block of query rows, 64 in the single-token form: nothing is
 * computed).
 * Returns MOE_ERR_INVALID_ARG for a null pointer or a value of dims outside its meaning;
 * MOE_ERR_UNSUPPORTED for values outside the limits of dims; MOE_ERR_MISALIGNED for a pointer off
 * its alignment or a stride that is not a multiple of 8; MOE_ERR_WORKSPACE; MOE_ERR_CUDA as in
 * moe.h.  n_tokens == 0 or n_seqs == 0 is a no-op. */
moe_status gqa_paged_attention(const gqa_paged_dims* dims, const uint16_t* q, const uint16_t* k_cache,
                               const uint16_t* v_cache, const int32_t* block_table, const int32_t* q_start,
                               const int32_t* kv_len, uint16_t* o, void* workspace, size_t workspace_bytes,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_PAGED_GB300_H_ */
