/*
 * fp4idx_step.h -- C ABI of the operators of libfp4idx.so that a serving step
 * needs around the caches: pages and maps of a batch built on the GPU, rotary
 * positions of the main queries and keys, and attention of packed prompts over
 * their own keys in 16 bits.  One GB300 GPU (sm_103a).
 *
 * A step, and the calls that make it:
 *   pages, slots, positions       fp4idx_batch_extend
 *   main queries and keys         fp4idx_rope_qk
 *   keys and values to the cache  fp4idx_kv_store_fp8        (fp4idx_attention.h)
 *   attention of whole prompts    fp4idx_prompt_attention
 *   attention of single tokens    fp4idx_paged_attention_fp8 (fp4idx_attention.h)
 *   pages of what has ended       fp4idx_pages_release
 *
 * The conventions are those of fp4idx.h and fp4idx_attention.h: device
 * pointers, buffers owned by the caller, nothing allocated and nothing
 * synchronised by the library, host-side checks before anything is enqueued,
 * errors of the kernel at the caller's next synchronisation.  Pages hold
 * FP4IDX_KV_BLOCK = 64 tokens.  Calls keep no state: two of them may run at
 * once on different streams if they do not write the same memory.
 */
#ifndef FP4IDX_STEP_H
#define FP4IDX_STEP_H

#include "fp4idx_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A bit of *err_flags beside those of fp4idx.h. */
#define FP4IDX_ERRFLAG_FULL 0x10u /* fp4idx_batch_extend: a sequence was not
                                     served; fp4idx_pages_release: a page found
                                     no place in free_pages                    */

/*
 * The next tokens of a batch: takes the pages that they need and writes the
 * maps that the step's other calls read.  Sequence b holds old = cached_lens[b]
 * tokens and gets new_lens[b] more (0: it pauses); a negative length counts as
 * 0.  With has = ceil(old / 64), want = ceil((old + new) / 64):
 *   the pages want - has come off the top of the stack of free pages, sequence
 *   by sequence: the j-th page taken in the call is free_pages[count - 1 - j];
 *   block_table[b][has .. want-1] = those pages; *free_count falls by all taken.
 * Tokens are numbered through the batch, sequence by sequence.  Token t, the
 * i-th of sequence b, stands at position p = old + i:
 *   slot_mapping[t] = block_table[b][p / 64] * 64 + p % 64,  positions[t] = p,
 *   seq_ids[t] = b,  row_lens[t] = p + 1  (the keys it may select from);
 *   q_starts[b] = the first token of sequence b (at most num_tokens), and
 *   q_starts[batch] their number;  context_lens[b] = old + new.
 * Tokens behind the last one (a step padded to num_tokens, say for a captured
 * graph) get slot -1, position 0, sequence 0 and row length 0.
 *
 * A sequence is served if its row holds want pages, its tokens end within
 * num_tokens, and free pages are left for it and for the sequences before it
 * that meet the first two conditions (one that needs none is served without).
 * One that is not served keeps its table row and context_lens[b] = old; its
 * tokens keep seq_ids = b and get slot -1, position 0 and row length 0, and
 * FP4IDX_ERRFLAG_FULL is raised.
 *
 *   cached_lens, new_lens   int32 [batch].
 *   block_table   int32, page p of sequence b at b*block_table_stride + p,
 *                 p < block_table_pages; read at the pages that hold the
 *                 sequences' last tokens, which a slot is made of as it stands.
 *                 A page belongs to one sequence where new tokens are written.
 *   free_pages    int32, a stack of free_capacity places, the lowest first.
 *   free_count    int32 [1], the pages in it; taken within [0, free_capacity].
 *   q_starts      int32 [batch+1];  context_lens int32 [batch].
 *   slot_mapping, positions  int64 [num_tokens];  seq_ids, row_lens int32
 *                 [num_tokens].  Each of the six outputs may be NULL; none may lie
 *                 in the memory of an input or of another (the lengths of the next
 *                 step are copied from context_lens).
 * Sums of lengths stay below 2^31.  batch == 0 writes what num_tokens asks for.
 */
fp4idx_status fp4idx_batch_extend(const int32_t* cached_lens, const int32_t* new_lens,
                                  int32_t* block_table, int64_t block_table_stride,
                                  int64_t block_table_pages, const int32_t* free_pages,
                                  int32_t* free_count, int64_t free_capacity, int32_t* q_starts,
                                  int32_t* context_lens, int64_t* slot_mapping,
                                  int64_t* positions, int32_t* seq_ids, int32_t* row_lens,
                                  int64_t batch, int64_t num_tokens, uint32_t* err_flags,
                                  void* stream);

/*
 * Gives pages back: of the pages that held_lens[b] tokens of sequence b fill,
 * those behind its first kept_lens[b] tokens (0: it has ended; fewer than held:
 * rejected drafts; as many or more: nothing).  The pages go onto the stack, the
 * first one of the first sequence last, so that a call which gives back what
 * fp4idx_batch_extend has just taken restores the stack; their table entries
 * become -1, and *free_count grows by them.  A page that several sequences
 * share is the caller's to keep (by kept_lens) until the last one ends.
 *
 *   held_lens, kept_lens   int32 [batch]; negative counts as 0.  Pages behind
 *                 block_table_pages are not there; the others are in the table.
 *   err_flags     optional: FP4IDX_ERRFLAG_FULL if the stack has no place for a
 *                 page (it is dropped; *free_count stops at free_capacity).
 * The other arguments as above.  batch == 0 enqueues nothing.
 */
fp4idx_status fp4idx_pages_release(const int32_t* held_lens, const int32_t* kept_lens,
                                   int32_t* block_table, int64_t block_table_stride,
                                   int64_t block_table_pages, int32_t* free_pages,
                                   int32_t* free_count, int64_t free_capacity, int64_t batch,
                                   uint32_t* err_flags, void* stream);

/* How the pairs of a row are shared out among several position axes. */
enum {
  FP4IDX_AXES_SECTIONS = 0,   /* axis 0 turns the first sections[0] pairs, axis
                                 1 the next sections[1], ...                   */
  FP4IDX_AXES_INTERLEAVED = 1 /* pair i: axis a = i % num_axes if i / num_axes
                                 < sections[a], else axis 0                    */
};

/*
 * Rotary positions of queries and keys.  Pair i of the R / 2 pairs of a row
 * (R = rope_dim) is (i, i + R/2) for FP4IDX_ROPE_NEOX, (2i, 2i + 1) for
 * FP4IDX_ROPE_INTERLEAVED.  With a the axis of pair i and p = positions[a][t]:
 *   x' = x cos[p][i] - y sin[p][i],  y' = y cos[p][i] + x sin[p][i],
 * products and sums rounded to fp32, the result once to the type; elements
 * behind R are copied.  Angles, and with them each axis's frequencies, are the
 * tables' matter.
 *
 *   q, k          16-bit, row (t, h) at t*token_stride + h*head_stride elements,
 *                 16-byte aligned, strides multiples of 8.  k may be NULL with
 *                 k_heads 0.
 *   q_out, k_out  the same, with strides of their own; an output's heads lie within
 *                 its token stride or a head's tokens within its head stride, so that
 *                 no two rows overlap (FP4IDX_ERR_ARG).  q_out may be q with q's
 *                 strides (in place; other strides return FP4IDX_ERR_ARG), and
 *                 k_out k; any other overlap of an output with an input is the
 *                 caller's error.
 *   q_heads       at least 1; q_heads + k_heads at most 65535.
 *   head_dim      a multiple of 8, 16 .. 1024;  rope_dim a multiple of 16, at
 *                 most head_dim.
 *   positions     int64, axis a of token t at a*axis_stride + t.
 *   sections      HOST int32 [num_axes], not negative, their sum R / 2; read
 *                 within the call.  num_axes 1 .. 4.
 *   cos, sin      fp32 [max_pos, R / 2] each, dense, 16-byte aligned.
 *   num_tokens    below 2^31, and num_tokens * ceil(head_dim / 16) * ceil((q_heads +
 *                 k_heads) / 8) below 2^32 - 256, as many threads as a call has;
 *                 more return FP4IDX_ERR_SHAPE and take several calls.
 *   err_flags     optional: FP4IDX_ERRFLAG_POSITION for a token with a position
 *                 outside [0, max_pos); its rows are left as they were.
 * num_tokens == 0 returns FP4IDX_OK and enqueues nothing.
 */
fp4idx_status fp4idx_rope_qk(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                             void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                             int64_t q_heads, const void* k, int64_t k_token_stride,
                             int64_t k_head_stride, void* k_out, int64_t k_out_token_stride,
                             int64_t k_out_head_stride, int64_t k_heads, int dtype,
                             int64_t head_dim, const int64_t* positions, int64_t axis_stride,
                             const int32_t* sections, int num_axes, int axis_order,
                             const float* cos, const float* sin, int64_t max_pos,
                             int64_t rope_dim, int rope_style, int64_t num_tokens,
                             uint32_t* err_flags, void* stream);

/*
 * Attention of packed sequences over keys and values in 16 bits.  Sequence b has
 * the n_b query tokens q_starts[b] .. q_starts[b+1] - 1 and the c_b keys
 * k_starts[b] .. k_starts[b+1] - 1; its last query stands at its last key: query
 * i at position p = c_b - n_b + i, and it sees the keys
 *   s <= p, and, if window > 0, also s > p - window or s < sinks.
 * Without k_starts the sequences are whole prompts (k_starts = q_starts).  With
 * x_s = softmax_scale * sum_d q[d] k_s[d] over the keys it sees:
 *   lse = log sum_s exp(x_s),  out[d] = sum_s exp(x_s - lse) v_s[d];
 * a query that sees no key (p < 0) gets out = 0 and lse = -inf.  Query head h
 * reads key head h / (num_heads / kv_heads).
 *
 * Products are exact in the tensor core, the softmax and both sums fp32;
 * probabilities are rounded to the elements' type before the product with the
 * values: bf16 by 2^-8 of themselves (those below 2^-120 of the row's largest count
 * as 0), fp16 by 2^-11 or 2^-35 of the row's largest.  A score carries fp32's
 * relative error into its exponent, so |x_s| is to stay below 2^20.  The sum over
 * the keys of exp(x_s - max x) |v_s[d]| is to stay below 2^125, as it does for values
 * below 2^125 divided by the keys; beyond it an output may be infinite.
 *
 *   q             16-bit, row (t, h) at t*q_token_stride + h*q_head_stride
 *                 elements; 16-byte aligned, strides multiples of 8.
 *   k, v          the same, k_tokens rows and kv_heads.  A token's heads lie
 *                 within its token stride (token_stride >= (kv_heads-1) *
 *                 head_stride + head_dim) or a head's tokens within its head
 *                 stride, that a multiple of the token stride.  The product
 *                 (kv_heads-1) * head_stride stays below 2^31 in the first form.
 *   q_starts      int32 [batch+1], ascending within [0, q_tokens].  Rows of out
 *                 and lse in no sequence are left as they were.
 *   k_starts      int32 [batch+1], ascending within [0, k_tokens], or NULL.
 *   max_q         a bound on n_b, at least 1; tokens of a sequence behind its
 *                 max_q-th are left unwritten.
 *   max_k         a bound on c_b; keys behind a sequence's max_k-th are not
 *                 seen.  The work split is chosen by both bounds, so loose ones
 *                 cost time, not correctness.
 *   softmax_scale not negative.
 *   head_dim      64 or 128;  kv_heads 1 .. 65535, num_heads a multiple of it.
 *   out           16-bit [q_tokens, num_heads, head_dim], dense, 16-byte
 *                 aligned;  lse optional fp32 [q_tokens, num_heads], natural
 *                 logarithm.  Neither lies in the memory of an input (out where q,
 *                 k or v begins: FP4IDX_ERR_ARG).
 *   workspace     fp4idx_prompt_workspace_bytes(batch, max_q, num_heads,
 *                 kv_heads, head_dim) bytes (0 bytes: arguments out of range;
 *                 20 MB for heads of 64, 40 MB for heads of 128, whatever the rest),
 *                 16-byte aligned, contents not kept; its own for each call in
 *                 flight (two captured graphs that may run at once too).
 *                 Fewer bytes return FP4IDX_ERR_SCRATCH.
 *   err_flags     optional: FP4IDX_ERRFLAG_TIMEOUT if a wait inside the kernel
 *                 ran out.
 * A value that is not finite among the keys or values that one query of a
 * sequence sees may reach other queries of the sequence, but no other sequence;
 * rows of k and v in no sequence may hold anything.
 */
size_t fp4idx_prompt_workspace_bytes(int64_t batch, int64_t max_q, int64_t num_heads,
                                     int64_t kv_heads, int64_t head_dim);

fp4idx_status fp4idx_prompt_attention(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
    int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
    int64_t v_head_stride, int dtype, const int32_t* q_starts, const int32_t* k_starts,
    int64_t max_q, int64_t max_k, int64_t window, int64_t sinks, float softmax_scale, void* out,
    float* lse, int64_t batch, int64_t q_tokens, int64_t k_tokens, int64_t num_heads,
    int64_t kv_heads, int64_t head_dim, void* workspace, size_t workspace_bytes,
    uint32_t* err_flags, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP4IDX_STEP_H */
