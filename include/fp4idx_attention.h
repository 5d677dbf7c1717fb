/*
 * fp4idx_attention.h -- C ABI of the operators of libfp4idx.so that follow
 * the index scorer: the 8-bit key/value cache (written, read back), the
 * selection of tokens from index logits, and attention over that cache, dense
 * or over the selected tokens.  One GB300 GPU (sm_103a).
 *
 * The steps of a sparse-attention layer, and the calls that make them:
 *   index keys and queries        fp4idx_indexer_prepass      (fp4idx.h)
 *   main keys and values          fp4idx_kv_store_fp8
 *   index logits                  fp4idx_paged_mqa_logits     (fp4idx.h)
 *   the k best tokens of a row    fp4idx_topk_tokens
 *   attention over them           fp4idx_sparse_attention_fp8
 *   attention over all of them    fp4idx_paged_attention_fp8  (dense layers,
 *                                 sliding windows, short contexts)
 *   cached tokens in 16 bits      fp4idx_kv_load_fp8
 *
 * The conventions are those of fp4idx.h: device pointers, buffers owned by
 * the caller, nothing allocated and nothing synchronised by the library,
 * host-side checks before anything is enqueued, errors of the kernel at the
 * caller's next synchronisation.  Pages hold FP4IDX_KV_BLOCK = 64 tokens, the
 * index cache's page size, so one block table serves both caches.  Calls keep
 * no state: two of them may run at once on different streams if they do not
 * write the same memory (each call needs a workspace of its own).
 *
 * Elements of 16 bits are bf16 or fp16 (fp4idx_dtype).
 */
#ifndef FP4IDX_ATTENTION_H
#define FP4IDX_ATTENTION_H

#include "fp4idx.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fp4idx_dtype { FP4IDX_BF16 = 0, FP4IDX_FP16 = 1 } fp4idx_dtype;

/*
 * The paged 8-bit cache of one layer.  Codes are E4M3 (e4m3fn), one fp32
 * scale, a power of two, for every page and head; the value of an element is
 * code * scale.
 *
 *   k_codes, v_codes   bytes, element (block, head, offset, d) at
 *                      block*code_block_stride + (head*64 + offset)*head_dim
 *                      + d.  16-byte aligned.
 *   k_scale, v_scale   fp32, (block, head) at block*scale_block_stride + head.
 *   code_block_stride  bytes, a multiple of 16, >= kv_heads*64*head_dim
 *   scale_block_stride floats, >= kv_heads
 *                      (keys and values may be halves of one tensor).
 *   kv_heads           1 .. 65535;  head_dim 64 or 128;
 *   num_blocks         1 .. 2^31-1.
 */
typedef struct fp4idx_kv_cache {
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scale;
  float* v_scale;
  int64_t num_blocks;
  int64_t code_block_stride;
  int64_t scale_block_stride;
  int32_t kv_heads;
  int32_t head_dim;
} fp4idx_kv_cache;

/*
 * Quantises keys and values as they are written.  Token t goes to slot
 * slot_mapping[t] = block*64 + offset (the slot mapping of the index keys);
 * a negative slot skips the token.
 *
 * A run is a set of consecutive tokens of the call whose slots are
 * consecutive and on one page.  For each run, head, and keys and values:
 *   amax  = max |x| over the run (NaN ignored; an infinity makes the scale
 *           2^127, which leaves nothing of the page's other values);
 *   scale = ceil_pow2(max(rn32(amax / 448), 2^-126)), the rule of the FP8
 *           output mode of the pre-pass; if the run starts at an offset > 0,
 *           the page's rows before it are kept and scale is at least the
 *           page's present scale;
 *   codes of the run = E4M3(x / scale) (round half to even, saturating);
 *   codes of the kept rows, if scale grew: E4M3(code * old / scale).
 * Rows of the page behind the run are left as they were.  So a page's first
 * row (offset 0) starts its scale anew, and appending to it never shrinks
 * the scale.
 *
 *   k, v          16-bit [num_tokens, kv_heads, head_dim], row (t, h) at
 *                 t*token_stride + h*head_stride elements; 16-byte aligned,
 *                 strides multiples of 8.
 *   slot_mapping  int64 [num_tokens].  A page is in one run of the call at
 *                 most (unspecified bytes on that page otherwise).
 *   err_flags     optional device uint32: FP4IDX_ERRFLAG_SLOT for a slot >=
 *                 num_blocks*64 (the token is skipped).
 * num_tokens == 0 returns FP4IDX_OK and enqueues nothing.
 */
fp4idx_status fp4idx_kv_store_fp8(const void* k, const void* v, int64_t k_token_stride,
                                  int64_t k_head_stride, int64_t v_token_stride,
                                  int64_t v_head_stride, int dtype, const int64_t* slot_mapping,
                                  const fp4idx_kv_cache* cache, int64_t num_tokens,
                                  uint32_t* err_flags, void* stream);

/*
 * Reads cached tokens back: k_out[t], v_out[t] = the values at slot
 * slot_mapping[t], rounded once to the output type.  Any order, repeated
 * slots included; a negative slot leaves the output row as it was.
 *
 *   k_out, v_out  16-bit [num_tokens, kv_heads, head_dim], dense, 16-byte
 *                 aligned.
 *   err_flags     optional: FP4IDX_ERRFLAG_SLOT as above (row untouched).
 */
fp4idx_status fp4idx_kv_load_fp8(const fp4idx_kv_cache* cache, const int64_t* slot_mapping,
                                 void* k_out, void* v_out, int dtype, int64_t num_tokens,
                                 uint32_t* err_flags, void* stream);

/*
 * Attention over the cache.  Sequence b has context_lens[b] cached tokens,
 * the last n_b of them its query tokens (their keys and values are stored
 * first), n_b = q_starts[b+1] - q_starts[b], or num_tokens / batch when
 * q_starts is NULL.  Query i of sequence b stands at position
 * p = context_lens[b] - n_b + i and sees the keys
 *   s <= p, and, if window > 0, also s > p - window or s < sinks.
 * With x_s = softmax_scale * sum_d q[d] k_s[d] over the keys it sees:
 *   lse = log sum_s exp(x_s),  out[d] = sum_s exp(x_s - lse) v_s[d];
 * a query that sees no key (p < 0) gets out = 0 and lse = -inf.  Query head h
 * reads key head h / (num_heads / kv_heads).
 *
 * Query elements are taken to within 2^-39 of their row's largest (those above
 * 2^-31 of it in bf16, 2^-28 in fp16, exactly); their products with keys are
 * exact in the tensor core, the softmax and both sums are fp32; probabilities are rounded to fp16 before the product
 * with the values, by 2^-11 of themselves or 2^-35 of the row's largest
 * contribution.  A score carries fp32's relative error into its exponent, so
 * |x_s| is to stay below 2^20; of scores so large that their spacing exceeds
 * the exponents' range, from about 2^23 on, the row's output is unspecified.
 *
 *   q             16-bit, row (t, h) at t*q_token_stride + h*q_head_stride
 *                 elements; 16-byte aligned, strides multiples of 8.  The
 *                 values are finite.
 *   block_table   int32, page p of sequence b at b*block_table_stride + p,
 *                 read for the pages that hold visible keys only;
 *                 block_table_stride >= ceil(max_context / 64).  May be NULL
 *                 where max_context is 0.
 *   context_lens  int32 [batch]; values are taken within [0, max_context].
 *   max_context   a bound on context_lens.  Kernel and work split are chosen
 *                 by it, so a loose one costs time, not correctness.
 *   q_starts      int32 [batch+1], ascending from 0 to num_tokens, or NULL.
 *   max_q         the largest n_b (ignored when q_starts is NULL); tokens of
 *                 a sequence behind its max_q-th are left unwritten.
 *   out           16-bit [num_tokens, num_heads, head_dim], dense, 16-byte
 *                 aligned.
 *   lse           optional fp32 [num_tokens, num_heads], natural logarithm.
 *   workspace     fp4idx_attention_workspace_bytes(batch, max_q, num_heads,
 *                 kv_heads, head_dim) bytes (max_q = num_tokens / batch
 *                 without q_starts; 0 bytes: arguments out of range), 16-byte
 *                 aligned, contents not kept; its own for each call in
 *                 flight (two captured graphs that may run at once too).
 *                 Fewer bytes return FP4IDX_ERR_SCRATCH.
 *   err_flags     optional: FP4IDX_ERRFLAG_PAGE for a block-table entry
 *                 outside [0, num_blocks) (its keys are left out),
 *                 FP4IDX_ERRFLAG_TIMEOUT if a wait inside the kernel ran out.
 * A NaN code among the keys or values that one query of a sequence sees may
 * reach other queries of the sequence.  What no query of the sequence sees
 * (behind context_lens, below the window and behind the first tokens) is never
 * used: its codes may hold anything, its pages' table entries too.
 */
size_t fp4idx_attention_workspace_bytes(int64_t batch, int64_t max_q, int64_t num_heads,
                                        int64_t kv_heads, int64_t head_dim);

fp4idx_status fp4idx_paged_attention_fp8(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
    const fp4idx_kv_cache* cache, const int32_t* block_table, int64_t block_table_stride,
    const int32_t* context_lens, const int32_t* q_starts, int64_t max_q, int64_t max_context,
    int64_t window, int64_t sinks, float softmax_scale, void* out, float* lse, int64_t batch,
    int64_t num_tokens, int64_t num_heads, void* workspace, size_t workspace_bytes,
    uint32_t* err_flags, void* stream);

/*
 * Attention over selected tokens: query token t sees the keys at positions
 * indices[t, 0 .. num_selected-1] of its sequence, the selection being shared
 * by all heads; negative entries are left out wherever they stand, and an
 * entry that occurs twice counts twice.  Everything else is as above.
 *
 *   block_table   int32, page p of sequence b at b*block_table_stride + p,
 *                 p < block_table_pages.  May be NULL where that is 0.
 *   seq_ids       int32 [num_tokens], the sequence of each token, in
 *                 [0, batch); or NULL: token t belongs to sequence
 *                 t / (num_tokens / batch).
 *   indices       int32, entry (t, i) at t*indices_stride + i.
 *   workspace     fp4idx_attention_workspace_bytes(num_tokens, 1, ...).
 *   err_flags     optional: FP4IDX_ERRFLAG_PAGE for an entry at or behind
 *                 block_table_pages*64, a sequence id outside [0, batch) or a
 *                 block-table entry outside [0, num_blocks) (left out).
 */
fp4idx_status fp4idx_sparse_attention_fp8(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
    const fp4idx_kv_cache* cache, const int32_t* block_table, int64_t block_table_stride,
    int64_t block_table_pages, const int32_t* seq_ids, const int32_t* indices,
    int64_t indices_stride, int64_t num_selected, float softmax_scale, void* out, float* lse,
    int64_t batch, int64_t num_tokens, int64_t num_heads, void* workspace, size_t workspace_bytes,
    uint32_t* err_flags, void* stream);

/*
 * The k largest logits of each row.  Row t has the entries s < row_lens[t]
 * (num_cols when row_lens is NULL); an entry that is -inf or NaN is never
 * selected, equal entries are selected from the lowest index up, and -0
 * equals +0.
 *   indices[t, 0 .. counts[t]-1]  the selected s, ascending;
 *   indices[t, counts[t] .. k-1]  -1;
 *   counts[t]                     min(k, entries that can be selected).
 *
 *   logits    fp32, row t at t*logits_stride, 4-byte aligned.
 *   row_lens  int32 [num_rows], taken within [0, num_cols], or NULL.
 *   indices   int32, row t at t*indices_stride; indices_stride >= k.
 *   counts    optional int32 [num_rows].
 *   k         1 .. 4096;  0 <= num_cols < 2^30.  Rows of more than 262,144
 *             columns take a slower method (about 3 us per 1,000 entries).
 */
fp4idx_status fp4idx_topk_tokens(const float* logits, int64_t logits_stride,
                                 const int32_t* row_lens, int32_t* indices,
                                 int64_t indices_stride, int32_t* counts, int64_t num_rows,
                                 int64_t num_cols, int64_t k, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP4IDX_ATTENTION_H */
