/*
 * mxfp4el_attention.h -- C ABI of the attention half of a decoder layer on
 * GB300: the operators a serving program runs next to the routed experts of
 * mxfp4_expert_linear.h, in the same library, with the same status codes,
 * dtypes and rules (device pointers owned by the caller, work enqueued on
 * `stream`, arguments checked before anything is enqueued).
 *
 *   mxfp4el_append_kv         norms of the query and key heads, the position
 *                             rotation, and the write of the new keys and
 *                             values into a paged cache, in one pass
 *   mxfp4el_attention_decode  attention of one new token of each sequence
 *   mxfp4el_attention_prefill attention of ragged prompts or prompt chunks
 *
 * Positions. A sequence holds seq_lens[b] tokens, its new ones included, and
 * its new tokens are its last ones: with m new tokens, new token i has
 * position seq_lens[b] - m + i. Key j of a sequence lives in slot
 * j % page_size of page page_table[b][j / page_size].
 *
 * Mask. The query at position a sees key j when 0 <= j <= a and, with a
 * window w > 0, when a - j < w or j < sinks. Keys and values that a query
 * does not see never reach its result, whatever they hold; slots past a
 * sequence's length and pages that no query sees are not read. A query that
 * sees no key gives zeros.
 *
 * Result. For query head h of key head h / (num_heads / num_kv_heads):
 *
 *   s_j = scale * q . k_j,   m = max over the visible s_j and sink_logits[h]
 *   out = sum_j exp(s_j - m) v_j / (sum_j exp(s_j - m) + exp(sink_logits[h] - m))
 *
 * with the last term only where sink_logits is given. Scores, softmax sums
 * and accumulators are float32; the result is rounded once to the token
 * dtype. On bf16 the weights exp(s_j - m) are rounded to bf16 where they
 * multiply the values (a relative error of 2^-8 at most, as the result's own
 * rounding); decode's sum adds the rounded weights, prefill's the float32
 * ones. A value that is infinite or NaN gives infinities or NaN, in its
 * column, to the queries that see its key. The order of every sum is fixed, so the same call on the same
 * inputs gives the same bits.
 */
#ifndef MXFP4EL_ATTENTION_H
#define MXFP4EL_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A paged cache of keys and values. k and v are (num_pages, num_kv_heads,
 * page_size, head_dim) arrays of `dtype` (MXFP4EL_DTYPE_F32 or _BF16) with
 * element strides of their own for pages, heads and slots, so both
 * (page, head, slot, width) and (page, slot, head, width) memory orders fit;
 * a row's head_dim elements are contiguous. Bases and strides are multiples
 * of 16 bytes. num_pages is at least 1; page_size is a power of two from 8 to
 * 1024; head_dim is 64 or 128.
 */
typedef struct mxfp4el_kv_cache {
  void* k;
  void* v;
  int64_t num_pages, num_kv_heads, page_size, head_dim;
  int64_t k_page_stride, k_head_stride, k_slot_stride;
  int64_t v_page_stride, v_head_stride, v_slot_stride;
  int64_t dtype;
} mxfp4el_kv_cache;

/*
 * The sequences of a call, in device memory. page_table is (num_seqs,
 * max_pages) int32 with a row stride of table_stride elements; entries past
 * a sequence's length are not read. seq_lens is (num_seqs) int32. q_offsets
 * is (num_seqs + 1) int32, starting at 0 and never falling: sequence b's new
 * tokens are rows q_offsets[b] .. q_offsets[b + 1] - 1 of the call's token
 * arrays. NULL: one new token per sequence, row b. All lie on 4-byte
 * boundaries, as sink_logits does.
 *
 * A page id outside [0, num_pages) is not followed: attention takes its keys
 * and values as zeros, the append drops the token's key and value. A length
 * beyond max_pages * page_size, or beyond 2^30, is cut to it. Each is counted for
 * mxfp4el_page_errors() where it is met.
 */
typedef struct mxfp4el_sequences {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* q_offsets;
  int64_t num_seqs, max_pages, table_stride;
} mxfp4el_sequences;

/*
 * mxfp4el_append_kv -- T new tokens, num_heads query heads.
 *
 * q is (T, num_heads, head_dim), k and v (T, num_kv_heads, head_dim), with
 * their own token and head strides in elements (the slices of one fused
 * projection fit); bases and strides are multiples of 16 bytes. Every query
 * and key row x is normed and turned:
 *
 *   y = x / sqrt(mean(x^2) + eps) * norm         (norm given; else y = x)
 *   (a, b) -> (a cos - b sin, b cos + a sin)     (first rotary_dim elements)
 *
 * with a, b the elements i and i + rotary_dim / 2 (interleaved == 0) or 2i
 * and 2i + 1 (interleaved != 0) and cos, sin the elements i and
 * rotary_dim / 2 + i of row `position` of cos_sin (max_positions, rotary_dim)
 * float32. rotary_dim is 0 (no rotation; cos_sin is not read) or a multiple
 * of 16 up to head_dim. q_norm and k_norm are (head_dim) in the token dtype,
 * or NULL. All in float32, rounded once. Turned queries go to q_out (T,
 * num_heads, head_dim), dense; turned keys and the values as they are go to
 * the token's cache slot.
 *
 * A token whose position is negative, beyond the page table or beyond
 * max_positions, or whose page id is out of range, appends nothing and is
 * counted; where it has no rotation its q_out row is zeros. Rows past
 * q_offsets[num_seqs] append nothing and get zeros in q_out. Two tokens of a
 * call must not share a slot.
 *
 * Returns MXFP4EL_OK, MXFP4EL_ERR_INVALID_ARGUMENT (null pointer, negative
 * or mismatched size, alignment, page_size, head_dim, rotary_dim),
 * MXFP4EL_ERR_UNSUPPORTED_DTYPE, MXFP4EL_ERR_ALIAS (q_out or the cache
 * overlaps an input), MXFP4EL_ERR_TOO_LARGE or MXFP4EL_ERR_CUDA.
 */
int mxfp4el_append_kv(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                      const void* k, int64_t k_token_stride, int64_t k_head_stride,
                      const void* v, int64_t v_token_stride, int64_t v_head_stride,
                      const void* q_norm, const void* k_norm, float eps,
                      const float* cos_sin, int64_t max_positions, int64_t rotary_dim,
                      int interleaved, const mxfp4el_kv_cache* cache,
                      const mxfp4el_sequences* seqs, void* q_out,
                      int64_t T, int64_t num_heads, void* stream);

/*
 * mxfp4el_attention_decode -- one new token of each sequence: row b of q
 * (num_seqs, num_heads, head_dim; strides as above) over the keys of
 * sequence b, the token's own among them. seqs->q_offsets must be NULL.
 * scale is positive. window 0: no window (sinks is then not used). sink_logits is (num_heads)
 * float32 or NULL. out is (num_seqs, num_heads, head_dim), dense.
 *
 * `workspace` is a device buffer of at least
 * mxfp4el_attention_workspace_size() bytes, 256-byte aligned, zeroed once
 * before its first use; every call leaves it ready for the next. Calls in
 * flight at once (on different streams) must not share it, and after
 * mxfp4el_wait_timeouts() reported a wait that gave up it is zeroed again.
 *
 * num_heads is a multiple of num_kv_heads, up to 128 query heads to a key
 * head. Returns the codes of mxfp4el_append_kv, plus MXFP4EL_ERR_WORKSPACE.
 */
int mxfp4el_attention_decode(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                             const mxfp4el_kv_cache* cache, const mxfp4el_sequences* seqs,
                             float scale, int64_t window, int64_t sinks,
                             const float* sink_logits, void* out, int64_t num_heads,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * mxfp4el_attention_prefill -- T new tokens of seqs->num_seqs sequences,
 * rows as seqs->q_offsets says (NULL: one token per sequence, T ==
 * num_seqs). Rows past q_offsets[num_seqs] give zeros. Everything else as
 * mxfp4el_attention_decode. (T + num_seqs + 1) * num_kv_heads beyond about
 * 2^31 is MXFP4EL_ERR_TOO_LARGE.
 */
int mxfp4el_attention_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                              const mxfp4el_kv_cache* cache, const mxfp4el_sequences* seqs,
                              float scale, int64_t window, int64_t sinks,
                              const float* sink_logits, void* out, int64_t T,
                              int64_t num_heads, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Bytes of workspace that any call of the two above needs. */
size_t mxfp4el_attention_workspace_size(void);

/*
 * Synchronises `stream`, then returns in *count how often the calls on the
 * current device met a page id, length or position out of range since the
 * last call of this function, and resets the count.
 */
int mxfp4el_page_errors(void* stream, int64_t* count);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4EL_ATTENTION_H */
