/*
 * replayssm_hybrid.h -- C ABI of libreplayssm.so, third part: the short
 * convolution before the layer operators of replayssm_block.h, and the attention
 * layers between such layers in a hybrid stack, forward only.
 *
 * rsm_causal_conv runs the convolution over packed prompts, rsm_causal_conv_step
 * over the new tokens of running requests; both keep the last inputs in a cache
 * whose rows go by token position, so that a rejected draft costs nothing to undo.
 * rsm_rotary_append turns the queries and keys of new tokens by their positions
 * and writes keys and values to their pages, rsm_paged_attention reads the pages,
 * rsm_copy_pages copies pages of all layers' pools in one call.
 *
 * Ownership, streams and errors are rsm_materialize's: device pointers, caller-
 * owned, kernels enqueued on `stream`, nothing allocated, no device memory read
 * on the host, no synchronization; host checks return RSM_EINVAL / RSM_ENOTSUP
 * with rsm_hybrid_last_error() before anything is enqueued.  Out-of-range metadata
 * is skipped on the device and flagged in *device_status (optional).
 *
 * Types.  Token tensors, caches and outputs: input_dtype (RSM_BF16 or RSM_F32);
 * weights, biases and frequencies fp32.  Sums are fp32 everywhere, and an output is
 * rounded to its type once; what attention rounds on the way stands at its call.
 *
 * Sizes.  Sequences, requests, a window, a window's heads (attention) and a token's values
 * (rsm_rotary_append) are at most 2^30 each; tokens, pages and pools may be more than 2^31 elements.
 */
#ifndef REPLAYSSM_HYBRID_H
#define REPLAYSSM_HYBRID_H

#include "replayssm_block.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RSM_STATUS_BAD_POSITION 64u /* a position < 0, or a length that is negative, less than the new tokens or past the page table */
#define RSM_STATUS_BAD_PAGE 128u    /* a page outside [0, num_pages) where a token or a copy needs one */

/*
 * The short causal convolution, over each channel c on its own: for token t of a
 * sequence,
 *     v = bias[c] + sum_{j < width} weight[c, width - 1 - j] in(t - j, c)
 *     out(t, c) = silu ? v / (1 + exp(-v)) : v
 * in() is the sequence's input.  Before the call's own tokens it is the cache's:
 * the input at position p (0, 1, ... from the sequence's start) lies in row
 * p mod cache_rows of the sequence's slot, [num_slots, cache_rows, channels], rows
 * contiguous, slots cache_slot_stride elements apart; at negative positions it is 0.
 *
 * Packed prompts: sequence s is tokens cu_seqlens[s] .. cu_seqlens[s+1]-1 of x (it
 * may be empty), at positions positions[s] (NULL: 0) and up, with its earlier inputs
 * in slot slots[s]; its last min(length, width - 1) inputs are stored there.
 * Without a cache, and with pad_slot_id, all earlier inputs are 0 and nothing is
 * stored.  A slot or a position out of range counts as pad_slot_id and is flagged.
 * Slots are distinct.  cache_rows >= width - 1.  Output rows outside every sequence are not
 * written; sequences outside [0, tokens], and all from where cu_seqlens goes back, are
 * skipped and flagged.  out does not overlap x.
 */
typedef struct rsm_causal_conv_args {
  const void *x;              /* [tokens, channels] */
  const float *weight, *bias; /* [channels, width]; [channels] or NULL */
  const int32_t *cu_seqlens;  /* [num_seqs + 1] */
  void *cache;                /* NULL: no earlier inputs, nothing stored */
  const int32_t *slots, *positions; /* [num_seqs]; positions may be NULL */
  void *out;                  /* [tokens, channels] */
  uint32_t *device_status;
  int64_t tokens, x_stride, out_stride, cache_slot_stride;
  int32_t num_seqs, num_slots, channels, width, cache_rows, input_dtype, silu, pad_slot_id; /* width: 2, 3 or 4 */
} rsm_causal_conv_args;

RSM_API int rsm_causal_conv(const rsm_causal_conv_args *args, void *stream);

/*
 * Running requests: `window` new tokens each, the first at position positions[b],
 * earlier inputs in slot slots[b]; all new inputs are stored to their rows.  With
 * cache_rows >= width - 1 + window the call leaves every row that a token at or after
 * positions[b] may look back to: if only the first k tokens are accepted, the next call
 * starts at positions[b] + k and writes over the others.  Slots are distinct.  A request
 * with pad_slot_id is skipped: its output rows are zero.  So is one with a slot or
 * position out of range, which is flagged.  out does not overlap x.
 */
typedef struct rsm_causal_conv_step_args {
  const void *x;              /* [batch, window, channels] */
  const float *weight, *bias;
  void *cache;
  const int32_t *slots, *positions; /* [batch] */
  void *out;                  /* [batch, window, channels] contiguous */
  uint32_t *device_status;
  int64_t x_batch_stride, x_stride, cache_slot_stride;
  int32_t batch, window, num_slots, channels, width, cache_rows, input_dtype, silu, pad_slot_id;
  int32_t reserved; /* 0 */
} rsm_causal_conv_step_args;

RSM_API int rsm_causal_conv_step(const rsm_causal_conv_step_args *args, void *stream);

/*
 * Pages.  A layer's keys and values are [num_pages, page_size, num_kv_heads, dim],
 * a head's row contiguous, the other strides given in elements.  Token i of request
 * b lies in row i mod page_size of page page_table[b, i / page_size]; entries that no
 * token of a call needs are not looked at.  lengths[b] counts the request's tokens,
 * the call's new ones among them, which are the last: of n new tokens, token i is at
 * position lengths[b] - n + i.  A request of length 0 is skipped, its output rows are
 * zero; so is one whose length is out of range (negative, less than its new tokens, past
 * the page table), which is flagged.
 */
typedef struct rsm_pages {
  void *k, *v;
  const int32_t *page_table; /* [requests, table_width] */
  const int32_t *lengths;    /* [requests] */
  int64_t k_page_stride, k_row_stride, k_head_stride, v_page_stride, v_row_stride, v_head_stride, table_stride;
  int32_t requests, table_width, num_pages, page_size;
} rsm_pages;

/*
 * Rotary positions.  The first rotary_dim columns of each head of q and k are pairs,
 * (2j, 2j + 1) where `interleaved`, else (j, j + rotary_dim / 2); at position p pair
 * (a, b) becomes
 *     amplitude (a cos(p f_j) - b sin(p f_j),  b cos(p f_j) + a sin(p f_j)),   f = inv_freq
 * with the angle exact to 2^-24 of a turn at every position; where |f_j| is not below 2^40 the pair becomes NaN.
 * rotary_dim is even and at most dim, dim at most 256; the other columns stay.  q goes to
 * q_out, k and v to their pages.  The tokens are packed, request b's new ones
 * cu_seqlens[b] .. cu_seqlens[b+1]-1 (any number, also none), or `window` of each request (cu_seqlens NULL).
 * The tokens of different requests lie in different rows of the pages, and keys in other rows than values.  A token whose
 * page is out of range is flagged, and its k and v are not kept.  Output rows outside every sequence are
 * not written; sequences outside [0, tokens], and all from where cu_seqlens goes back, are skipped and flagged.
 * q_out may be q.
 */
typedef struct rsm_rotary_append_args {
  const void *q, *k, *v;     /* [tokens, heads, dim] or [requests, window, heads, dim] */
  const float *inv_freq;     /* [rotary_dim / 2] */
  const int32_t *cu_seqlens; /* [requests + 1] or NULL */
  void *q_out;
  uint32_t *device_status;
  rsm_pages pages;
  int64_t tokens;            /* of a packed call */
  int64_t q_batch_stride, q_stride, k_batch_stride, k_stride, v_batch_stride, v_stride, out_batch_stride, out_stride;
  int32_t window, num_heads, num_kv_heads, dim, rotary_dim, input_dtype, interleaved;
  float amplitude;
} rsm_rotary_append_args;

RSM_API int rsm_rotary_append(const rsm_rotary_append_args *args, void *stream);

/*
 * Attention of new tokens over their requests' pages: for new token t at position p
 * and head h (key head h / (num_heads / num_kv_heads)),
 *     out = sum_{i <= p} softmax_i(scale q . k_i) v_i
 * Tokens in a page out of range are not seen, and flagged; a row that sees none, or none
 * with a score above -infinity, is zero.  dim: 1 .. 256.
 *
 * Arithmetic.  Scores, maxima and sums fp32, and the weights (each softmax's numerators) where inputs are fp32 or rows
 * are no whole 16-byte vectors.  With bf16 inputs the weights meet v with 16 bits where num_heads / num_kv_heads * window
 * is at most 24 (8 if dim is above 128), else rounded to bf16.  So, with u = 2^-8 for bf16 outputs and 2^-24 for fp32,
 * r = 0, 2^-15 or 2^-8 for the weights, s the largest sum over |scale q_c k_c| of a score of the row, n its tokens
 * and M the sum of the absolute values of an output's terms, the output is, to first order, within
 *     u |y| + (r + 2 s (dim + 2) 2^-23 + 2^-20 + n 2^-23) M.
 * Values that are not finite reach the rows whose token sees them, and no others; a numerator is at most one,
 * to within its score's rounding, where it meets its value, so an output is finite where the number of tokens times
 * the largest value is well below the largest fp32 value.
 */
typedef struct rsm_paged_attention_args {
  const void *q;   /* [requests, window, num_heads, dim] */
  void *out;       /* the same, contiguous; may be q itself where that is contiguous */
  void *workspace; /* rsm_paged_attention_workspace() bytes, 256-byte aligned; one call's at a time */
  uint32_t *device_status;
  rsm_pages pages; /* read only */
  int64_t q_batch_stride, q_stride, workspace_bytes;
  int32_t window, num_heads, num_kv_heads, dim, input_dtype;
  float scale;
} rsm_paged_attention_args;

RSM_API int rsm_paged_attention(const rsm_paged_attention_args *args, void *stream);

/* Bytes of workspace rsm_paged_attention needs for *args on the current device
 * (its pointers are not looked at), or a negative return code. */
RSM_API int64_t rsm_paged_attention_workspace(const rsm_paged_attention_args *args);

/*
 * Copies of pages: for every pool l and pair i, page dst_pages[i] of pool l becomes
 * page src_pages[i].  Pools' base addresses and page strides (in elements) are tables
 * on the device, as rsm_materialize's; a page is page_elements contiguous elements of
 * `dtype` (any rsm_dtype).  A pair with a negative page is skipped, one with a page
 * past num_pages is skipped and flagged.  Destinations are distinct and no pair's
 * source, but a pair of one page with itself, which copies nothing, is allowed.
 */
typedef struct rsm_copy_pages_args {
  const int64_t *page_ptrs, *page_strides; /* [num_pools] */
  const int32_t *src_pages, *dst_pages;    /* [num_pairs] */
  uint32_t *device_status;
  int64_t page_elements;
  int32_t num_pools, num_pairs, num_pages, dtype;
} rsm_copy_pages_args;

RSM_API int rsm_copy_pages(const rsm_copy_pages_args *args, void *stream);

/* Message of the last failing call of this header on this thread ("" if none). */
RSM_API const char *rsm_hybrid_last_error(void);

/* sizeof of the five argument structs, in the order above (index 0 .. 4), for
 * bindings that check their layout; 0 for another index. */
RSM_API int rsm_hybrid_args_size(int index);

#ifdef __cplusplus
}
#endif

#endif /* REPLAYSSM_HYBRID_H */
