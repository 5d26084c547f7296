/*
 * replayssm_block.h -- C ABI of libreplayssm.so, second part: the operators of
 * the layer around rsm_materialize, forward only.
 *
 * The layer is linear attention with a decay for each head.  Per sequence and
 * head h (B and C group g(h) = h / (num_heads / num_groups)), for token t
 *     S_t = exp(dt_t A[h]) S_{t-1} + dt_t x_t (x) B_t      [dim, dstate]
 *     y_t = S_t C_t + D[h] x_t                             [dim]
 * rsm_ssm_prefill runs it over packed prompts (chunked form), rsm_ssm_step over
 * the new tokens of running requests (state slot to state slot), and
 * rsm_replayssm_decode over new tokens from a checkpoint slot and its replay
 * ring, writing the ring and leaving the state to a later rsm_materialize.
 * rsm_add_rms_norm and rsm_gated_rms_norm are the norms before and after it.
 *
 * Ownership, streams and errors are rsm_materialize's: device pointers, caller-
 * owned, kernels enqueued on `stream`, nothing allocated, no device memory read
 * on the host, no synchronization; host checks return RSM_EINVAL / RSM_ENOTSUP
 * with rsm_block_last_error() before anything is enqueued.  Out-of-range metadata is
 * skipped on the device and flagged in *device_status (optional).
 *
 * Types.  x, B, C and the output: input_dtype (RSM_BF16 or RSM_F32).  dt, A, D:
 * fp32; dt is the final step size and dt A <= 0 (a growing state is computed as
 * written, but may overflow before it would in exact arithmetic).  States: fp32,
 * bf16, fp16; the ring form also reads int8 and fp8 e4m3 with a scale per (head,
 * dim row).  (dim, dstate): (16,16), (64,64), (64,128); one-byte (64,128) only.
 *
 * Arithmetic.  Sums and states are fp32 everywhere, and a state is rounded to its
 * type once a call, when it is stored.  With fp32 inputs, and states that are not 64
 * x 128, all else is fp32 too.  With bf16 inputs and 64 x 128 states products may run
 * on the tensor cores, and their operands are rounded:
 *   prompts (8 tokens and more whose rows are whole 16-byte vectors): the weight of a
 *     token pair, D in a token's own, and the state as outputs read it, to bf16; what a
 *     token adds to the state to 16 bits, or to bf16 where no final state is kept or it is bf16
 *   2 to 8 tokens of a step, and up to 16 after a ring (but one, on fp16 states):
 *     the weights, D in them, to bf16; an fp32 state as outputs read it, and what a
 *     token adds to a state, to 16 bits
 * With M the sum of the absolute values of the terms an element is made of, such an
 * output is within 2^-8 |y| + (2^-8 + 2^-15) M, and a state within 2^-15 M (bf16
 * states after a prompt: as outputs) and the rounding to its type.
 *
 * Layout.  A token's x is [num_heads, dim], B and C [num_groups, dstate], dt
 * [num_heads], all contiguous; strides between tokens (and requests) are given
 * in elements, so slices of one projection need no copy.  A state slot is
 * [num_heads, dim, dstate], contiguous; slots are state_slot_stride elements apart.
 *
 * A value that is not finite spreads to where the recurrence takes it, and may
 * also reach earlier tokens of its own chunk of up to 128 tokens of a prompt, or of
 * its own call where the new tokens are several; it never reaches another sequence, request or head of another group.
 */
#ifndef REPLAYSSM_BLOCK_H
#define REPLAYSSM_BLOCK_H

#include "replayssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RSM_STATUS_BAD_SEQUENCE 32u /* cu_seqlens goes back, or lies outside [0, tokens] */

/*
 * Prompts.  Sequence s is tokens cu_seqlens[s] .. cu_seqlens[s+1]-1 of the
 * packed tensors (it may be empty).  Its state starts from
 * state[initial_slots[s]] (NULL, or pad_slot_id: from zero) and ends in
 * state[final_slots[s]] (NULL, or pad_slot_id: not kept).  Final slots are
 * distinct and are no other sequence's initial slot; a sequence's own may
 * coincide.  Output rows outside every sequence are not written.  A sequence that
 * lies outside [0, tokens] is skipped, and so are all from where cu_seqlens goes
 * back; a slot out of range counts as pad_slot_id.  Both are flagged.
 */
typedef struct rsm_ssm_prefill_args {
  const void *x, *B, *C; /* [tokens, ...] input_dtype */
  const float *dt, *A, *D; /* [tokens, num_heads], [num_heads], [num_heads] or NULL */
  const int32_t *cu_seqlens; /* [num_seqs + 1] */
  void *state;             /* [num_slots, num_heads, dim, dstate]; NULL when no slots are given */
  const int32_t *initial_slots, *final_slots; /* [num_seqs] or NULL */
  void *out;               /* [tokens, num_heads, dim] input_dtype */
  void *workspace;         /* rsm_ssm_prefill_workspace() bytes, 256-byte aligned */
  uint32_t *device_status;
  int64_t tokens;
  int64_t x_stride, B_stride, C_stride, dt_stride, out_stride; /* between tokens, in elements */
  int64_t state_slot_stride;
  int64_t workspace_bytes;
  int32_t num_seqs, num_slots, num_heads, num_groups, dim, dstate;
  int32_t state_dtype, input_dtype, pad_slot_id;
} rsm_ssm_prefill_args;

RSM_API int rsm_ssm_prefill(const rsm_ssm_prefill_args *args, void *stream);

/* Bytes of workspace rsm_ssm_prefill needs for *args on the current device
 * (its pointers are not looked at), or a negative return code. */
RSM_API int64_t rsm_ssm_prefill_workspace(const rsm_ssm_prefill_args *args);

/*
 * Running requests: `window` new tokens of each of `batch` requests, applied in
 * order to state[src_slots[b]] and stored to state[dst_slots[b]] (NULL: in
 * place).  A request whose source slot is pad_slot_id is skipped: its output
 * rows are zero and nothing is stored; a destination of pad_slot_id is not
 * stored.  Destinations are distinct and are no other request's source (requests
 * have no order among themselves); a request's own may coincide.  Slots out of
 * range count as pad_slot_id and are flagged.
 */
typedef struct rsm_ssm_step_args {
  const void *x, *B, *C;   /* [batch, window, ...] input_dtype */
  const float *dt, *A, *D;
  void *state;             /* [num_slots, num_heads, dim, dstate], fp32, bf16 or fp16 */
  const int32_t *src_slots, *dst_slots; /* [batch] */
  void *out;               /* [batch, window, num_heads, dim] contiguous */
  uint32_t *device_status;
  int64_t x_batch_stride, x_stride, B_batch_stride, B_stride, C_batch_stride, C_stride, dt_batch_stride, dt_stride;
  int64_t state_slot_stride;
  int32_t batch, window, num_slots, num_heads, num_groups, dim, dstate;
  int32_t state_dtype, input_dtype, pad_slot_id;
} rsm_ssm_step_args;

RSM_API int rsm_ssm_step(const rsm_ssm_step_args *args, void *stream);

/*
 * The same from a checkpoint and its replay ring: the state in slot slots[b]
 * is advanced, for the outputs only, by ring rows ring_start[b] ..
 * ring_start[b] + ring_len[b] - 1 (modulo ring_buffer_len), then by the new
 * tokens, whose x, B and dt are written to the ring rows that follow.  The
 * caller advances ring_len and later commits a prefix with rsm_materialize,
 * whose cache layout this is: x [ring_buffer_len, num_heads, dim], B
 * [ring_buffer_len, num_groups, dstate], dt [ring_buffer_len, num_heads] per
 * slot.  ring_len + window <= min(ring_buffer_len, 64).  Slots of the batch are
 * distinct.  A request with the pad slot is skipped (zero output rows, ring
 * untouched); one with a slot, ring_start or ring_len out of range likewise,
 * and flagged.
 */
typedef struct rsm_replayssm_decode_args {
  const void *x, *B, *C;
  const float *dt, *A, *D;
  const void *state;        /* any state_dtype; read only */
  const float *state_scale; /* [num_slots, num_heads, dim], one-byte state only */
  void *x_cache, *B_cache;  /* input_dtype */
  float *dt_cache;
  const int32_t *slots, *ring_start, *ring_len; /* [batch] */
  void *out;
  uint32_t *device_status;
  int64_t x_batch_stride, x_stride, B_batch_stride, B_stride, C_batch_stride, C_stride, dt_batch_stride, dt_stride;
  int64_t state_slot_stride, scale_slot_stride, x_cache_slot_stride, B_cache_slot_stride, dt_cache_slot_stride;
  int32_t batch, window, num_slots, num_heads, num_groups, dim, dstate, ring_buffer_len;
  int32_t state_dtype, input_dtype, pad_slot_id;
} rsm_replayssm_decode_args;

RSM_API int rsm_replayssm_decode(const rsm_replayssm_decode_args *args, void *stream);

/*
 * The norm before a block: r = residual + residual_scale x; residual_out = r
 * (rounded once); out = r / sqrt(mean(r^2) + eps) * weight, from the unrounded
 * r.  x and out: input_dtype; residual and residual_out: residual_dtype (both
 * RSM_F32 or RSM_BF16).  residual_out may be residual, and out may be x.
 */
typedef struct rsm_add_rms_norm_args {
  const void *x, *residual;
  const float *weight; /* [dim] */
  void *out, *residual_out;
  int64_t rows, x_stride, residual_stride, out_stride, residual_out_stride;
  int32_t dim, input_dtype, residual_dtype;
  float residual_scale, eps;
} rsm_add_rms_norm_args;

RSM_API int rsm_add_rms_norm(const rsm_add_rms_norm_args *args, void *stream);

/*
 * The norm after a block, over groups of `group_size` columns: with v = x
 * silu(z), out = v / sqrt(mean(v^2) + eps) * weight; with norm_before_gate,
 * out = x / sqrt(mean(x^2) + eps) * weight * silu(z).  out may be x.
 */
typedef struct rsm_gated_rms_norm_args {
  const void *x, *z;
  const float *weight; /* [dim] */
  void *out;
  int64_t rows, x_stride, z_stride, out_stride;
  int32_t dim, group_size, input_dtype, norm_before_gate;
  float eps;
  int32_t reserved; /* 0 */
} rsm_gated_rms_norm_args;

RSM_API int rsm_gated_rms_norm(const rsm_gated_rms_norm_args *args, void *stream);

/* Message of the last failing call of this header on this thread ("" if none). */
RSM_API const char *rsm_block_last_error(void);

/* sizeof of the five argument structs, in the order above (index 0 .. 4), for
 * bindings that check their layout; 0 for another index. */
RSM_API int rsm_block_args_size(int index);

#ifdef __cplusplus
}
#endif

#endif /* REPLAYSSM_BLOCK_H */
