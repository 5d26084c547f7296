// ssm_params.h -- what the linear-attention kernels (prompts, running requests,
// ring decode) are given, and the compiled (dim, dstate) sizes.
#pragma once
#include <cstdint>

#include "../../include/replayssm_block.h"
#include "ssm_sequences.h"

namespace ssm {

// Where a unit's tokens and state come from.
enum Mode : int32_t { kPrefill = 0, kStep = 1, kDecode = 2 };

struct Params {
  const void *x, *B, *C;
  const float *dt, *A, *D;
  const int32_t* cu_seqlens;
  void* state;
  const float* scale;
  void *x_cache, *B_cache;
  float* dt_cache;
  const int32_t *src, *dst;  // prefill: initial and final slots; decode: dst unused
  const int32_t *ring_start, *ring_len;
  void* out;
  uint32_t* status;
  int64_t tokens;
  int64_t x_bs, x_ts, B_bs, B_ts, C_bs, C_ts, dt_bs, dt_ts, out_bs, out_ts;  // batch and token strides, elements
  int64_t state_ss, scale_ss, xc_ss, Bc_ss, dtc_ss;                         // slot strides, elements
  int32_t units, window, num_slots, H, G, R, pad, mode, state_dtype;
  int32_t heads_per_cta, tokens_max, wide;  // token kernel: tokens of a request at most; rows of x and B are 16-byte vectors
};

constexpr int kSeqTokens = 16;  // tokens staged in shared memory at a time (sequential kernel)

// The sequential kernel of an (input type, dim, dstate); NULL when not compiled.
const void* seq_kernel(int input_dtype, int dim, int dstate, int* threads);

// The new-token kernel of 64 x 128 states, 256 threads; NULL when not compiled.
// mode: 0 the ring form, 1 one token a request, state to state, 2 several;
// 3 and 4 the ring form on the tensor cores, up to 8 and up to 16 new tokens.
const void* token_kernel(int input_dtype, int state_dtype, int mode);
constexpr int kTokenThreads = 256;
constexpr int kTokenMaxNew = 16;  // new tokens of a request
constexpr int kTokenMaxAll = 64;  // with the ring's
constexpr int kTokenMaxHeads = 16;  // of a CTA
constexpr int kTokenMaxSmem = 75 * 1024;  // of a CTA: three an SM (one head of the longest ring takes 67 KB)
uint32_t token_smem(int mode, int input_bytes, int heads, int fresh, int all);

}  // namespace ssm
