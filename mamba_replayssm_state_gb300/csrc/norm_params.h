// norm_params.h -- what the norm kernels are given.
#pragma once
#include <cstdint>

#include "../../include/replayssm_block.h"

namespace rmsnorm {

struct Params {
  const void *x, *other;  // other: the residual, or the gate z
  const float* weight;
  void *out, *residual_out;
  int64_t rows, x_rs, other_rs, out_rs, res_rs;  // row strides, elements
  int32_t dim, group, groups;                    // columns of a row, of one norm; norms of a row
  float scale, eps;
};

// Whether CTAs stay for many groups.  Two groups have to fit a thread's 64 registers.
// (8192 rows, 8 groups of 2048 bf16 columns, gated: 124 us, 149 with a CTA a group.
// The residual sum writes as much as it reads and gains nothing: 8192 rows of 4096
// columns, fp32 residuals: 72 us, 62 with a CTA a row.)
constexpr bool can_loop(int kind, bool bf16_inputs, int vectors) { return kind == 1 && bf16_inputs && vectors <= 2; }

// kind 0: add, 1: gate then norm, 2: norm then gate; types are rsm_dtype codes
// (other_dtype: the residual's; the gate has the input's).  vectors: of a
// thread (1, 2 or 4; 0: the two-pass kernel); warp: a group a warp; loop: CTAs stay.
const void* kernel(int kind, int input_dtype, int other_dtype, int vectors, bool warp, bool loop);

}  // namespace rmsnorm
