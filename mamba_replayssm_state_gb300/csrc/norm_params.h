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
  int32_t dim, group;                            // group: columns of one norm
  float scale, eps;
};

// kind 0: add, 1: gate then norm, 2: norm then gate; types are rsm_dtype codes
// (other_dtype: the residual's; the gate has the input's).
const void* kernel(int kind, int input_dtype, int other_dtype);

}  // namespace rmsnorm
