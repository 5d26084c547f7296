// Instances of the convolution kernels.
#include "conv_kernel.cuh"

namespace hybrid {

namespace {

template <typename IT, int V>
const void* pick(int width) {
  switch (width) {
    case 2: return reinterpret_cast<const void*>(&conv_prompt_kernel<IT, 2, V>);
    case 3: return reinterpret_cast<const void*>(&conv_prompt_kernel<IT, 3, V>);
    default: return reinterpret_cast<const void*>(&conv_prompt_kernel<IT, 4, V>);
  }
}

template <typename IT, int V>
const void* pick_step(int width) {
  switch (width) {
    case 2: return reinterpret_cast<const void*>(&conv_step_kernel<IT, 2, V>);
    case 3: return reinterpret_cast<const void*>(&conv_step_kernel<IT, 3, V>);
    default: return reinterpret_cast<const void*>(&conv_step_kernel<IT, 4, V>);
  }
}

}  // namespace

const void* conv_kernel(int input_dtype, int width, bool vec) {
  if (input_dtype == RSM_BF16) return vec ? pick<uint16_t, 8>(width) : pick<uint16_t, 1>(width);
  return vec ? pick<float, 4>(width) : pick<float, 1>(width);
}

const void* conv_step_kernel_of(int input_dtype, int width, bool vec) {
  if (input_dtype == RSM_BF16) return vec ? pick_step<uint16_t, 8>(width) : pick_step<uint16_t, 1>(width);
  return vec ? pick_step<float, 4>(width) : pick_step<float, 1>(width);
}

}  // namespace hybrid
