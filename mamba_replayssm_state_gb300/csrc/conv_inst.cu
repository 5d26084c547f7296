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

template <typename IT, int V, int N>
const void* pick_step(int width) {
  switch (width) {
    case 2: return reinterpret_cast<const void*>(&conv_step_kernel<IT, 2, V, N>);
    case 3: return reinterpret_cast<const void*>(&conv_step_kernel<IT, 3, V, N>);
    default: return reinterpret_cast<const void*>(&conv_step_kernel<IT, 4, V, N>);
  }
}

}  // namespace

const void* conv_kernel(int input_dtype, int width, bool vec) {
  if (input_dtype == RSM_BF16) return vec ? pick<uint16_t, 8>(width) : pick<uint16_t, 1>(width);
  return vec ? pick<float, 4>(width) : pick<float, 1>(width);
}

const void* conv_step_kernel(int input_dtype, int width, bool vec, int requests) {
  if (input_dtype == RSM_BF16) {
    if (!vec) return pick_step<uint16_t, 1, 1>(width);
    return requests == 1 ? pick_step<uint16_t, 8, 1>(width) : pick_step<uint16_t, 8, 2>(width);
  }
  if (!vec) return pick_step<float, 1, 1>(width);
  return requests == 1 ? pick_step<float, 4, 1>(width) : pick_step<float, 4, 2>(width);
}

}  // namespace hybrid
