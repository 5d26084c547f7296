// Instances of the new-token kernel, f32 inputs.
#include "ssm_token_kernel.cuh"

namespace ssm {

namespace {
template <int SF>
const void* pick(int mode) {
  if (mode >= 3) return nullptr;
  if (mode == 0) return reinterpret_cast<const void*>(&ssm_token_kernel<float, SF, 0>);
  if constexpr (SF == RSM_F32 || SF == RSM_BF16 || SF == RSM_F16)
    return mode == 1 ? reinterpret_cast<const void*>(&ssm_token_kernel<float, SF, 1>)
                     : reinterpret_cast<const void*>(&ssm_token_kernel<float, SF, 2>);
  return nullptr;
}
}  // namespace

const void* token_kernel_f32(int state_dtype, int mode) {
  switch (state_dtype) {
    case RSM_F32: return pick<RSM_F32>(mode);
    case RSM_BF16: return pick<RSM_BF16>(mode);
    case RSM_F16: return pick<RSM_F16>(mode);
    case RSM_I8: return pick<RSM_I8>(mode);
    case RSM_FP8_E4M3: return pick<RSM_FP8_E4M3>(mode);
    default: return nullptr;
  }
}

}  // namespace ssm
