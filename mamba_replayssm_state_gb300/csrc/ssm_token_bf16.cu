// Instances of the new-token kernel, bf16 inputs.
#include "ssm_token_kernel.cuh"

namespace ssm {

namespace {
template <int SF>
const void* pick_step(int mode) {
  if constexpr (SF == RSM_F32 || SF == RSM_BF16 || SF == RSM_F16)
    return mode == 1 ? reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 1>)
                     : reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 2>);
  return nullptr;
}

// The ring form is on the tensor cores wherever the state's elements are exact in bf16.
template <int SF>
const void* pick(int mode) {
  if constexpr (SF == RSM_BF16 || SF == RSM_I8 || SF == RSM_FP8_E4M3)
    return mode == 0 ? nullptr : mode == 3 ? reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 3>)
                     : mode == 4  ? reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 4>)
                                  : pick_step<SF>(mode);
  else
    return mode == 0 ? reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 0>) : mode >= 3 ? nullptr : pick_step<SF>(mode);
}
}  // namespace

const void* token_kernel_bf16(int state_dtype, int mode) {
  switch (state_dtype) {
    case RSM_F32: return pick<RSM_F32>(mode);
    case RSM_BF16: return pick<RSM_BF16>(mode);
    case RSM_F16: return pick<RSM_F16>(mode);
    case RSM_I8: return pick<RSM_I8>(mode);
    case RSM_FP8_E4M3: return pick<RSM_FP8_E4M3>(mode);
    default: return nullptr;
  }
}

uint32_t token_smem(int mode, int input_bytes, int heads, int fresh, int all) {
  return tok_layout(mode, input_bytes, heads, fresh, all).bytes;
}

}  // namespace ssm
