// Instances of the new-token kernel, bf16 inputs.
#include "ssm_token_kernel.cuh"

namespace ssm {

namespace {
template <int SF>
const void* pick(int mode) {
  if (mode == 3) return reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 3>);
  if (mode == 4) return reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 4>);
  if constexpr (SF == RSM_F32 || SF == RSM_BF16 || SF == RSM_F16) {
    if (mode == 1) return reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 1>);
    if (mode == 2) return reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 2>);
    if (mode == 5) return reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 5>);
  }
  if constexpr (SF == RSM_F16) return reinterpret_cast<const void*>(&ssm_token_kernel<uint16_t, SF, 0>);
  return nullptr;
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
