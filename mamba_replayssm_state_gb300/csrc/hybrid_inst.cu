// Instances of the rotary, page copy and plain attention kernels.
#include "attn_plain_kernel.cuh"
#include "page_copy_kernel.cuh"
#include "rotary_kernel.cuh"

namespace hybrid {

const void* rotary_kernel(int input_dtype, int at_once) {
  return input_dtype == RSM_F32 ? reinterpret_cast<const void*>(&rotary_append_kernel<float, 4>)
         : at_once == 8         ? reinterpret_cast<const void*>(&rotary_append_kernel<uint16_t, 8>)
                                : reinterpret_cast<const void*>(&rotary_append_kernel<uint16_t, 4>);
}

const void* rotary_token_kernel_of(int input_dtype, int at_once) {
  if (input_dtype == RSM_F32)
    return at_once == 4 ? reinterpret_cast<const void*>(&rotary_token_kernel<float, 4>) : reinterpret_cast<const void*>(&rotary_token_kernel<float, 1>);
  return at_once == 8   ? reinterpret_cast<const void*>(&rotary_token_kernel<uint16_t, 8>)
         : at_once == 4 ? reinterpret_cast<const void*>(&rotary_token_kernel<uint16_t, 4>)
                        : reinterpret_cast<const void*>(&rotary_token_kernel<uint16_t, 1>);
}

const void* copy_kernel() { return reinterpret_cast<const void*>(&copy_pages_kernel); }

const void* attn_plain_kernel(int input_dtype) {
  return input_dtype == RSM_BF16 ? reinterpret_cast<const void*>(&attn_plain_kernel_t<uint16_t>)
                                 : reinterpret_cast<const void*>(&attn_plain_kernel_t<float>);
}

}  // namespace hybrid
