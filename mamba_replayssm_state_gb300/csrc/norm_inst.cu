// Instances of the norm kernels.
#include "norm_kernel.cuh"

namespace rmsnorm {

const void* kernel(int kind, int input_dtype, int other_dtype) {
#define NORM_PICK(K, IC, IT, OC, OT) \
  if (kind == K && input_dtype == IC && other_dtype == OC) return reinterpret_cast<const void*>(&norm_kernel<K, IT, OT>);
  NORM_PICK(0, RSM_BF16, uint16_t, RSM_BF16, uint16_t)
  NORM_PICK(0, RSM_BF16, uint16_t, RSM_F32, float)
  NORM_PICK(0, RSM_F32, float, RSM_BF16, uint16_t)
  NORM_PICK(0, RSM_F32, float, RSM_F32, float)
  NORM_PICK(1, RSM_BF16, uint16_t, RSM_BF16, uint16_t)
  NORM_PICK(1, RSM_F32, float, RSM_F32, float)
  NORM_PICK(2, RSM_BF16, uint16_t, RSM_BF16, uint16_t)
  NORM_PICK(2, RSM_F32, float, RSM_F32, float)
#undef NORM_PICK
  return nullptr;
}

}  // namespace rmsnorm
