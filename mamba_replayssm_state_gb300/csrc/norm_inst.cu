// Instances of the norm kernels.
#include "norm_kernel.cuh"

namespace rmsnorm {

namespace {

template <int KIND, typename IT, typename RT>
const void* pick(int vectors, bool warp) {
  if (vectors == 0) return reinterpret_cast<const void*>(&norm_plain_kernel<KIND, IT, RT>);
  if (vectors == 1)
    return warp ? reinterpret_cast<const void*>(&norm_vec_kernel<KIND, IT, RT, 1, true>)
                : reinterpret_cast<const void*>(&norm_vec_kernel<KIND, IT, RT, 1, false>);
  if (vectors == 2)
    return warp ? reinterpret_cast<const void*>(&norm_vec_kernel<KIND, IT, RT, 2, true>)
                : reinterpret_cast<const void*>(&norm_vec_kernel<KIND, IT, RT, 2, false>);
  return warp ? nullptr : reinterpret_cast<const void*>(&norm_vec_kernel<KIND, IT, RT, 4, false>);
}

template <int KIND>
const void* pick_type(int input_dtype, int other_dtype, int vectors, bool warp) {
  const bool ib = input_dtype == RSM_BF16, ob = other_dtype == RSM_BF16;
  if (ib && ob) return pick<KIND, uint16_t, uint16_t>(vectors, warp);
  if (!ib && !ob) return pick<KIND, float, float>(vectors, warp);
  if constexpr (KIND == 0) return ib ? pick<0, uint16_t, float>(vectors, warp) : pick<0, float, uint16_t>(vectors, warp);
  return nullptr;
}

}  // namespace

const void* kernel(int kind, int input_dtype, int other_dtype, int vectors, bool warp) {
  switch (kind) {
    case 0: return pick_type<0>(input_dtype, other_dtype, vectors, warp);
    case 1: return pick_type<1>(input_dtype, other_dtype, vectors, warp);
    default: return pick_type<2>(input_dtype, other_dtype, vectors, warp);
  }
}

}  // namespace rmsnorm
