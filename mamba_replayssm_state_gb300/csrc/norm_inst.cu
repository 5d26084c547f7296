// Instances of the norm kernels.
#include "norm_kernel.cuh"

namespace rmsnorm {

namespace {

template <int KIND, typename IT, typename RT, int V, bool WARP>
const void* vec(bool loop) {
  if constexpr (can_loop(KIND, sizeof(IT) == 2, V)) {
    if (loop) return reinterpret_cast<const void*>(&norm_vec_kernel<KIND, IT, RT, V, WARP, true>);
  }
  return reinterpret_cast<const void*>(&norm_vec_kernel<KIND, IT, RT, V, WARP, false>);
}

template <int KIND, typename IT, typename RT>
const void* pick(int vectors, bool warp, bool loop) {
  if (vectors == 0) return reinterpret_cast<const void*>(&norm_plain_kernel<KIND, IT, RT>);
  if (vectors == 1) return warp ? vec<KIND, IT, RT, 1, true>(loop) : vec<KIND, IT, RT, 1, false>(loop);
  if (vectors == 2) return warp ? vec<KIND, IT, RT, 2, true>(loop) : vec<KIND, IT, RT, 2, false>(loop);
  return warp ? nullptr : vec<KIND, IT, RT, 4, false>(loop);
}

template <int KIND>
const void* pick_type(int input_dtype, int other_dtype, int vectors, bool warp, bool loop) {
  const bool ib = input_dtype == RSM_BF16, ob = other_dtype == RSM_BF16;
  if (ib && ob) return pick<KIND, uint16_t, uint16_t>(vectors, warp, loop);
  if (!ib && !ob) return pick<KIND, float, float>(vectors, warp, loop);
  if constexpr (KIND == 0) return ib ? pick<0, uint16_t, float>(vectors, warp, loop) : pick<0, float, uint16_t>(vectors, warp, loop);
  return nullptr;
}

}  // namespace

const void* kernel(int kind, int input_dtype, int other_dtype, int vectors, bool warp, bool loop) {
  switch (kind) {
    case 0: return pick_type<0>(input_dtype, other_dtype, vectors, warp, loop);
    case 1: return pick_type<1>(input_dtype, other_dtype, vectors, warp, loop);
    default: return pick_type<2>(input_dtype, other_dtype, vectors, warp, loop);
  }
}

}  // namespace rmsnorm
