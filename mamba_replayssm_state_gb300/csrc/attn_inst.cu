// Instances of the tiled attention kernel and its join.
#include "attn_tile_kernel.cuh"

namespace hybrid {

namespace {

struct Kernels {
  const void *tiles, *boxes, *join;
};

template <typename Math, int DIM>
Kernels kernels() {
  return {reinterpret_cast<const void*>(&attn_tile_kernel<Math, DIM, false>), reinterpret_cast<const void*>(&attn_tile_kernel<Math, DIM, true>),
          reinterpret_cast<const void*>(&attn_join_kernel<Math, DIM>)};
}

template <int DIM>
Kernels bf16(int rows) {
  if (rows == 8) return kernels<AttnBf16<DIM, 1>, DIM>();
  if constexpr (DIM < 256) {
    if (rows == 24) return kernels<AttnBf16<DIM, 3>, DIM>();
    if (rows == 32) return kernels<AttnBf16<DIM, 4>, DIM>();
  }
  return kernels<AttnBf16<DIM, 2>, DIM>();
}

template <int DIM>
Kernels f32(int rows) {
  if (rows == 1) return kernels<AttnF32<DIM, 1>, DIM>();
  if (rows == 2) return kernels<AttnF32<DIM, 2>, DIM>();
  if constexpr (DIM < 256) {
    if (rows == 8) return kernels<AttnF32<DIM, 8>, DIM>();
  }
  return kernels<AttnF32<DIM, 4>, DIM>();
}

Kernels pick(int input_dtype, int dim, int rows) {
  if (input_dtype == RSM_F32) return dim == 64 ? f32<64>(rows) : dim == 128 ? f32<128>(rows) : f32<256>(rows);
  return dim == 64 ? bf16<64>(rows) : dim == 128 ? bf16<128>(rows) : bf16<256>(rows);
}

}  // namespace

const void* attn_tile_kernel_of(int input_dtype, int dim, int rows, bool boxes) {
  const Kernels k = pick(input_dtype, dim, rows);
  return boxes ? k.boxes : k.tiles;
}
const void* attn_join_kernel_of(int input_dtype, int dim, int rows) { return pick(input_dtype, dim, rows).join; }

}  // namespace hybrid
