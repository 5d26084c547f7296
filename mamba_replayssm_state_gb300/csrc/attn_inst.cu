// Instances of the tiled attention kernel and its join.
#include "attn_tile_kernel.cuh"

namespace hybrid {

namespace {

struct Kernels {
  const void *tiles, *boxes, *join;
};

template <int DIM, int N>
Kernels bf16() {
  using Math = AttnBf16<DIM, N>;
  return {reinterpret_cast<const void*>(&attn_tile_kernel<Math, DIM, false>), reinterpret_cast<const void*>(&attn_tile_kernel<Math, DIM, true>),
          reinterpret_cast<const void*>(&attn_join_kernel<Math, DIM>)};
}

template <int DIM>
Kernels f32() {
  using Math = AttnF32<DIM>;
  return {reinterpret_cast<const void*>(&attn_tile_kernel<Math, DIM, false>), nullptr, reinterpret_cast<const void*>(&attn_join_kernel<Math, DIM>)};
}

template <int DIM>
Kernels pick_rows(int rows) {
  switch (rows) {
    case 8: return bf16<DIM, 1>();
    case 16: return bf16<DIM, 2>();
    case 24: return bf16<DIM, 3>();
    default: return bf16<DIM, 4>();
  }
}

Kernels pick(int input_dtype, int dim, int rows) {
  if (input_dtype == RSM_F32) return dim == 64 ? f32<64>() : f32<128>();
  if (dim == 256) return rows == 8 ? bf16<256, 1>() : bf16<256, 2>();
  return dim == 64 ? pick_rows<64>(rows) : pick_rows<128>(rows);
}

}  // namespace

const void* attn_tile_kernel_of(int input_dtype, int dim, int rows, bool boxes) {
  const Kernels k = pick(input_dtype, dim, rows);
  return boxes ? k.boxes : k.tiles;
}
const void* attn_join_kernel_of(int input_dtype, int dim, int rows) { return pick(input_dtype, dim, rows).join; }

}  // namespace hybrid
