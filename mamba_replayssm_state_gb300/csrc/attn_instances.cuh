// attn_instances.cuh -- the tiled attention's kernels for one type and head size, which a
// translation unit each compiles.
#pragma once
#include "attn_tile_kernel.cuh"

namespace hybrid {

template <typename Math, int DIM>
AttnKernels attn_kernels() {
  return {{reinterpret_cast<const void*>(&attn_tile_kernel<Math, DIM, AttnLoads::kRows>),
           reinterpret_cast<const void*>(&attn_tile_kernel<Math, DIM, AttnLoads::kBoxes>),
           reinterpret_cast<const void*>(&attn_tile_kernel<Math, DIM, AttnLoads::kGather>)},
          reinterpret_cast<const void*>(&attn_join_kernel<Math, DIM>)};
}

template <int DIM>
AttnKernels attn_bf16(int rows, bool three, bool low) {
  if constexpr (DIM < 256) {
    if (three && rows == 8) return attn_kernels<AttnBf16<DIM, 1, true, true>, DIM>();
    if (rows == 24) return low ? attn_kernels<AttnBf16<DIM, 3, false, true>, DIM>() : attn_kernels<AttnBf16<DIM, 3, false, false>, DIM>();
    if (rows == 32) return attn_kernels<AttnBf16<DIM, 4, false, false>, DIM>();
  }
  if constexpr (DIM > 64) {
    if (rows == 8) return attn_kernels<AttnBf16<DIM, 1, false, true>, DIM>();
  }
  return attn_kernels<AttnBf16<DIM, 2, DIM == 64, DIM < 256>, DIM>();
}

template <int DIM>
AttnKernels attn_f32(int rows) {
  if (rows == 1) return attn_kernels<AttnF32<DIM, 1>, DIM>();
  if (rows == 2) return attn_kernels<AttnF32<DIM, 2>, DIM>();
  if constexpr (DIM < 256) {
    if (rows == 8) return attn_kernels<AttnF32<DIM, 8>, DIM>();
  }
  return attn_kernels<AttnF32<DIM, 4>, DIM>();
}

}  // namespace hybrid
