// Instances of the tiled attention kernel and its join.
#include "attn_tile_kernel.cuh"

namespace hybrid {

namespace {

struct Pair {
  const void *tiles, *join;
};

template <typename IT, int DIM, int M>
Pair pair() {
  return {reinterpret_cast<const void*>(&attn_tile_kernel<IT, DIM, M>), reinterpret_cast<const void*>(&attn_join_kernel<IT, DIM, M>)};
}

Pair pick(int input_dtype, int dim, int groups) {
  if (input_dtype == RSM_BF16) {
    if (dim == 64) return groups == 1 ? pair<uint16_t, 64, 1>() : pair<uint16_t, 64, 2>();
    if (dim == 128) return groups == 1 ? pair<uint16_t, 128, 1>() : pair<uint16_t, 128, 2>();
    if (dim == 256 && groups == 1) return pair<uint16_t, 256, 1>();
  } else if (groups == 1) {
    if (dim == 64) return pair<float, 64, 1>();
    if (dim == 128) return pair<float, 128, 1>();
  }
  return {nullptr, nullptr};
}

}  // namespace

const void* attn_tile_kernel_of(int input_dtype, int dim, int groups) { return pick(input_dtype, dim, groups).tiles; }
const void* attn_join_kernel_of(int input_dtype, int dim, int groups) { return pick(input_dtype, dim, groups).join; }

}  // namespace hybrid
