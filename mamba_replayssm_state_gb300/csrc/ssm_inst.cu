// Instances of the sequential linear-attention kernel.
#include "ssm_seq_kernel.cuh"

namespace ssm {

const void* token_kernel_bf16(int state_dtype, int mode);  // ssm_token_bf16.cu
const void* token_kernel_f32(int state_dtype, int mode);   // ssm_token_f32.cu

const void* token_kernel(int input_dtype, int state_dtype, int mode) {
  return input_dtype == RSM_BF16 ? token_kernel_bf16(state_dtype, mode) : token_kernel_f32(state_dtype, mode);
}

namespace {
template <typename IT>
const void* pick(int dim, int dstate, int* threads) {
  *threads = 4 * dim;
  if (dim == 16 && dstate == 16) return reinterpret_cast<const void*>(&ssm_seq_kernel<IT, 16, 16>);
  if (dim == 64 && dstate == 64) return reinterpret_cast<const void*>(&ssm_seq_kernel<IT, 64, 64>);
  if (dim == 64 && dstate == 128) return reinterpret_cast<const void*>(&ssm_seq_kernel<IT, 64, 128>);
  return nullptr;
}
}  // namespace

const void* seq_kernel(int input_dtype, int dim, int dstate, int* threads) {
  return input_dtype == RSM_BF16 ? pick<uint16_t>(dim, dstate, threads) : pick<float>(dim, dstate, threads);
}

}  // namespace ssm
