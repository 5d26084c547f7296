// norm_kernel.cuh -- RMS norms fused with what stands around a block: the
// residual sum before it, the gate after it.
//   kind 0: r = residual + scale x,  out = r / sqrt(mean(r^2) + eps) w, r kept
//   kind 1: v = x silu(z),           out = v / sqrt(mean(v^2) + eps) w
//   kind 2: out = x / sqrt(mean(x^2) + eps) w silu(z)
// One CTA per (row, group); two passes over the group, sums in fp32.
#pragma once
#include <cuda_runtime.h>

#include "norm_params.h"
#include "rsm_formats.cuh"

namespace rmsnorm {

constexpr int kThreads = 256;

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = static_cast<uint16_t>(rsm::pack_bf16x2(v, 0.0f)); }

__device__ __forceinline__ float silu(float z) { return z / (1.0f + expf(-z)); }

template <int KIND, typename IT, typename RT>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Params p) {
  __shared__ float part[kThreads / 32];
  const int groups = p.dim / p.group;
  const int64_t row = blockIdx.x / groups;
  const int c0 = static_cast<int>(blockIdx.x % groups) * p.group;
  const IT* x = static_cast<const IT*>(p.x) + row * p.x_rs + c0;
  const RT* other = static_cast<const RT*>(p.other) + row * p.other_rs + c0;
  IT* out = static_cast<IT*>(p.out) + row * p.out_rs + c0;
  const float* w = p.weight + c0;
  auto value = [&](int i) {
    const float v = get(x + i);
    if constexpr (KIND == 0) return fmaf(p.scale, v, get(other + i));
    if constexpr (KIND == 1) return v * silu(get(other + i));
    return v;
  };
  float sum = 0.0f;
  for (int i = threadIdx.x; i < p.group; i += kThreads) {
    const float v = value(i);
    sum = fmaf(v, v, sum);
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) sum += part[i];
  const float r = 1.0f / sqrtf(sum / static_cast<float>(p.group) + p.eps);
  for (int i = threadIdx.x; i < p.group; i += kThreads) {
    const float v = value(i);
    if constexpr (KIND == 0) put(static_cast<RT*>(p.residual_out) + row * p.res_rs + c0 + i, v);
    float y = v * r * __ldg(w + i);
    if constexpr (KIND == 2) y *= silu(get(other + i));
    put(out + i, y);
  }
}

}  // namespace rmsnorm
