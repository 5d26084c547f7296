// norm_kernel.cuh -- RMS norms fused with what stands around a block: the
// residual sum before it, the gate after it.
//   kind 0: r = residual + scale x,  out = r / sqrt(mean(r^2) + eps) w, r kept
//   kind 1: v = x silu(z),           out = v / sqrt(mean(v^2) + eps) w
//   kind 2: out = x / sqrt(mean(x^2) + eps) w silu(z)
// Sums and norms in fp32; r is normalised unrounded.
//
// Memory bounds it: each input read once, each output written once.  A group
// (a row's columns that share a norm) is held in registers from its one read to
// its one write, eight columns to a vector, V vectors to a thread, so that the
// reduction in between costs no second pass.  A warp takes a group of up to 32 V
// vectors, whole CTAs the longer ones.  Measured on a GB300: gated, 8192 rows of 16384
// bf16 columns, groups of 2048: 124 us, 6.5 TB/s; residual sum, 8192 rows of 4096
// columns, fp32 residuals: 62 us, 6.5 TB/s.  Groups whose columns are not whole
// aligned vectors, or more than 4096 of them, go through the two-pass kernel.
#pragma once
#include <cuda_runtime.h>

#include "norm_params.h"
#include "rsm_formats.cuh"

namespace rmsnorm {

constexpr int kPlainThreads = 256;

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = static_cast<uint16_t>(rsm::pack_bf16x2(v, 0.0f)); }

// silu(z); for bf16 inputs the exponential and the quotient are the fast ones,
// within 2^-17 for |z| < 80, far below the inputs' own 2^-8.
template <typename IT>
__device__ __forceinline__ float silu(float z) {
  if constexpr (sizeof(IT) == 2)
    return __fdividef(z, 1.0f + __expf(-z));
  else
    return z / (1.0f + expf(-z));
}

// eight columns
__device__ __forceinline__ void get8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void put8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(rsm::pack_bf16x2(v[0], v[1]), rsm::pack_bf16x2(v[2], v[3]),
                                            rsm::pack_bf16x2(v[4], v[5]), rsm::pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// eight columns as they lie in memory
template <typename T>
struct Raw {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = rsm::bf16lo(w[i]);
        v[2 * i + 1] = rsm::bf16hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[4 * i] = __uint_as_float(u[i].x), v[4 * i + 1] = __uint_as_float(u[i].y);
        v[4 * i + 2] = __uint_as_float(u[i].z), v[4 * i + 3] = __uint_as_float(u[i].w);
      }
    }
  }
};

// WARP: a group a warp, blockDim / 32 groups a CTA at a time; otherwise a group a CTA.
// LOOP: the CTAs stay, and ask for their next group before they are done with one.
// (An output may be an input's own place: a group is read before it is written.)
template <int KIND, typename IT, typename RT, int V, bool WARP, bool LOOP>
__global__ void __launch_bounds__(1024) norm_vec_kernel(const __grid_constant__ Params p) {
  __shared__ float part[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int threads = WARP ? 32 : blockDim.x, tid = WARP ? lane : threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (WARP ? blockDim.x >> 5 : 1);
  const int64_t units = p.rows * p.groups;
  int64_t unit = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  if (WARP && unit >= units) return;
  Raw<IT> x[V];
  Raw<RT> other[V];
  auto ask = [&](int64_t at) {
    const int64_t row = at / p.groups;
    const int c0 = static_cast<int>(at - row * p.groups) * p.group;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (tid + v * threads);
      if (c < p.group) {
        x[v].load(static_cast<const IT*>(p.x) + row * p.x_rs + c0 + c);
        other[v].load(static_cast<const RT*>(p.other) + row * p.other_rs + c0 + c);
      }
    }
  };
  ask(unit);
  for (int turn = 0;; turn ^= 1) {
    const int64_t row = unit / p.groups;
    const int c0 = static_cast<int>(unit - row * p.groups) * p.group;
    float val[V][8], gate[KIND == 2 ? V : 1][8], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (8 * (tid + v * threads) >= p.group) break;
      float o[8];
      x[v].values(val[v]);
      other[v].values(o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (KIND == 0) val[v][i] = fmaf(p.scale, val[v][i], o[i]);
        if constexpr (KIND == 1) val[v][i] *= silu<IT>(o[i]);
        if constexpr (KIND == 2) gate[v][i] = silu<IT>(o[i]);
        sum = fmaf(val[v][i], val[v][i], sum);
      }
    }
    const int64_t next = unit + step;
    if (LOOP && next < units) ask(next);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if constexpr (!WARP) {  // two places in turn: one barrier a group is enough
      if (lane == 0) part[turn][warp] = sum;
      __syncthreads();
      sum = lane < (threads >> 5) ? part[turn][lane] : 0.0f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    const float r = rsqrtf(sum / static_cast<float>(p.group) + p.eps);
    IT* out = static_cast<IT*>(p.out) + row * p.out_rs + c0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (tid + v * threads);
      if (c >= p.group) break;
      float w[8];
      get8(p.weight + c0 + c, w);
      if constexpr (KIND == 0) put8(static_cast<RT*>(p.residual_out) + row * p.res_rs + c0 + c, val[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] *= val[v][i] * r;
        if constexpr (KIND == 2) w[i] *= gate[v][i];
      }
      put8(out + c, w);
    }
    if (!LOOP || next >= units) return;
    unit = next;
  }
}

// Any size, stride and alignment: a group a CTA, read twice.
template <int KIND, typename IT, typename RT>
__global__ void __launch_bounds__(kPlainThreads) norm_plain_kernel(const __grid_constant__ Params p) {
  __shared__ float part[kPlainThreads / 32];
  const int64_t row = blockIdx.x / static_cast<uint32_t>(p.groups);
  const int c0 = static_cast<int>(blockIdx.x % static_cast<uint32_t>(p.groups)) * p.group;
  const IT* x = static_cast<const IT*>(p.x) + row * p.x_rs + c0;
  const RT* other = static_cast<const RT*>(p.other) + row * p.other_rs + c0;
  IT* out = static_cast<IT*>(p.out) + row * p.out_rs + c0;
  const float* w = p.weight + c0;
  auto value = [&](int i) {
    const float v = get(x + i);
    if constexpr (KIND == 0) return fmaf(p.scale, v, get(other + i));
    if constexpr (KIND == 1) return v * silu<IT>(get(other + i));
    return v;
  };
  float sum = 0.0f;
  for (int i = threadIdx.x; i < p.group; i += kPlainThreads) {
    const float v = value(i);
    sum = fmaf(v, v, sum);
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int i = 0; i < kPlainThreads / 32; ++i) sum += part[i];
  const float r = rsqrtf(sum / static_cast<float>(p.group) + p.eps);
  for (int i = threadIdx.x; i < p.group; i += kPlainThreads) {
    const float v = value(i);
    if constexpr (KIND == 0) put(static_cast<RT*>(p.residual_out) + row * p.res_rs + c0 + i, v);
    float y = v * r * __ldg(w + i);
    if constexpr (KIND == 2) y *= silu<IT>(get(other + i));
    put(out + i, y);
  }
}

}  // namespace rmsnorm
