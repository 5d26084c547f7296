// hybrid_device.cuh -- what the kernels of hybrid stacks share: rows of bf16 or
// fp32 values, the sequences of a packed call, the status word.
#pragma once
#include <cuda_runtime.h>

#include "hybrid_params.h"
#include "rsm_formats.cuh"
#include "ssm_sequences.h"

namespace hybrid {

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bits) {
  if (status != nullptr) atomicOr(status, bits);
}

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = static_cast<uint16_t>(rsm::pack_bf16x2(v, 0.0f)); }

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// V neighbouring values as they lie in memory: one, 8 bytes or 16.
template <typename T, int V>
struct alignas(V * sizeof(T)) Row {
  static constexpr int kBytes = V * static_cast<int>(sizeof(T));
  static_assert(V == 1 || kBytes == 8 || kBytes == 16);
  T v[V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1)
      v[0] = *p;
    else if constexpr (kBytes == 8)
      *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
    else
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V == 1)
      *p = v[0];
    else if constexpr (kBytes == 8)
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v);
    else
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = T(0);
  }
  __device__ __forceinline__ void values(float (&f)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = v[i];
    } else if constexpr (V == 1) {
      f[0] = get(v);
    } else {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) f[2 * i] = rsm::bf16lo(w[i]), f[2 * i + 1] = rsm::bf16hi(w[i]);
    }
  }
  __device__ __forceinline__ void round(const float (&f)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = f[i];
    } else if constexpr (V == 1) {
      put(v, f[0]);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = rsm::pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
  }
};

// How many of a packed call's sequences come before the first at which cu_seqlens
// goes back: the others are skipped.  For a whole CTA, with a barrier; `report`: flags what is
// wrong with any of them.
__device__ __forceinline__ int live_sequences(const int32_t* cu, int seqs, int64_t tokens, uint32_t* status, bool report) {
  __shared__ int live;
  if (threadIdx.x == 0) live = seqs;
  __syncthreads();
  bool bad = false;
  for (int s = threadIdx.x; s < seqs; s += blockDim.x) {
    const int a = cu[s], b = cu[s + 1];
    if (ssm::goes_back(a, b)) atomicMin(&live, s);
    bad |= !ssm::within(a, b, tokens);
  }
  if (report && bad) flag(status, RSM_STATUS_BAD_SEQUENCE);
  __syncthreads();
  return live;
}

// The same by one warp.
__device__ __forceinline__ int live_sequences_warp(const int32_t* cu, int seqs, int64_t tokens, uint32_t* status, bool report) {
  int live = seqs;
  bool bad = false;
  for (int s = threadIdx.x & 31; s < seqs; s += 32) {
    const int a = cu[s], b = cu[s + 1];
    if (ssm::goes_back(a, b)) live = min(live, s);
    bad |= !ssm::within(a, b, tokens);
  }
  if (report && bad) flag(status, RSM_STATUS_BAD_SEQUENCE);
#pragma unroll
  for (int o = 16; o; o >>= 1) live = min(live, __shfl_xor_sync(0xFFFFFFFFu, live, o));
  return live;
}

// The first of `live` sequences that ends after token t (`live`: none does).
__device__ __forceinline__ int sequence_at(const int32_t* cu, int live, int64_t t) {
  int lo = 0, hi = live;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (cu[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

}  // namespace hybrid
