// page_copy_kernel.cuh -- pages of all pools copied in one launch.  Memory bounds it:
// each page read once and written once.  A CTA takes kCopyBytes of one page, so the
// pairs and the pools are divided among CTAs and the addresses looked up once a CTA.
// Measured on a GB300: 61 pages of 32 KB in each of 96 pools, 384 MB read and written, 51 us (some of
// the sources repeat, and come from the L2).
#pragma once
#include "hybrid_device.cuh"

namespace hybrid {

template <typename T>
__device__ __forceinline__ void copy_bytes(char* to, const char* from, int64_t bytes) {
  constexpr int U = kCopyBytes / kCopyThreads / 16;
  const int64_t n = bytes / static_cast<int64_t>(sizeof(T));
  for (int64_t i = threadIdx.x; i < n; i += kCopyThreads * U) {
    T v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * kCopyThreads < n) v[u] = reinterpret_cast<const T*>(from)[i + u * kCopyThreads];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * kCopyThreads < n) reinterpret_cast<T*>(to)[i + u * kCopyThreads] = v[u];
  }
  for (int64_t i = n * static_cast<int64_t>(sizeof(T)) + threadIdx.x; i < bytes; i += kCopyThreads) to[i] = from[i];
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  const int64_t pieces = (p.page_bytes + kCopyBytes - 1) / kCopyBytes;
  const int64_t unit = blockIdx.x / pieces, begin = (blockIdx.x - unit * pieces) * kCopyBytes;
  const int64_t pool = unit / p.pairs, pair = unit - pool * p.pairs;
  const int src = p.src[pair], dst = p.dst[pair];
  if (src < 0 || dst < 0 || src == dst) return;
  if (src >= p.pages || dst >= p.pages) {
    if (threadIdx.x == 0 && unit < p.pairs && begin == 0) flag(p.status, RSM_STATUS_BAD_PAGE);
    return;
  }
  char* const base = reinterpret_cast<char*>(p.ptrs[pool]);
  const int64_t stride = p.strides[pool] * p.esize;
  const char* from = base + src * stride + begin;
  char* to = base + dst * stride + begin;
  const int64_t bytes = min(p.page_bytes - begin, static_cast<int64_t>(kCopyBytes));
  const uintptr_t both = reinterpret_cast<uintptr_t>(from) | reinterpret_cast<uintptr_t>(to);
  if (both % 16 == 0)
    copy_bytes<uint4>(to, from, bytes);
  else if (both % 4 == 0)
    copy_bytes<uint32_t>(to, from, bytes);
  else
    copy_bytes<char>(to, from, bytes);
}

}  // namespace hybrid
