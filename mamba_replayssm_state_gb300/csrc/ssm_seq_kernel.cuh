// ssm_seq_kernel.cuh -- linear attention with a decay for each head, in the
// order of its definition: for every token
//   S = exp(dt A) S + (dt x) (x) B,   y = S C + D x.
//
// One CTA holds one head's state of one sequence or request in registers, as
// fp32: four threads to a dim row, each with every fourth float4 of the row's
// dstate columns, so that a warp's reads of B and C broadcast four float4s.
// Tokens are staged in shared memory as fp32, kSeqTokens at a time.  A row's
// output is a sum over its four threads (two shuffles).
//
// It serves every size, type and stride: prompts whose inputs are fp32 or
// whose state is not 64 x 128, unaligned slices, and the shortest.  What bounds it is
// the way through a token, 0.75 us (one sequence of 2048 tokens, 80 heads of 64 x 128:
// 1561 us): 2 dim dstate FMAs on one SM with nothing to overlap them but other heads.
#pragma once
#include <cuda_runtime.h>

#include "rsm_formats.cuh"
#include "ssm_params.h"

namespace ssm {

__device__ __forceinline__ float load_in(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_in(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}
__device__ __forceinline__ void store_in(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_in(uint16_t* p, float v) {
  *p = static_cast<uint16_t>(rsm::pack_bf16x2(v, 0.0f) & 0xFFFFu);
}

// The lo half of values split into bf16 hi + lo, from value - hi.  Where hi is infinite that
// is no number, and takes an infinite sum with it: lo is kept within 2^119, which the
// remainder of a finite value never exceeds.
__device__ __forceinline__ uint32_t bounded_lo(uint32_t lo) {
  uint32_t v;
  asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(lo), "r"(0x7B007B00u));
  return v;
}

__device__ __forceinline__ float load_state(const void* base, int64_t at, int fmt) {
  switch (fmt) {
    case RSM_F32: return static_cast<const float*>(base)[at];
    case RSM_BF16: return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at]) << 16);
    case RSM_F16: return __half2float(static_cast<const __half*>(base)[at]);
    case RSM_I8: return static_cast<float>(static_cast<const int8_t*>(base)[at]);
    default: return rsm::e4m3x2_to_f32(static_cast<const uint8_t*>(base)[at]).x;
  }
}

__device__ __forceinline__ void store_state(void* base, int64_t at, int fmt, float v) {
  switch (fmt) {
    case RSM_F32: static_cast<float*>(base)[at] = v; break;
    case RSM_BF16: static_cast<uint16_t*>(base)[at] = static_cast<uint16_t>(rsm::pack_bf16x2(v, 0.0f)); break;
    default: static_cast<__half*>(base)[at] = __float2half_rn(v); break;
  }
}

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bits) {
  if (status != nullptr && bits != 0u) atomicOr(status, bits);
}

// A slot of a table: -1 for the pad, for one out of range (flagged) and where there is no table.
__device__ __forceinline__ int slot_of(const Params& p, const int32_t* table, int unit, bool say) {
  if (table == nullptr) return -1;
  const int s = __ldg(table + unit);
  if (s == p.pad) return -1;
  if (s < 0 || s >= p.num_slots) {
    if (say) flag(p.status, RSM_STATUS_BAD_SLOT);
    return -1;
  }
  return s;
}

template <typename IT, int D, int N>
__global__ void __launch_bounds__(4 * D) ssm_seq_kernel(const __grid_constant__ Params p) {
  constexpr int kThreads = 4 * D;
  constexpr int V = N / 16;  // float4s of a thread
  __shared__ __align__(16) float sx[kSeqTokens][D];
  __shared__ __align__(16) float sB[kSeqTokens][N];
  __shared__ __align__(16) float sC[kSeqTokens][N];
  __shared__ float sdt[kSeqTokens];
  const int tid = threadIdx.x, d = tid >> 2, q = tid & 3;
  const int unit = static_cast<int>(blockIdx.x / static_cast<uint32_t>(p.H));
  const int h = static_cast<int>(blockIdx.x % static_cast<uint32_t>(p.H));
  const int g = h / (p.H / p.G);
  const bool say = h == 0 && tid == 0;

  int64_t t0 = 0;
  int n_new = p.window, n_ring = 0, ring0 = 0;
  int src = slot_of(p, p.src, unit, say), dst = slot_of(p, p.dst, unit, say);
  bool live = true;
  if (p.mode == kPrefill) {
    t0 = __ldg(p.cu_seqlens + unit);
    const int64_t t1 = __ldg(p.cu_seqlens + unit + 1);
    int runs = within(static_cast<int>(t0), static_cast<int>(t1), p.tokens) ? 1 : 0;
    if (unit > 0) {  // nor does cu_seqlens go back before it
      for (int i = tid; i < unit; i += kThreads) runs &= goes_back(__ldg(p.cu_seqlens + i), __ldg(p.cu_seqlens + i + 1)) ? 0 : 1;
      runs = __syncthreads_and(runs);
    }
    if (runs == 0) {
      if (say) flag(p.status, RSM_STATUS_BAD_SEQUENCE);
      return;
    }
    n_new = static_cast<int>(t1 - t0);
  } else {
    live = src >= 0;
    if (p.mode == kStep) {
      if (p.dst == nullptr) dst = src;
    } else if (live) {
      ring0 = __ldg(p.ring_start + unit);
      n_ring = __ldg(p.ring_len + unit);
      uint32_t bad = 0;
      if (ring0 < 0 || ring0 >= p.R) bad |= RSM_STATUS_BAD_RING_START;
      if (n_ring < 0 || n_ring > p.R - n_new || n_ring > 64 - n_new) bad |= RSM_STATUS_BAD_PREFIX_LEN;
      if (say) flag(p.status, bad);
      live = bad == 0;
    }
  }
  const int64_t batch = p.mode == kPrefill ? 0 : unit;
  const IT* x = static_cast<const IT*>(p.x) + batch * p.x_bs + t0 * p.x_ts + static_cast<int64_t>(h) * D;
  const IT* B = static_cast<const IT*>(p.B) + batch * p.B_bs + t0 * p.B_ts + static_cast<int64_t>(g) * N;
  const IT* C = static_cast<const IT*>(p.C) + batch * p.C_bs + t0 * p.C_ts + static_cast<int64_t>(g) * N;
  const float* dt = p.dt + batch * p.dt_bs + t0 * p.dt_ts + h;
  IT* out = static_cast<IT*>(p.out) + batch * p.out_bs + t0 * p.out_ts + static_cast<int64_t>(h) * D;
  if (!live) {
    for (int64_t i = tid; i < static_cast<int64_t>(n_new) * D; i += kThreads) store_in(out + (i / D) * p.out_ts + i % D, 0.0f);
    return;
  }

  float4 S[V];
  const int64_t tile = (static_cast<int64_t>(h) * D + d) * N;
  if (src >= 0) {
    const int64_t at = src * p.state_ss + tile;
    const float sc = p.scale != nullptr ? __ldg(p.scale + src * p.scale_ss + static_cast<int64_t>(h) * D + d) : 1.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int64_t e = at + 4 * (q + 4 * k);
      S[k] = make_float4(sc * load_state(p.state, e, p.state_dtype), sc * load_state(p.state, e + 1, p.state_dtype),
                         sc * load_state(p.state, e + 2, p.state_dtype), sc * load_state(p.state, e + 3, p.state_dtype));
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) S[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  const float A = __ldg(p.A + h);
  const float skip = p.D != nullptr ? __ldg(p.D + h) : 0.0f;

  const int total = n_ring + n_new;
  for (int c0 = 0; c0 < total; c0 += kSeqTokens) {
    const int n = min(kSeqTokens, total - c0);
    for (int i = tid; i < n * (D + N); i += kThreads) {
      const int t = i / (D + N), k = i % (D + N), tok = c0 + t;
      float v;
      if (tok < n_ring) {
        const int64_t row = (ring0 + tok) % p.R;
        v = k < D ? load_in(static_cast<const IT*>(p.x_cache) + src * p.xc_ss + (row * p.H + h) * D + k)
                  : load_in(static_cast<const IT*>(p.B_cache) + src * p.Bc_ss + (row * p.G + g) * N + (k - D));
      } else {
        const int64_t r = tok - n_ring;
        v = k < D ? load_in(x + r * p.x_ts + k) : load_in(B + r * p.B_ts + (k - D));
      }
      if (k < D)
        sx[t][k] = v;
      else
        sB[t][k - D] = v;
    }
    for (int i = tid; i < n * N; i += kThreads) {
      const int t = i / N, k = i % N, r = c0 + t - n_ring;
      if (r >= 0) sC[t][k] = load_in(C + static_cast<int64_t>(r) * p.C_ts + k);
    }
    if (tid < n) {
      const int tok = c0 + tid;
      sdt[tid] = tok < n_ring ? __ldg(p.dt_cache + src * p.dtc_ss + static_cast<int64_t>((ring0 + tok) % p.R) * p.H + h)
                              : __ldg(dt + static_cast<int64_t>(tok - n_ring) * p.dt_ts);
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float step = sdt[t], a = expf(step * A), xv = sx[t][d], w = step * xv;
      const float4* Bt = reinterpret_cast<const float4*>(sB[t]) + q;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float4 b = Bt[4 * k];
        S[k].x = fmaf(a, S[k].x, w * b.x);
        S[k].y = fmaf(a, S[k].y, w * b.y);
        S[k].z = fmaf(a, S[k].z, w * b.z);
        S[k].w = fmaf(a, S[k].w, w * b.w);
      }
      const int r = c0 + t - n_ring;
      if (r < 0) continue;
      const float4* Ct = reinterpret_cast<const float4*>(sC[t]) + q;
      float y = 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float4 c = Ct[4 * k];
        y = fmaf(S[k].x, c.x, fmaf(S[k].y, c.y, fmaf(S[k].z, c.z, fmaf(S[k].w, c.w, y))));
      }
      y += __shfl_xor_sync(0xFFFFFFFFu, y, 1);
      y += __shfl_xor_sync(0xFFFFFFFFu, y, 2);
      if (q == 0) store_in(out + static_cast<int64_t>(r) * p.out_ts + d, fmaf(skip, xv, y));
    }
    if (p.mode == kDecode) {
      // the new tokens join the ring: this head's x and dt, and B once a group
      for (int t = 0; t < n; ++t) {
        const int r = c0 + t - n_ring;
        if (r < 0) continue;
        const int64_t row = (ring0 + c0 + t) % p.R;
        IT* xc = static_cast<IT*>(p.x_cache) + src * p.xc_ss + (row * p.H + h) * D;
        for (int k = tid; k < D; k += kThreads) store_in(xc + k, sx[t][k]);
        if (h % (p.H / p.G) == 0) {
          IT* Bc = static_cast<IT*>(p.B_cache) + src * p.Bc_ss + (row * p.G + g) * N;
          for (int k = tid; k < N; k += kThreads) store_in(Bc + k, sB[t][k]);
        }
        if (tid == 0) p.dt_cache[src * p.dtc_ss + row * p.H + h] = sdt[t];
      }
    }
    __syncthreads();
  }
  if (p.mode != kDecode && dst >= 0) {
    const int64_t at = dst * p.state_ss + tile;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int64_t e = at + 4 * (q + 4 * k);
      store_state(p.state, e, p.state_dtype, S[k].x);
      store_state(p.state, e + 1, p.state_dtype, S[k].y);
      store_state(p.state, e + 2, p.state_dtype, S[k].z);
      store_state(p.state, e + 3, p.state_dtype, S[k].w);
    }
  }
}

}  // namespace ssm
