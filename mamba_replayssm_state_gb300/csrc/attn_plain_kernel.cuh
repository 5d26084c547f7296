// attn_plain_kernel.cuh -- attention over pages for any head size up to 256, stride and
// alignment: a CTA a new token and head, its warps taking the tokens of the cache in
// turn, each with a running maximum and sum of its own; all arithmetic fp32.
#pragma once
#include "hybrid_device.cuh"

namespace hybrid {

// The request's tokens, or 0 where it is skipped.
__device__ __forceinline__ int64_t request_tokens(const rsm_pages& pg, int64_t b, int window, uint32_t* status, bool report) {
  const int64_t len = pg.lengths[b];
  if (len >= window && len <= static_cast<int64_t>(pg.table_width) * pg.page_size) return len;
  if (report && len != 0) flag(status, RSM_STATUS_BAD_POSITION);
  return 0;
}

template <typename IT>
__global__ void __launch_bounds__(kAttnPlainThreads) attn_plain_kernel_t(const __grid_constant__ AttnParams p) {
  constexpr int kWarps = kAttnPlainThreads / 32, kMax = 8;  // columns of a lane
  __shared__ float acc_s[kWarps][32 * kMax], m_s[kWarps], l_s[kWarps];
  const rsm_pages& pg = p.pages;
  const int64_t bt = blockIdx.x / static_cast<uint32_t>(p.H), b = bt / p.window, t = bt - b * p.window;
  const int h = static_cast<int>(blockIdx.x - bt * p.H), g = h / p.per;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool report = h == 0 && t == 0 && lane == 0;
  const int64_t len = request_tokens(pg, b, p.window, p.status, report && warp == 0), seen = len == 0 ? 0 : len - p.window + t + 1;
  const IT* q = static_cast<const IT*>(p.q) + b * p.q_bs + t * p.q_ts + static_cast<int64_t>(h) * p.dim;
  float qv[kMax], acc[kMax], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < kMax; ++i) {
    const int c = lane + 32 * i;
    qv[i] = c < p.dim ? get(q + c) : 0.0f;
    acc[i] = 0.0f;
  }
  for (int64_t at = warp; at < seen; at += kWarps) {
    const int page = pg.page_table[b * pg.table_stride + at / pg.page_size];
    if (page < 0 || page >= pg.num_pages) {
      if (g * p.per == h && lane == 0) flag(p.status, RSM_STATUS_BAD_PAGE);
      continue;
    }
    const int64_t row = at % pg.page_size;
    const IT* k = static_cast<const IT*>(pg.k) + page * pg.k_page_stride + row * pg.k_row_stride + g * pg.k_head_stride;
    const IT* v = static_cast<const IT*>(pg.v) + page * pg.v_page_stride + row * pg.v_row_stride + g * pg.v_head_stride;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kMax; ++i)
      if (lane + 32 * i < p.dim) s = fmaf(qv[i], get(k + lane + 32 * i), s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= p.scale_log2;
    const float next = fmaxf(m, s), base = next == -INFINITY ? 0.0f : next;
    const float keep = exp2f(m - base), w = exp2f(s - base);
    m = next;
    l = fmaf(l, keep, w);
#pragma unroll
    for (int i = 0; i < kMax; ++i)
      if (lane + 32 * i < p.dim) acc[i] = fmaf(acc[i], keep, w * get(v + lane + 32 * i));
  }
#pragma unroll
  for (int i = 0; i < kMax; ++i) acc_s[warp][lane + 32 * i] = acc[i];
  if (lane == 0) m_s[warp] = m, l_s[warp] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.0f, scale[kWarps];
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    scale[w] = top == -INFINITY ? 0.0f : exp2f(m_s[w] - top);
    sum = fmaf(l_s[w], scale[w], sum);
  }
  IT* out = static_cast<IT*>(p.out) + (bt * p.H + h) * p.dim;
  for (int c = threadIdx.x; c < p.dim; c += kAttnPlainThreads) {
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) y = fmaf(acc_s[w][c], scale[w], y);
    put(out + c, sum == 0.0f ? 0.0f : y / sum);
  }
}

}  // namespace hybrid
