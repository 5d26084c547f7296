// conv_kernel.cuh -- the short causal convolution over each channel, width W:
//   v(t) = bias + sum_{j < W} w[W-1-j] in(t-j),  out = v or v / (1 + exp(-v))
// Sums in fp32, rounded to the output's type once; cached inputs are copied as they are.
//
// Memory bounds it: each input read once, each output written once.  A thread keeps
// its channels' weights and last W-1 inputs in registers and walks along the tokens.
#pragma once
#include "hybrid_device.cuh"

namespace hybrid {

// silu(v); for bf16 the exponential and the quotient are the fast ones, within 2^-17
// for |v| < 80, far below the output's own 2^-9.
template <typename IT>
__device__ __forceinline__ float silu(float v) {
  if constexpr (sizeof(IT) == 2)
    return __fdividef(v, 1.0f + __expf(-v));
  else
    return v / (1.0f + expf(-v));
}

template <int W, int V>
struct Taps {
  float w[W][V], b[V];
  __device__ __forceinline__ void load(const float* weight, const float* bias, int c) {
    float flat[W * V];
    if constexpr (V == 1) {
#pragma unroll
      for (int i = 0; i < W; ++i) flat[i] = __ldg(weight + static_cast<int64_t>(c) * W + i);
    } else {
#pragma unroll
      for (int i = 0; i < W * V / 4; ++i)
        *reinterpret_cast<float4*>(flat + 4 * i) = __ldg(reinterpret_cast<const float4*>(weight + static_cast<int64_t>(c) * W) + i);
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) w[j][i] = flat[i * W + j];
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = bias == nullptr ? 0.0f : __ldg(bias + c + i);
  }
};

// One token: h[j] is the input j + 1 tokens before it; both move on by one.
template <typename IT, int W, int V>
__device__ __forceinline__ Row<IT, V> conv_token(const Taps<W, V>& k, float (&h)[W - 1][V], const Row<IT, V>& in, bool act) {
  float x[V], y[V];
  in.values(x);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float v = k.b[i];
#pragma unroll
    for (int j = W - 1; j >= 1; --j) v = fmaf(k.w[W - 1 - j][i], h[j - 1][i], v);
    v = fmaf(k.w[W - 1][i], x[i], v);
    y[i] = act ? silu<IT>(v) : v;
#pragma unroll
    for (int j = W - 2; j >= 1; --j) h[j][i] = h[j - 1][i];
    h[0][i] = x[i];
  }
  Row<IT, V> out;
  out.round(y);
  return out;
}

// Packed prompts: a CTA takes kConvTokens tokens of kConvThreads * V channels.  The
// first W - 1 tokens of a sequence belong to the CTA in which it starts, which so is
// the only one to look into the cache and to store there: it reads before it writes.
template <typename IT, int W, int V>
__global__ void __launch_bounds__(kConvThreads) conv_prompt_kernel(const __grid_constant__ ConvParams p) {
  constexpr int U = V == 1 ? 4 : 8;  // rows asked for at a time
  const uint32_t block = blockIdx.x / static_cast<uint32_t>(p.cblocks), cb = blockIdx.x - block * static_cast<uint32_t>(p.cblocks);
  const int64_t first_token = static_cast<int64_t>(block) * kConvTokens;
  const int64_t last_token = min(first_token + kConvTokens, p.tokens);
  const int live = live_sequences(p.cu, p.seqs, p.tokens, p.status, blockIdx.x == 0);
  const int64_t c = (static_cast<int64_t>(cb) * kConvThreads + threadIdx.x) * V;
  if (c >= p.C) return;
  const IT* const x = static_cast<const IT*>(p.x) + c;
  IT* const out = static_cast<IT*>(p.out) + c;
  Taps<W, V> taps;
  taps.load(p.weight, p.bias, static_cast<int>(c));
  const bool act = p.silu != 0;
  for (int s = sequence_at(p.cu, live, first_token); s < live; ++s) {
    const int64_t s0 = p.cu[s], s1 = p.cu[s + 1];
    if (s0 >= last_token) break;
    if (s0 < 0 || s1 > p.tokens || s0 == s1) continue;
    const bool starts = s0 >= first_token;
    int64_t t = starts ? s0 : max(first_token, s0 + (W - 1));
    const int64_t end = min(s1, max(last_token, s0 + (W - 1)));
    float h[W - 1][V];
    IT* slot_rows = nullptr;
    uint32_t pos = 0;
    if (starts) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) h[j][i] = 0.0f;
      if (p.cache != nullptr) {
        const int slot = p.slots[s], at = p.positions == nullptr ? 0 : p.positions[s];
        if (slot == p.pad) {
        } else if (slot < 0 || slot >= p.num_slots || at < 0) {
          if (c == 0) flag(p.status, at < 0 ? RSM_STATUS_BAD_POSITION : RSM_STATUS_BAD_SLOT);
        } else {
          slot_rows = static_cast<IT*>(p.cache) + slot * p.cache_ss + c;
          pos = static_cast<uint32_t>(at);
#pragma unroll
          for (int j = 1; j < W; ++j)
            if (at >= j) {
              Row<IT, V> r;
              r.load(slot_rows + static_cast<int64_t>((pos - j) % static_cast<uint32_t>(p.R)) * p.C);
              r.values(h[j - 1]);
            }
        }
      }
    } else if (t < end) {
#pragma unroll
      for (int j = 1; j < W; ++j) {
        Row<IT, V> r;
        r.load(x + (t - j) * p.x_ts);
        r.values(h[j - 1]);
      }
    }
    while (t < end) {
      Row<IT, V> in[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t + u < end) in[u].load(x + (t + u) * p.x_ts);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t + u < end) conv_token<IT, W, V>(taps, h, in[u], act).store(out + (t + u) * p.out_ts);
      t += U;
    }
    if (slot_rows != nullptr) {
      const uint32_t n = static_cast<uint32_t>(s1 - s0);
#pragma unroll
      for (int j = 1; j < W; ++j)
        if (n >= static_cast<uint32_t>(j)) {
          Row<IT, V> r;
          r.load(x + (s1 - j) * p.x_ts);
          r.store(slot_rows + static_cast<int64_t>((pos + n - j) % static_cast<uint32_t>(p.R)) * p.C);
        }
    }
  }
}

// New tokens: a thread takes N requests, whose loads are all asked for before the first
// is used, and goes through their windows together.  Rows that are written are none
// that the window looks back to (R >= W - 1 + window).
template <typename IT, int W, int V, int N>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const __grid_constant__ ConvParams p) {
  const uint32_t group = blockIdx.x / static_cast<uint32_t>(p.cblocks), cb = blockIdx.x - group * static_cast<uint32_t>(p.cblocks);
  const int64_t c = (static_cast<int64_t>(cb) * kConvThreads + threadIdx.x) * V;
  if (c >= p.C) return;
  const uint32_t R = static_cast<uint32_t>(p.R);
  Row<IT, V> back[N][W - 1], in[N];
  IT* rows[N];
  uint32_t at[N];
  const IT* x[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int64_t b = static_cast<int64_t>(group) * N + n;
    rows[n] = nullptr;
    at[n] = 0;
    x[n] = static_cast<const IT*>(p.x) + b * p.x_bs + c;
    if (b < p.seqs) {
      const int slot = p.slots[b], pos = p.positions[b];
      if (slot == p.pad) {
      } else if (slot < 0 || slot >= p.num_slots || pos < 0) {
        if (c == 0) flag(p.status, slot < 0 || slot >= p.num_slots ? RSM_STATUS_BAD_SLOT : RSM_STATUS_BAD_POSITION);
      } else {
        rows[n] = static_cast<IT*>(p.cache) + slot * p.cache_ss + c;
        at[n] = static_cast<uint32_t>(pos);
        in[n].load(x[n]);
#pragma unroll
        for (int j = 1; j < W; ++j) {
          back[n][j - 1].zero();
          if (pos >= j) back[n][j - 1].load(rows[n] + static_cast<int64_t>((at[n] - j) % R) * p.C);
        }
      }
    }
  }
  Taps<W, V> taps;
  taps.load(p.weight, p.bias, static_cast<int>(c));
  const bool act = p.silu != 0;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int64_t b = static_cast<int64_t>(group) * N + n;
    if (b >= p.seqs) break;
    IT* out = static_cast<IT*>(p.out) + b * p.window * p.out_ts + c;
    if (rows[n] == nullptr) {
      Row<IT, V> none;
      none.zero();
      for (int t = 0; t < p.window; ++t) none.store(out + t * p.out_ts);
      continue;
    }
    float h[W - 1][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) back[n][j].values(h[j]);
    uint32_t row = at[n] % R;
    Row<IT, V> now = in[n];
    for (int t = 0; t < p.window; ++t) {
      const Row<IT, V> cur = now;
      if (t + 1 < p.window) now.load(x[n] + (t + 1) * p.x_ts);
      cur.store(rows[n] + static_cast<int64_t>(row) * p.C);
      row = row + 1 == R ? 0 : row + 1;
      conv_token<IT, W, V>(taps, h, cur, act).store(out + t * p.out_ts);
    }
  }
}

}  // namespace hybrid
