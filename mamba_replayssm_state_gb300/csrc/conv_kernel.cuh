// conv_kernel.cuh -- the short causal convolution over each channel, width W:
//   v(t) = bias + sum_{j < W} w[W-1-j] in(t-j),  out = v or v / (1 + exp(-v))
// Sums in fp32, rounded to the output's type once; cached inputs are copied as they are.
//
// Memory bounds it: each input read once, each output written once.  But eight channels
// of a token are 32 multiplications, 16 exponentials and reciprocals and some forty other
// instructions for 32 bytes, so these are kept few: channels in pairs (fma.rn.f32x2),
// the fast exponential and reciprocal without the handling of denormals, whole groups
// of tokens without a test in between.  A thread keeps its channels' weights and last
// W-1 inputs in registers and walks along the tokens, the next ones' loads on their way.
#pragma once
#include "hybrid_device.cuh"

namespace hybrid {

// Two fp32 values, or one where a thread has one channel.
template <int V>
struct Lanes {
  static constexpr int N = V / 2;
  using T = uint64_t;
  __device__ __forceinline__ static T make(float a, float b) {
    T r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ static void split(T v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
  __device__ __forceinline__ static T fma(T a, T b, T c) {
    T r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
  }
  __device__ __forceinline__ static void from(const float (&f)[V], T (&t)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = make(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ static void to(const T (&t)[N], float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < N; ++i) split(t[i], f[2 * i], f[2 * i + 1]);
  }
};
template <>
struct Lanes<1> {
  static constexpr int N = 1;
  using T = float;
  __device__ __forceinline__ static T fma(T a, T b, T c) { return fmaf(a, b, c); }
  __device__ __forceinline__ static void from(const float (&f)[1], T (&t)[1]) { t[0] = f[0]; }
  __device__ __forceinline__ static void to(const T (&t)[1], float (&f)[1]) { f[0] = t[0]; }
};

// silu(v); for bf16 by the fast exponential and reciprocal, within 2^-17 for |v| < 80, far below
// the output's own 2^-9.
template <typename IT>
__device__ __forceinline__ float silu(float v) {
  if constexpr (sizeof(IT) == 2) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.44269504088896340736f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return v * r;
  } else {
    return v / (1.0f + expf(-v));
  }
}

template <int W, int V>
struct Taps {
  using L = Lanes<V>;
  typename L::T w[W][L::N], b[L::N];
  __device__ __forceinline__ void load(const float* weight, const float* bias, int c) {
    float flat[W * V], one[V];
    if constexpr (V == 1) {
#pragma unroll
      for (int i = 0; i < W; ++i) flat[i] = __ldg(weight + static_cast<int64_t>(c) * W + i);
    } else {
#pragma unroll
      for (int i = 0; i < W * V / 4; ++i)
        *reinterpret_cast<float4*>(flat + 4 * i) = __ldg(reinterpret_cast<const float4*>(weight + static_cast<int64_t>(c) * W) + i);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) one[i] = flat[i * W + j];
      L::from(one, w[j]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) one[i] = bias == nullptr ? 0.0f : __ldg(bias + c + i);
    L::from(one, b);
  }
};

// The last W - 1 inputs: v[j] is the one j + 1 tokens back.
template <int W, int V>
struct Past {
  using L = Lanes<V>;
  typename L::T v[W - 1][L::N];
  __device__ __forceinline__ void zero() {
    const float none[V] = {};
#pragma unroll
    for (int j = 0; j < W - 1; ++j) L::from(none, v[j]);
  }
  template <typename IT>
  __device__ __forceinline__ void set(int j, const Row<IT, V>& row) {
    float f[V];
    row.values(f);
    L::from(f, v[j]);
  }
};

// One token's output; the past moves on by it.
template <typename IT, int W, int V>
__device__ __forceinline__ Row<IT, V> conv_token(const Taps<W, V>& k, Past<W, V>& h, const Row<IT, V>& in, bool act) {
  using L = Lanes<V>;
  float f[V];
  typename L::T x[L::N], y[L::N];
  in.values(f);
  L::from(f, x);
#pragma unroll
  for (int i = 0; i < L::N; ++i) {
    y[i] = k.b[i];
#pragma unroll
    for (int j = W - 1; j >= 1; --j) y[i] = L::fma(k.w[W - 1 - j][i], h.v[j - 1][i], y[i]);
    y[i] = L::fma(k.w[W - 1][i], x[i], y[i]);
#pragma unroll
    for (int j = W - 2; j >= 1; --j) h.v[j][i] = h.v[j - 1][i];
    h.v[0][i] = x[i];
  }
  L::to(y, f);
  if (act) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = silu<IT>(f[i]);
  }
  Row<IT, V> out;
  out.round(f);
  return out;
}

// Packed prompts: a CTA takes p.block tokens of kConvThreads * V channels, four tokens at
// a time.  The first W - 1 tokens of a sequence belong to the CTA in which it
// starts, which so is the only one to look into the cache and to store there: it reads
// before it writes.
template <typename IT, int W, int V>
__global__ void __launch_bounds__(kConvThreads, V == 1 ? 8 : 4) conv_prompt_kernel(const __grid_constant__ ConvParams p) {
  constexpr int U = 4;  // tokens at a time
  constexpr int64_t kNever = int64_t{1} << 62;
  const uint32_t block = blockIdx.x / static_cast<uint32_t>(p.cblocks), cb = blockIdx.x - block * static_cast<uint32_t>(p.cblocks);
  const int64_t first = static_cast<int64_t>(block) * p.block, last = min(first + p.block, p.tokens);
  const int64_t c = (static_cast<int64_t>(cb) * kConvThreads + threadIdx.x) * V;
  const bool mine = c < p.C;
  const IT* const x = static_cast<const IT*>(p.x) + c;
  IT* const out = static_cast<IT*>(p.out) + c;
  // what does not depend on the sequences is on its way before they are looked up
  Row<IT, V> next[U], before[W - 1];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (mine && first + u < last) next[u].load(x + (first + u) * p.x_ts);
#pragma unroll
  for (int j = 1; j < W; ++j) {
    before[j - 1].zero();
    if (mine && first >= j) before[j - 1].load(x + (first - j) * p.x_ts);
  }
  const int live = live_sequences(p.cu, p.seqs, p.tokens, p.status, blockIdx.x == 0);
  if (!mine) return;
  Taps<W, V> taps;
  taps.load(p.weight, p.bias, static_cast<int>(c));
  const bool act = p.silu != 0;
  Past<W, V> h;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) h.set(j, before[j]);

  // The sequence at hand: tokens s0 .. s1 - 1, of which this CTA has those from `own` on.
  int s = sequence_at(p.cu, live, first) - 1;
  int64_t s0 = 0, s1 = first, own = 0;
  auto advance = [&](int64_t t) {  // to the first sequence that ends after t
    while (s1 <= t) {
      if (++s >= live) {
        s0 = s1 = own = kNever;
        return;
      }
      s0 = p.cu[s], s1 = p.cu[s + 1];
      own = s0 >= first ? s0 : s0 + (W - 1);
      if (s0 < 0 || s1 > p.tokens) own = kNever;  // not to be done
    }
  };
  auto start = [&]() {  // at token s0: what came before it, and what it leaves behind
    h.zero();
    if (p.cache == nullptr) return;
    const int slot = p.slots[s], at = p.positions == nullptr ? 0 : p.positions[s];
    if (slot == p.pad) return;
    if (slot < 0 || slot >= p.num_slots || at < 0) {
      if (c == 0) flag(p.status, at < 0 ? RSM_STATUS_BAD_POSITION : RSM_STATUS_BAD_SLOT);
      return;
    }
    IT* const rows = static_cast<IT*>(p.cache) + slot * p.cache_ss + c;
    const uint32_t pos = static_cast<uint32_t>(at), R = static_cast<uint32_t>(p.R), n = static_cast<uint32_t>(s1 - s0);
#pragma unroll
    for (int j = 1; j < W; ++j)
      if (at >= j) {
        Row<IT, V> r;
        r.load(rows + static_cast<int64_t>((pos - j) % R) * p.C);
        h.set(j - 1, r);
      }
#pragma unroll
    for (int j = 1; j < W; ++j)
      if (n >= static_cast<uint32_t>(j)) {
        Row<IT, V> r;
        r.load(x + (s1 - j) * p.x_ts);
        r.store(rows + static_cast<int64_t>((pos + n - j) % R) * p.C);
      }
  };
  auto one = [&](int64_t t) {  // any token
    advance(t);
    if (t < s0) return;
    if (t == s0 && own == s0) start();
    Row<IT, V> in;
    in.load(x + t * p.x_ts);
    const Row<IT, V> y = conv_token<IT, W, V>(taps, h, in, act);
    if (t >= own) y.store(out + t * p.out_ts);
  };
  advance(first);
  for (int64_t t = first; t < last; t += U) {
    Row<IT, V> in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) in[u] = next[u];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t + U + u < last) next[u].load(x + (t + U + u) * p.x_ts);
    if (t > s0 && t >= own && t + U <= min(s1, last)) {
#pragma unroll
      for (int u = 0; u < U; ++u) conv_token<IT, W, V>(taps, h, in[u], act).store(out + (t + u) * p.out_ts);
    } else {
      for (int64_t i = t; i < min(t + U, last); ++i) one(i);
    }
  }
  // the rest of the first W - 1 tokens of a sequence that starts here
  if (own == s0)
    for (int64_t t = last; t < min(s1, s0 + (W - 1)); ++t) one(t);
}

// New tokens: a CTA takes p.block requests one after the other, the next one's loads on
// their way.  Rows that are written are none that a window looks back to (R >= W - 1 + window).
template <typename IT, int W, int V>
__global__ void __launch_bounds__(kConvThreads, V == 1 ? 8 : 4) conv_step_kernel(const __grid_constant__ ConvParams p) {
  __shared__ int slot_s[kConvStepRequests];
  __shared__ int pos_s[kConvStepRequests];
  const uint32_t group = blockIdx.x / static_cast<uint32_t>(p.cblocks), cb = blockIdx.x - group * static_cast<uint32_t>(p.cblocks);
  const int64_t c = (static_cast<int64_t>(cb) * kConvThreads + threadIdx.x) * V, b0 = static_cast<int64_t>(group) * p.block;
  const int count = static_cast<int>(min(static_cast<int64_t>(p.block), p.seqs - b0));
  const uint32_t R = static_cast<uint32_t>(p.R);
  if (static_cast<int>(threadIdx.x) < count) {
    int slot = p.slots[b0 + threadIdx.x];
    const int pos = p.positions[b0 + threadIdx.x];
    if (slot == p.pad) {
      slot = -1;
    } else if (slot < 0 || slot >= p.num_slots || pos < 0) {
      if (cb == 0) flag(p.status, slot < 0 || slot >= p.num_slots ? RSM_STATUS_BAD_SLOT : RSM_STATUS_BAD_POSITION);
      slot = -1;
    }
    slot_s[threadIdx.x] = slot;
    pos_s[threadIdx.x] = pos;
  }
  __syncthreads();
  if (c >= p.C) return;
  const IT* const x = static_cast<const IT*>(p.x) + b0 * p.x_bs + c;
  IT* out = static_cast<IT*>(p.out) + b0 * p.window * p.out_ts + c;
  IT* const cache = static_cast<IT*>(p.cache) + c;
  Row<IT, V> back[W - 1], in;
  auto ask = [&](int n) {
    const int slot = slot_s[n];
    if (slot < 0) return;
    const uint32_t pos = static_cast<uint32_t>(pos_s[n]);
    in.load(x + n * p.x_bs);
    uint32_t row = pos % R;
#pragma unroll
    for (int j = 1; j < W; ++j) {
      row = row == 0 ? R - 1 : row - 1;
      back[j - 1].zero();
      if (pos >= static_cast<uint32_t>(j)) back[j - 1].load(cache + slot * p.cache_ss + static_cast<int64_t>(row) * p.C);
    }
  };
  ask(0);
  Taps<W, V> taps;
  taps.load(p.weight, p.bias, static_cast<int>(c));
  const bool act = p.silu != 0;
  for (int n = 0; n < count; ++n, out += p.window * p.out_ts) {
    const int slot = slot_s[n];
    Past<W, V> h;
    Row<IT, V> now = in;
    if (slot >= 0) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) h.set(j, back[j]);
    }
    if (n + 1 < count) ask(n + 1);
    if (slot < 0) {
      Row<IT, V> none;
      none.zero();
      for (int t = 0; t < p.window; ++t) none.store(out + t * p.out_ts);
      continue;
    }
    uint32_t row = static_cast<uint32_t>(pos_s[n]) % R;
    IT* const rows = cache + slot * p.cache_ss;
    for (int t = 0; t < p.window; ++t) {
      const Row<IT, V> cur = now;
      if (t + 1 < p.window) now.load(x + n * p.x_bs + (t + 1) * p.x_ts);
      cur.store(rows + static_cast<int64_t>(row) * p.C);
      row = row + 1 == R ? 0 : row + 1;
      conv_token<IT, W, V>(taps, h, cur, act).store(out + t * p.out_ts);
    }
  }
}

}  // namespace hybrid
