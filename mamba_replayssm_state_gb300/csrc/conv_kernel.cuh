// conv_kernel.cuh -- the short causal convolution over each channel, width W:
//   v(t) = bias + sum_{j < W} w[W-1-j] in(t-j),  out = v or v / (1 + exp(-v))
// Sums in fp32, rounded to the output's type once; cached inputs are copied as they are.
//
// Memory bounds it: each input read once, each output written once.  But eight channels
// of a token are 32 multiplications, 16 exponentials and reciprocals and some forty other
// instructions for 32 bytes, so these are kept few: channels in pairs (fma.rn.f32x2),
// the fast exponential and reciprocal without the handling of denormals, whole groups
// of tokens without a test in between.  A thread keeps its channels' weights and last
// W-1 inputs in registers and walks along the tokens.  The rows to come lie in shared memory, or are
// on their way there (cp.async), each in a place that only its thread writes and reads: no barriers,
// and more bytes in flight than registers would hold.
//
// Measured on a GB300 (graphs of calls on changing inputs): 8192 tokens of 18432 bf16 channels 96 us, 6.3
// TB/s (129 with the rows to come in registers), of fp32 190 us, 6.4 TB/s; 256 requests'
// single tokens 13.5 us, 4.2 TB/s with the launch's 2.3; 37 tokens of 5376 channels 4.8 us.  One channel a thread,
// where rows are no whole 16 bytes: 8192 tokens of 5377 bf16 channels 151 us, 1.2 TB/s.
#pragma once
#include "hybrid_device.cuh"
#include "rsm_ptx.cuh"

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
  __device__ __forceinline__ static T mul(T a, T b) {
    T r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
  }
  __device__ __forceinline__ static T add(T a, T b) {
    T r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp2_ftz(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// silu(v); for bf16 by the fast exponential and reciprocal, within 2^-17 for |v| < 80, far below
// the output's own 2^-9.
template <typename IT>
__device__ __forceinline__ float silu(float v) {
  if constexpr (sizeof(IT) == 2)
    return v * rcp_ftz(1.0f + exp2_ftz(v * -kLog2e));
  else
    return v / (1.0f + expf(-v));
}

// A thread's own places in shared memory, 16 bytes each, [place][thread].
struct Places {
  uint32_t base;
  __device__ __forceinline__ explicit Places(const void* smem) : base(rsm::smem_addr(smem) + threadIdx.x * 16) {}
  __device__ __forceinline__ uint32_t at(int place) const { return base + place * (kConvThreads * 16); }
  template <typename T>
  __device__ __forceinline__ void ask(int place, const T* from) const {
    rsm::cp_async_16(at(place), from);
  }
  template <typename R>
  __device__ __forceinline__ R get(int place) const {
    R r;
    *reinterpret_cast<uint4*>(r.v) = rsm::lds128(at(place));
    return r;
  }
};

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
  if (act) {
    if constexpr (V > 1 && sizeof(IT) == 2) {
      const uint64_t scale = L::make(-kLog2e, -kLog2e), one = L::make(1.0f, 1.0f);
#pragma unroll
      for (int i = 0; i < L::N; ++i) {  // silu() of two at a time
        float a, b;
        L::split(L::mul(y[i], scale), a, b);
        L::split(L::add(L::make(exp2_ftz(a), exp2_ftz(b)), one), a, b);
        y[i] = L::mul(y[i], L::make(rcp_ftz(a), rcp_ftz(b)));
      }
      L::to(y, f);
    } else {
      L::to(y, f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = silu<IT>(f[i]);
    }
  } else {
    L::to(y, f);
  }
  Row<IT, V> out;
  out.round(f);
  return out;
}

// Packed prompts: a CTA takes p.block tokens of kConvThreads * V channels, four tokens at
// a time, kConvAhead on their way.  The first W - 1 tokens of a sequence belong to the CTA in
// which it starts, which so is the only one to look into the cache and to store
// there: it reads before it writes.
template <typename IT, int W, int V>
__global__ void __launch_bounds__(kConvThreads, V == 1 ? 8 : 4) conv_prompt_kernel(const __grid_constant__ ConvParams p) {
  constexpr int U = 4;
  constexpr int64_t kNever = int64_t{1} << 62;
  static_assert(kConvAhead % U == 0);
  __shared__ __align__(16) uint4 ring[V == 1 ? 1 : (kConvAhead + W - 1) * kConvThreads];
  const uint32_t block = blockIdx.x / static_cast<uint32_t>(p.cblocks), cb = blockIdx.x - block * static_cast<uint32_t>(p.cblocks);
  const int64_t first = static_cast<int64_t>(block) * p.block, last = min(first + p.block, p.tokens);
  const int64_t c = (static_cast<int64_t>(cb) * kConvThreads + threadIdx.x) * V;
  const bool mine = c < p.C;
  const IT* const x = static_cast<const IT*>(p.x) + c;
  IT* const out = static_cast<IT*>(p.out) + c;
  // what does not depend on the sequences is on its way before they are looked up
  const Places place(ring);
  auto ask = [&](int64_t t, int at) {  // tokens t .. t + U - 1 to the places from `at`
    if constexpr (V > 1) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t + u < last) place.ask(at + u, x + (t + u) * p.x_ts);
      cp_async_commit();
    }
  };
  if (mine) {
#pragma unroll
    for (int k = 0; k < kConvAhead; k += U) ask(first + k, k);
  }
  Row<IT, V> before[W - 1];
#pragma unroll
  for (int j = 1; j < W; ++j) {
    before[j - 1].zero();
    if (mine && first >= j) before[j - 1].load(x + (first - j) * p.x_ts);
  }
  Taps<W, V> taps;
  if (mine) taps.load(p.weight, p.bias, static_cast<int>(c));
  const int live = live_sequences(p.cu, p.seqs, p.tokens, p.status, blockIdx.x == 0);
  if (!mine) return;
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
        s0 = s1 = kNever;  // (own is not s0: nothing starts here)
        own = kNever + 1;
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
    // All are asked for at once, the last inputs, which only pass through, by way of places of their own (8192 tokens of
    // 5376 channels in 512 and 2048 sequences: 54 and 101 us, 64 and 131 of one row after the other; through
    // registers 55 and 97, but then 4096 tokens of four sequences 24 instead of 21.5).
    if constexpr (V > 1) {
#pragma unroll
      for (int j = 1; j < W; ++j)
        if (n >= static_cast<uint32_t>(j)) place.ask(kConvAhead + j - 1, x + (s1 - j) * p.x_ts);
      cp_async_commit();
    }
    Row<IT, V> was[W - 1];
#pragma unroll
    for (int j = 1; j < W; ++j) {
      was[j - 1].zero();
      if (at >= j) was[j - 1].load(rows + static_cast<int64_t>((pos - j) % R) * p.C);
    }
#pragma unroll
    for (int j = 1; j < W; ++j) h.set(j - 1, was[j - 1]);
    if constexpr (V > 1) cp_async_wait<0>();
#pragma unroll
    for (int j = 1; j < W; ++j)
      if (n >= static_cast<uint32_t>(j)) {
        Row<IT, V> r;
        if constexpr (V > 1)
          r = place.get<Row<IT, V>>(kConvAhead + j - 1);
        else
          r.load(x + (s1 - j) * p.x_ts);
        r.store(rows + static_cast<int64_t>((pos + n - j) % R) * p.C);
      }
  };
  auto one = [&](int64_t t, int at) {  // any token, one of the block's in place `at`
    advance(t);
    if (t < s0) return;
    if (t == s0 && own == s0) start();
    Row<IT, V> in;
    if (V == 1 || t >= last) {
      in.load(x + t * p.x_ts);
    } else if constexpr (V > 1) {
      in = place.get<Row<IT, V>>(at);
    }
    const Row<IT, V> y = conv_token<IT, W, V>(taps, h, in, act);
    if (t >= own) y.store(out + t * p.out_ts);
  };
  advance(first);
  int at = 0;
  for (int64_t t = first; t < last; t += U) {
    if constexpr (V > 1) cp_async_wait<kConvAhead / U - 1>();
    if (V > 1 && t > s0 && t >= own && t + U <= min(s1, last)) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        conv_token<IT, W, V>(taps, h, place.get<Row<IT, V>>(at + u), act).store(out + (t + u) * p.out_ts);
    } else {
      for (int64_t i = t; i < min(t + U, last); ++i) one(i, at + static_cast<int>(i - t));
    }
    ask(t + kConvAhead, at);
    at = at + U == kConvAhead ? 0 : at + U;
  }
  if constexpr (V > 1) cp_async_wait<0>();
  // the rest of the first W - 1 tokens of a sequence that starts here
  if (own == s0 && s0 < last)
    for (int64_t t = last; t < min(s1, s0 + (W - 1)); ++t) one(t, 0);
}

// New tokens: a CTA takes p.block requests one after the other, in items of up to U tokens,
// the next two items' rows on their way.  Rows that are written are none that a window
// looks back to (R >= W - 1 + window).
template <typename IT, int W, int V>
__global__ void __launch_bounds__(kConvThreads, V == 1 ? 8 : 4) conv_step_kernel(const __grid_constant__ ConvParams p) {
  constexpr int U = 4, kRows = W - 1 + U, kItems = 3;
  struct Request {
    int64_t back[W - 1];  // offsets in the cache of the rows before, -1: none
    int64_t slot;         // of the slot, -1: skipped
    uint32_t row;         // of the first token
  };
  __shared__ Request request[kConvStepRequests];
  __shared__ __align__(16) uint4 ring[V == 1 ? 1 : kItems * kRows * kConvThreads];
  const uint32_t group = blockIdx.x / static_cast<uint32_t>(p.cblocks), cb = blockIdx.x - group * static_cast<uint32_t>(p.cblocks);
  const int64_t c = (static_cast<int64_t>(cb) * kConvThreads + threadIdx.x) * V, b0 = static_cast<int64_t>(group) * p.block;
  const int count = static_cast<int>(min(static_cast<int64_t>(p.block), p.seqs - b0));
  const uint32_t R = static_cast<uint32_t>(p.R);
  const IT* const x = static_cast<const IT*>(p.x) + b0 * p.x_bs + c;
  IT* const out = static_cast<IT*>(p.out) + b0 * p.window * p.out_ts + c;
  IT* const cache = static_cast<IT*>(p.cache) + c;
  const bool mine = c < p.C;
  const Places place(ring);
  const int chunks = (p.window + U - 1) / U;
  auto ask_tokens = [&](int n, int k, int at) {  // of item (n, k), request n's chunk k
    const IT* from = x + n * p.x_bs + k * U * p.x_ts;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k * U + u < p.window) place.ask(at + W - 1 + u, from + u * p.x_ts);
  };
  // the first items' own rows do not depend on where the requests are
  if (V > 1 && mine) {
#pragma unroll
    for (int i = 0; i < kItems - 1; ++i)
      if (i < count * chunks) ask_tokens(i / chunks, i % chunks, i * kRows);
  }
  if (static_cast<int>(threadIdx.x) < count) {
    Request r;
    const int slot = p.slots[b0 + threadIdx.x], pos = p.positions[b0 + threadIdx.x];
    r.slot = -1;
    r.row = 0;
    if (slot == p.pad) {
    } else if (slot < 0 || slot >= p.num_slots || pos < 0) {
      if (cb == 0) flag(p.status, slot < 0 || slot >= p.num_slots ? RSM_STATUS_BAD_SLOT : RSM_STATUS_BAD_POSITION);
    } else {
      r.slot = slot * p.cache_ss;
      r.row = static_cast<uint32_t>(pos) % R;
    }
    uint32_t row = r.row;
#pragma unroll
    for (int j = 1; j < W; ++j) {
      row = row == 0 ? R - 1 : row - 1;
      r.back[j - 1] = r.slot >= 0 && pos >= j ? r.slot + static_cast<int64_t>(row) * p.C : -1;
    }
    request[threadIdx.x] = r;
  }
  Taps<W, V> taps;
  if (mine) taps.load(p.weight, p.bias, static_cast<int>(c));
  __syncthreads();
  if (!mine) return;
  const bool act = p.silu != 0;
  int ask_n = 0, ask_k = 0, ask_at = 0;
  auto ask = [&](bool first) {  // the next item's rows
    if constexpr (V > 1) {
      if (ask_n < count && request[ask_n].slot >= 0) {
        if (ask_k == 0) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
            if (request[ask_n].back[j] >= 0) place.ask(ask_at + j, cache + request[ask_n].back[j]);
        }
        if (!first) ask_tokens(ask_n, ask_k, ask_at);
      }
      cp_async_commit();
      if (++ask_k == chunks) ask_k = 0, ++ask_n;
      ask_at = ask_at + kRows == kItems * kRows ? 0 : ask_at + kRows;
    }
  };
#pragma unroll
  for (int i = 0; i < kItems - 1; ++i) ask(true);
  int at = 0;
  for (int n = 0; n < count; ++n) {
    const int64_t slot = request[n].slot;
    IT* y = out + n * p.window * p.out_ts;
    uint32_t row = request[n].row;
    Past<W, V> h;
    for (int k = 0; k < chunks; ++k) {
      ask(false);
      if constexpr (V > 1) cp_async_wait<kItems - 1>();
      if (k == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          Row<IT, V> r;
          r.zero();
          if (request[n].back[j] >= 0) {
            if constexpr (V > 1)
              r = place.get<Row<IT, V>>(at + j);
            else
              r.load(cache + request[n].back[j]);
          }
          h.set(j, r);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k * U + u >= p.window) break;
        Row<IT, V> in;
        if (slot < 0) {
          in.zero();
          in.store(y);
        } else {
          if constexpr (V > 1)
            in = place.get<Row<IT, V>>(at + W - 1 + u);
          else
            in.load(x + n * p.x_bs + (k * U + u) * p.x_ts);
          in.store(cache + slot + static_cast<int64_t>(row) * p.C);
          row = row + 1 == R ? 0 : row + 1;
          conv_token<IT, W, V>(taps, h, in, act).store(y);
        }
        y += p.out_ts;
      }
      at = at + kRows == kItems * kRows ? 0 : at + kRows;
    }
  }
  if constexpr (V > 1) cp_async_wait<0>();
}

}  // namespace hybrid
