// rotary_kernel.cuh -- rotary positions on the queries and keys of new tokens, keys
// and values to their pages.
//
// The angle p f of a far position has to be taken modulo a turn before it is rounded
// to 24 bits.  Here the fraction of a turn that one position makes, f / (2 pi) mod 1,
// is a 64-bit integer (in units of 2^-64 turns, from two-term fp64 products), so that
// times the position it wraps by itself: the error, a unit a position, stays below
// 2^-32 turns, and the upper 32 bits are what sine and cosine are taken of.
//
// Memory bounds it: q, k, v read once and written once.  So whole tokens pass through
// shared memory by bulk copies, a ring of them in a CTA that stays for a run of tokens: one
// warp looks up where they go, makes their sines and cosines (once for all heads) and
// issues the copies in and out; the others turn the pairs in place, and touch nothing
// else.  Few tokens (rotary_few()), fp32 heads turned whole in halves, rows that are not whole 16-byte vectors and rows too
// long for a ring go through rotary_token_kernel.
//
// Measured on a GB300 (graphs of calls on changing inputs): 8192 tokens, 32 heads and 8 of 128, half of each
// turned, bf16: 38 to 39 us, 5.2 TB/s (43 through registers, 16 bytes a thread and four tokens ahead); one token
// 3.3 to 3.8 us, of which a launch is 2.3.  A value at a time, where pairs or rows are no whole vectors (6 of 128 turned): 179 us.
#pragma once
#include "hybrid_device.cuh"
#include "rsm_ptx.cuh"

namespace hybrid {

struct RotaryToken {
  int64_t out;            // element offset of the token's queries in the results
  int64_t k_row, v_row;   // of its rows in the pages; -1: none
  uint32_t pos;
  int live;               // 0: no sequence's, 1: a skipped request's, 2: to be done
};

// f / (2 pi) mod 1 in units of 2^-64.  1 / (2 pi) is given to 106 bits, as the sum of two doubles: below 2^40 what they
// leave out, times 2^31 positions, stays below 2^-24 turns.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double d = fabs(static_cast<double>(f)), t = d * hi, e = fma(d, hi, -t) + d * lo;
  const double part = t - floor(t);  // exact: part has no bits that t has not
  const uint64_t n = __double2ull_rz(part * 0x1p64) + static_cast<uint64_t>(__double2ll_rn(e * 0x1p64));
  return f < 0.0f ? 0 - n : n;
}

// Of a frequency that is none, or 2^40 or more, every turn is NaN.
__device__ __forceinline__ float amplitude_of(float f, float amplitude) { return fabsf(f) < 0x1p40f ? amplitude : __int_as_float(0x7FFFFFFF); }

// Where token i of the call goes.
__device__ __forceinline__ RotaryToken rotary_token(const RotaryParams& p, int live, int64_t i) {
  const rsm_pages& pg = p.pages;
  RotaryToken k;
  int64_t b, t, n;
  k.live = 1;
  if (p.cu != nullptr) {
    b = sequence_at(p.cu, live, i);
    t = n = 0;
    if (b == live || p.cu[b] < 0 || p.cu[b] > i || p.cu[b + 1] > p.tokens)
      k.live = 0;
    else
      t = i - p.cu[b], n = p.cu[b + 1] - p.cu[b];
    k.out = i * p.out_ts;
  } else {
    b = i / p.window, t = i - b * p.window, n = p.window;
    k.out = b * p.out_bs + t * p.out_ts;
  }
  k.pos = 0;
  k.k_row = k.v_row = -1;
  if (k.live == 0) return k;
  const int64_t len = pg.lengths[b];
  if (len < n || len > static_cast<int64_t>(pg.table_width) * pg.page_size) {
    if (len != 0) flag(p.status, RSM_STATUS_BAD_POSITION);
    return k;
  }
  k.live = 2;
  k.pos = static_cast<uint32_t>(len - n + t);
  const uint32_t at = k.pos / static_cast<uint32_t>(pg.page_size);
  const int64_t row = k.pos - at * static_cast<uint32_t>(pg.page_size);
  const int page = pg.page_table[b * pg.table_stride + at];
  if (page < 0 || page >= pg.num_pages)
    flag(p.status, RSM_STATUS_BAD_PAGE);
  else
    k.k_row = page * pg.k_page_stride + row * pg.k_row_stride, k.v_row = page * pg.v_page_stride + row * pg.v_row_stride;
  return k;
}

// Cosine and sine of `pos` times a step, with the amplitude.
__device__ __forceinline__ float2 rotary_turn(uint32_t pos, uint64_t step, float amplitude) {
  const int32_t upper = static_cast<int32_t>(static_cast<uint32_t>((pos * step) >> 32));
  float s, c;
  sincospif(static_cast<float>(upper) * 0x1p-31f, &s, &c);
  return make_float2(c * amplitude, s * amplitude);
}

__device__ __forceinline__ void bulk_store(void* to, uint32_t from, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the last N groups of this thread's stores have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// V: values that a thread turns at once.
template <typename IT, int V>
__global__ void __launch_bounds__(kRotaryThreads) rotary_append_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int kWide = 16 / sizeof(IT), kWarps = kRotaryThreads / 32 - 1;  // that turn
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(8) uint64_t full_s[kRotaryMaxStages], done_s[kRotaryMaxStages];
  __shared__ int live_s[kRotaryMaxStages];
  const rsm_pages& pg = p.pages;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, S = p.stages;
  const int64_t begin = blockIdx.x * p.tokens / gridDim.x, count = (blockIdx.x + 1) * p.tokens / gridDim.x - begin;
  const int qn = p.H * p.dim, kn = p.G * p.dim;
  const uint32_t token_bytes = (qn + 2 * kn) * static_cast<uint32_t>(sizeof(IT)), ring = rsm::smem_addr(smem);
  float2* const turns = reinterpret_cast<float2*>(smem + S * token_bytes);
  const uint32_t full = rsm::smem_addr(full_s), done = rsm::smem_addr(done_s);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) rsm::mbar_init(full + 8 * s, 2), rsm::mbar_init(done + 8 * s, kWarps);
    rsm::fence_mbar_init();
  }
  __syncthreads();

  if (warp == 0) {
    // the rows come in whatever becomes of them
    auto load = [&](int64_t i, int s) {
      if (lane != 0) return;
      const uint32_t at = ring + s * token_bytes, qb = qn * sizeof(IT), kb = kn * sizeof(IT);
      int64_t q, k, v;
      if (p.cu != nullptr) {
        q = (begin + i) * p.q_ts, k = (begin + i) * p.k_ts, v = (begin + i) * p.v_ts;
      } else {
        const int64_t b = (begin + i) / p.window, t = begin + i - b * p.window;
        q = b * p.q_bs + t * p.q_ts, k = b * p.k_bs + t * p.k_ts, v = b * p.v_bs + t * p.v_ts;
      }
      mbar_arrive_expect_tx(full + 8 * s, token_bytes);
      rsm::bulk_g2s(at, static_cast<const IT*>(p.q) + q, qb, full + 8 * s);
      rsm::bulk_g2s(at + qb, static_cast<const IT*>(p.k) + k, kb, full + 8 * s);
      rsm::bulk_g2s(at + qb + kb, static_cast<const IT*>(p.v) + v, kb, full + 8 * s);
    };
    for (int i = 0; i < S - 1 && i < count; ++i) load(i, i);
    float freq[kRotaryMaxHalf / 32];  // (on their way while the first tokens are looked up)
#pragma unroll
    for (int j = 0; j < kRotaryMaxHalf / 32; ++j) freq[j] = lane + 32 * j < p.half ? p.inv_freq[lane + 32 * j] : 0.0f;
    const int live = p.cu == nullptr ? 0 : live_sequences_warp(p.cu, pg.requests, p.tokens, p.status, blockIdx.x == 0);
    RotaryToken mine{};  // of 32 tokens, a lane each
    if (lane < count) mine = rotary_token(p, live, begin + lane);
    uint64_t step[kRotaryMaxHalf / 32];
    float amplitude[kRotaryMaxHalf / 32];
#pragma unroll
    for (int j = 0; j < kRotaryMaxHalf / 32; ++j) step[j] = turns_per_position(freq[j]), amplitude[j] = amplitude_of(freq[j], p.amplitude);
    auto info = [&](int64_t i, int s) {
      if (i > 0 && i % 32 == 0 && i + lane < count) mine = rotary_token(p, live, begin + i + lane);
      const int from = static_cast<int>(i % 32);
      const uint32_t pos = __shfl_sync(0xFFFFFFFFu, mine.pos, from);
      const int state = __shfl_sync(0xFFFFFFFFu, mine.live, from);
      if (lane == 0) live_s[s] = state;
      if (state == 2) {
#pragma unroll
        for (int j = 0; j < kRotaryMaxHalf / 32; ++j)
          if (lane + 32 * j < p.half) turns[s * p.half + lane + 32 * j] = rotary_turn(pos, step[j], amplitude[j]);
      }
      __syncwarp();
      if (lane == 0) rsm::mbar_arrive(full + 8 * s);
    };
    // info runs with the loads; where a token goes is asked of the 32 at hand, so the last
    // round's places are kept for those still on their way out
    RotaryToken last{};
    auto prepare = [&](int64_t i, int s) {
      if (i % 32 == 0) last = mine;
      info(i, s);
    };
    for (int i = 0; i < S - 1 && i < count; ++i) prepare(i, i);
    int64_t asked = min(static_cast<int64_t>(S - 1), count);
    int s = 0, ask_s = S - 1;
    uint32_t phase = 0;
    for (int64_t i = 0; i < count; ++i) {
      if (!rsm::mbar_wait(done + 8 * s, phase, kRotaryTimeoutNs)) {  // (never expected)
        if (lane == 0) flag(p.status, RSM_STATUS_WAIT_TIMEOUT);
        bulk_wait_read<0>();
        for (int k = 0; k < S; ++k) (void)rsm::mbar_wait(full + 8 * k, k < s ? phase ^ 1u : phase, 1000000ull);  // copies on the way
        return;
      }
      // round 32 of tokens i belongs to `last` once `mine` is of the next one
      const bool old = i / 32 != (asked - 1) / 32;
      const int from = static_cast<int>(i % 32);
      auto of = [&](int64_t m, int64_t l) { return __shfl_sync(0xFFFFFFFFu, old ? l : m, from); };
      const int64_t out = of(mine.out, last.out), kr = of(mine.k_row, last.k_row), vr = of(mine.v_row, last.v_row);
      const int state = __shfl_sync(0xFFFFFFFFu, old ? last.live : mine.live, from);
      const uint32_t at = ring + s * token_bytes, qb = qn * sizeof(IT), kb = kn * sizeof(IT), hb = p.dim * sizeof(IT);
      if (lane == 0 && state != 0) bulk_store(static_cast<IT*>(p.q_out) + out, at, qb);
      if (kr >= 0) {
        if (pg.k_head_stride == p.dim || p.G == 1) {
          if (lane == 1) bulk_store(static_cast<IT*>(pg.k) + kr, at + qb, kb);
        } else {
          for (int g = lane; g < p.G; g += 32) bulk_store(static_cast<IT*>(pg.k) + kr + g * pg.k_head_stride, at + qb + g * hb, hb);
        }
        if (pg.v_head_stride == p.dim || p.G == 1) {
          if (lane == 2) bulk_store(static_cast<IT*>(pg.v) + vr, at + qb + kb, kb);
        } else {
          for (int g = lane; g < p.G; g += 32) bulk_store(static_cast<IT*>(pg.v) + vr + g * pg.v_head_stride, at + qb + kb + g * hb, hb);
        }
      }
      bulk_commit();
      if (asked < count) {
        bulk_wait_read<1>();  // the token before this one has left its place
        __syncwarp();
        load(asked, ask_s);
        prepare(asked, ask_s);
        ++asked;
        ask_s = ask_s + 1 == S ? 0 : ask_s + 1;
      }
      if (++s == S) s = 0, phase ^= 1u;
    }
    bulk_wait_read<0>();
    return;
  }

  // ---- the turning warps ----
  const bool near = p.interleaved != 0;
  const int parts = (near ? 2 * p.half : p.half) / V, items = (p.H + p.G) * parts;
  int s = 0;
  uint32_t phase = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (!rsm::mbar_wait(full + 8 * s, phase, kRotaryTimeoutNs)) {
      flag(p.status, RSM_STATUS_WAIT_TIMEOUT);
      return;
    }
    IT* const token = reinterpret_cast<IT*>(smem + s * token_bytes);
    const int state = live_s[s];
    if (state == 2) {
      const float2* const turn = turns + s * p.half;
      for (int k = threadIdx.x - 32; k < items; k += 32 * kWarps) {
        const int h = k / parts, j = k - h * parts;
        IT* const at = token + h * p.dim + j * V;
        Row<IT, V> a, b;
        float x[V], y[V], u[V], v[V];
        a.load(at);
        a.values(x);
        if (near) {
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const float2 w = turn[j * (V / 2) + e / 2];
            u[e] = x[e] * w.x - x[e + 1] * w.y;
            u[e + 1] = x[e + 1] * w.x + x[e] * w.y;
          }
        } else {
          b.load(at + p.half);
          b.values(y);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 w = turn[j * V + e];
            u[e] = x[e] * w.x - y[e] * w.y;
            v[e] = y[e] * w.x + x[e] * w.y;
          }
          b.round(v);
          b.store(at + p.half);
        }
        a.round(u);
        a.store(at);
      }
    } else if (state == 1) {  // a skipped request's queries
      for (int k = threadIdx.x - 32; k < qn / kWide; k += 32 * kWarps) *reinterpret_cast<uint4*>(token + k * kWide) = make_uint4(0, 0, 0, 0);
    }
    rsm::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) rsm::mbar_arrive(done + 8 * s);
    if (++s == S) s = 0, phase ^= 1u;
  }
}

// A CTA a token: few tokens, whose way through is shorter than a ring's, and with V = 1 any
// size, stride and alignment.  A thread's first row is on its way before the token is looked up, its next
// one before it stores (256 tokens of 56 fp32 heads of 128: 5.1 us, 5.6 of one row after the other).
template <typename IT, int V>
__global__ void __launch_bounds__(kRotaryPlainThreads) rotary_token_kernel(const __grid_constant__ RotaryParams p) {
  __shared__ RotaryToken token;
  __shared__ float2 turn[kRotaryMaxHalf];
  const rsm_pages& pg = p.pages;
  // A head's parts: V pairs of two halves (or V columns of neighbouring pairs), then V columns that stay
  const bool near = V > 1 && p.interleaved, near_one = V == 1 && p.interleaved;
  const int turning = (near ? 2 * p.half : p.half) / V, parts = turning + (p.dim - 2 * p.half) / V, items = (p.H + 2 * p.G) * parts;
  struct Item {
    Row<IT, V> a, b;
    int h, part, ca, cb;
  };
  int64_t q, k, v;
  if (p.cu != nullptr) {
    q = blockIdx.x * p.q_ts, k = blockIdx.x * p.k_ts, v = blockIdx.x * p.v_ts;
  } else {
    const int64_t b = blockIdx.x / static_cast<uint32_t>(p.window), t = blockIdx.x - b * p.window;
    q = b * p.q_bs + t * p.q_ts, k = b * p.k_bs + t * p.k_ts, v = b * p.v_bs + t * p.v_ts;
  }
  auto load = [&](int i) {
    Item it;
    it.h = i / parts;
    it.part = i - it.h * parts;
    it.ca = it.part >= turning ? 2 * p.half + (it.part - turning) * V : near_one ? 2 * it.part : it.part * V;
    it.cb = it.part >= turning || near ? it.ca : near_one ? it.ca + 1 : it.ca + p.half;
    const IT* from = it.h >= p.H + p.G ? static_cast<const IT*>(p.v) + v + static_cast<int64_t>(it.h - p.H - p.G) * p.dim
                     : it.h >= p.H     ? static_cast<const IT*>(p.k) + k + static_cast<int64_t>(it.h - p.H) * p.dim
                                       : static_cast<const IT*>(p.q) + q + static_cast<int64_t>(it.h) * p.dim;
    it.a.load(from + it.ca);
    if (it.cb != it.ca) it.b.load(from + it.cb);
    return it;
  };
  Item it;
  if (static_cast<int>(threadIdx.x) < items) it = load(threadIdx.x);
  uint64_t step = 0;
  float amplitude = 0.0f;
  if (static_cast<int>(threadIdx.x) < p.half) {
    const float f = p.inv_freq[threadIdx.x];
    step = turns_per_position(f), amplitude = amplitude_of(f, p.amplitude);
  }
  const int live = p.cu == nullptr ? 0 : live_sequences(p.cu, pg.requests, p.tokens, p.status, blockIdx.x == 0);
  if (threadIdx.x == kRotaryPlainThreads - 1) token = rotary_token(p, live, blockIdx.x);
  __syncthreads();
  const RotaryToken to = token;
  if (to.live == 0) return;
  if (static_cast<int>(threadIdx.x) < p.half) turn[threadIdx.x] = rotary_turn(to.pos, step, amplitude);
  __syncthreads();
  Item ahead;
  for (int i = threadIdx.x; i < items; i += kRotaryPlainThreads, it = ahead) {
    if (i + kRotaryPlainThreads < items) ahead = load(i + kRotaryPlainThreads);
    const bool query = it.h < p.H, value = it.h >= p.H + p.G;
    if (!query && to.k_row < 0) continue;
    IT* const row = query   ? static_cast<IT*>(p.q_out) + to.out + static_cast<int64_t>(it.h) * p.dim
                    : value ? static_cast<IT*>(pg.v) + to.v_row + (it.h - p.H - p.G) * pg.v_head_stride
                            : static_cast<IT*>(pg.k) + to.k_row + (it.h - p.H) * pg.k_head_stride;
    if (to.live == 1) {  // a skipped request's queries
      it.a.zero();
      it.b.zero();
    } else if (!value && it.part < turning) {
      float x[V], y[V], u[V], w[V];
      it.a.values(x);
      if (near) {
#pragma unroll
        for (int e = 0; e + 1 < V; e += 2) {
          const float2 cs = turn[it.part * (V / 2) + e / 2];
          u[e] = x[e] * cs.x - x[e + 1] * cs.y;
          u[e + 1] = x[e + 1] * cs.x + x[e] * cs.y;
        }
      } else {
        it.b.values(y);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 cs = turn[it.part * V + e];
          u[e] = x[e] * cs.x - y[e] * cs.y;
          w[e] = y[e] * cs.x + x[e] * cs.y;
        }
        it.b.round(w);
      }
      it.a.round(u);
    }
    it.a.store(row + it.ca);
    if (it.cb != it.ca) it.b.store(row + it.cb);
  }
}

}  // namespace hybrid
