// rotary_kernel.cuh -- rotary positions on the queries and keys of new tokens, keys
// and values to their pages.
//
// The angle p f of a far position has to be taken modulo a turn before it is rounded
// to 24 bits.  Here the fraction of a turn that one position makes, f / (2 pi) mod 1,
// is a 64-bit integer (in units of 2^-64 turns, from two-term fp64 products), so that
// times the position it wraps by itself: the error, a unit a position, stays below
// 2^-32 turns, and the upper 32 bits are what sine and cosine are taken of.
//
// Memory bounds it: q, k, v read once and written once.  A CTA stays for a run of tokens,
// kRotaryTokens at a time: eight warps move them, each thread the same 16 bytes (twice
// that for two halves of a head) of a head for all the tokens; a ninth meanwhile
// looks up where the next ones go, which takes three loads that wait for one another, and
// makes their sines and cosines, once for all heads.
#pragma once
#include "hybrid_device.cuh"

namespace hybrid {

constexpr int kRotaryMaxHalf = 128, kRotaryTokens = 4;

struct RotaryToken {
  int64_t q, k, v, out;   // element offsets of the token's rows
  int64_t k_row, v_row;   // of its rows in the pages; -1: none
  uint32_t pos;
  int live;               // 0: no sequence's, 1: a skipped request's, 2: to be done
};

// f / (2 pi) mod 1 in units of 2^-64.  1 / (2 pi) is given to 106 bits, as the sum of two doubles.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double d = fabs(static_cast<double>(f)), t = d * hi, e = fma(d, hi, -t) + d * lo;
  const double part = t - floor(t);  // exact: part has no bits that t has not
  const uint64_t n = __double2ull_rz(part * 0x1p64) + static_cast<uint64_t>(__double2ll_rn(e * 0x1p64));
  return f < 0.0f ? 0 - n : n;
}

template <typename IT, int V>
__global__ void __launch_bounds__(kRotaryThreads, kRotaryCtas) rotary_append_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int kMovers = kRotaryThreads - 32, T = kRotaryTokens;
  __shared__ RotaryToken token_s[2][T];
  __shared__ uint64_t step[kRotaryMaxHalf];
  __shared__ float2 turn_s[2][T * kRotaryMaxHalf];
  const int64_t begin = blockIdx.x * p.tokens / gridDim.x, end = (blockIdx.x + 1) * p.tokens / gridDim.x;
  const rsm_pages& pg = p.pages;
  int live = 0;
  if (p.cu != nullptr) live = live_sequences(p.cu, pg.requests, p.tokens, p.status, blockIdx.x == 0);

  // ---- the ninth warp: tokens first .. first + T - 1 ----
  const int lane = threadIdx.x - kMovers;
  auto look_up = [&](int64_t first, int to) {
    if (lane < T && first + lane < end) {
      RotaryToken k;
      const int64_t i = first + lane;
      int64_t b, t, n;
      k.live = 1;
      if (p.cu != nullptr) {
        b = sequence_at(p.cu, live, i);
        t = n = 0;
        if (b == live || p.cu[b] < 0 || p.cu[b] > i || p.cu[b + 1] > p.tokens)
          k.live = 0;
        else
          t = i - p.cu[b], n = p.cu[b + 1] - p.cu[b];
        k.q = i * p.q_ts, k.k = i * p.k_ts, k.v = i * p.v_ts, k.out = i * p.out_ts;
      } else {
        b = i / p.window, t = i - b * p.window, n = p.window;
        k.q = b * p.q_bs + t * p.q_ts, k.k = b * p.k_bs + t * p.k_ts, k.v = b * p.v_bs + t * p.v_ts;
        k.out = b * p.out_bs + t * p.out_ts;
      }
      k.pos = 0;
      k.k_row = k.v_row = -1;
      if (k.live != 0) {
        const int64_t len = pg.lengths[b];
        if (len < n || len > static_cast<int64_t>(pg.table_width) * pg.page_size) {
          if (len != 0) flag(p.status, RSM_STATUS_BAD_POSITION);
        } else {
          k.live = 2;
          k.pos = static_cast<uint32_t>(len - n + t);
          const uint32_t at = k.pos / static_cast<uint32_t>(pg.page_size);
          const int64_t row = k.pos - at * static_cast<uint32_t>(pg.page_size);
          const int page = pg.page_table[b * pg.table_stride + at];
          if (page < 0 || page >= pg.num_pages)
            flag(p.status, RSM_STATUS_BAD_PAGE);
          else
            k.k_row = page * pg.k_page_stride + row * pg.k_row_stride, k.v_row = page * pg.v_page_stride + row * pg.v_row_stride;
        }
      }
      token_s[to][lane] = k;
    }
    __syncwarp();
    for (int t = 0; t < T && first + t < end; ++t) {
      const uint32_t pos = token_s[to][t].pos;
      for (int j = lane; j < p.half; j += 32) {
        const int32_t upper = static_cast<int32_t>(static_cast<uint32_t>((pos * step[j]) >> 32));
        float s, c;
        sincospif(static_cast<float>(upper) * 0x1p-31f, &s, &c);
        turn_s[to][t * p.half + j] = make_float2(c * p.amplitude, s * p.amplitude);
      }
    }
  };

  // ---- the movers' parts of a head: those that turn (V pairs from two halves, or V / 2
  // neighbouring ones), then those that are copied; a value head is copied whole ----
  const bool near = V > 1 && p.interleaved, near_one = V == 1 && p.interleaved;
  const uint32_t turning = V > 1 ? (near ? 2 * p.half / V : p.half / V) : p.half;
  const uint32_t parts = turning + (p.dim - 2 * p.half) / V, copied = p.dim / V;
  const uint32_t heads = (p.H + p.G) * parts, per = heads + p.G * copied;
  auto move = [&](uint32_t i, int of, int nt) {
    const bool value = i >= heads;
    const uint32_t in = value ? i - heads : i, h = in / (value ? copied : parts), part = in - h * (value ? copied : parts);
    const bool key = !value && h >= static_cast<uint32_t>(p.H);
    const uint32_t g = key ? h - p.H : h;
    const bool turns = !value && part < turning;
    // columns of the part, and of its other half
    const uint32_t ca = value ? part * V : !turns ? 2 * p.half + (part - turning) * V : near_one ? 2 * part : part * V;
    const uint32_t cb = near_one ? ca + 1 : ca + p.half;
    const bool two = turns && !near;
    const IT* const from = (value ? static_cast<const IT*>(p.v) : key ? static_cast<const IT*>(p.k) : static_cast<const IT*>(p.q)) +
                           static_cast<int64_t>(g) * p.dim;
    IT* const to = value ? static_cast<IT*>(pg.v) + g * pg.v_head_stride
                   : key ? static_cast<IT*>(pg.k) + g * pg.k_head_stride
                         : static_cast<IT*>(p.q_out) + static_cast<int64_t>(g) * p.dim;
    const RotaryToken* const token = token_s[of];
    Row<IT, V> a[T], b[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
      if (t < nt) {
        const RotaryToken& k = token[t];
        if (k.live == 2) {
          const IT* row = from + (value ? k.v : key ? k.k : k.q);
          a[t].load(row + ca);
          if (two) b[t].load(row + cb);
        } else {
          a[t].zero();  // a skipped request's queries
          b[t].zero();
        }
      }
#pragma unroll
    for (int t = 0; t < T; ++t)
      if (t < nt) {
        const RotaryToken& k = token[t];
        const int64_t row = value ? k.v_row : key ? k.k_row : k.live == 0 ? -1 : k.out;
        if (row < 0) continue;
        if (turns) {
          float x[V], y[V], u[V], v[V];
          const float2* cs = turn_s[of] + t * p.half;
          a[t].values(x);
          if (near) {
#pragma unroll
            for (int j = 0; j + 1 < V; j += 2) {
              const float2 w = cs[part * (V / 2) + j / 2];
              u[j] = x[j] * w.x - x[j + 1] * w.y;
              u[j + 1] = x[j + 1] * w.x + x[j] * w.y;
            }
            a[t].round(u);
          } else {
            b[t].values(y);
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const float2 w = cs[part * V + j];
              u[j] = x[j] * w.x - y[j] * w.y;
              v[j] = y[j] * w.x + x[j] * w.y;
            }
            a[t].round(u);
            b[t].round(v);
            b[t].store(to + row + cb);
          }
        }
        a[t].store(to + row + ca);
      }
  };

  if (lane >= 0) {
    for (int j = lane; j < p.half; j += 32) step[j] = turns_per_position(p.inv_freq[j]);
    __syncwarp();
    look_up(begin, 0);
  }
  __syncthreads();
  int of = 0;
  for (int64_t first = begin; first < end; first += T, of ^= 1) {
    if (lane >= 0) {
      if (first + T < end) look_up(first + T, of ^ 1);
    } else {
      const int nt = static_cast<int>(min(static_cast<int64_t>(T), end - first));
      for (uint32_t i = threadIdx.x; i < per; i += kMovers) move(i, of, nt);
    }
    __syncthreads();
  }
}

}  // namespace hybrid
