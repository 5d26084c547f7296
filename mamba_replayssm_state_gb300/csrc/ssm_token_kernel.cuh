// ssm_token_kernel.cuh -- new tokens of running requests, 64 x 128 states: the
// recurrent form (state slot to state slot) and the ring form (state only read).
//
// Ring form.  With tokens s = 0 .. m-1 (the ring's, then the T new ones), a_s =
// dt_s A and c_t = a_0 + .. + a_t, token t's output is
//   y_t = e^{c_t} S C_t + sum_{s<=t} (e^{c_t - c_s} dt_s (B_s . C_t) + [s = t] D) x_s,
// so the state is read once, whatever T and the ring's length, and the dots B_s .
// C_t belong to the group, not the head.
//
// Memory bounds both: the states' bytes, once (ring form) or once each way.  A CTA
// takes heads of one request and group; four warps share a head, 16 dim rows each,
// and go through the CTA's heads two at a time, asking for the next head's rows as
// soon as the last's have had their use, before the sums and the ring's part.  A lane holds eight dstate columns of eight
// rows: sixteen lanes to a row, a 16-byte load (16-bit states) an instruction and two
// rows.  Sums over a row's sixteen lanes are taken for eight rows at once, halving the
// values at each exchange: eight shuffles, not 32; lane l then has row 2 ((l >> 1) & 7)
// + (l >> 4), the same in lanes 2i and 2i + 1, which split the ring's tokens by parity.
#pragma once
#include <cuda_runtime.h>

#include "ssm_seq_kernel.cuh"

namespace ssm {

constexpr int kTokThreads = kTokenThreads;
constexpr int kTokMaxNew = kTokenMaxNew;
constexpr int kTokMaxAll = 64;    // with the ring's
constexpr int kTokRows = 16;      // dim rows of a warp
constexpr int kTokLoads = 8;      // row pairs of a warp

// raw bytes of eight consecutive state elements
template <int SF> struct Raw { uint4 v; };
template <> struct Raw<RSM_F32> { float4 a, b; };
template <> struct Raw<RSM_I8> { uint2 v; };
template <> struct Raw<RSM_FP8_E4M3> { uint2 v; };

__device__ __forceinline__ uint4 ldg128_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg64_once(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int SF>
__device__ __forceinline__ void load_raw(Raw<SF>& r, const unsigned char* p) {
  if constexpr (SF == RSM_F32) {
    const uint4 a = ldg128_once(p), b = ldg128_once(p + 16);
    r.a = make_float4(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w));
    r.b = make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w));
  } else if constexpr (SF == RSM_BF16 || SF == RSM_F16) {
    r.v = ldg128_once(p);
  } else {
    r.v = ldg64_once(p);
  }
}

template <int SF>
__device__ __forceinline__ void unpack(const Raw<SF>& r, float2 (&v)[4]) {
  if constexpr (SF == RSM_F32) {
    v[0] = make_float2(r.a.x, r.a.y), v[1] = make_float2(r.a.z, r.a.w);
    v[2] = make_float2(r.b.x, r.b.y), v[3] = make_float2(r.b.z, r.b.w);
  } else if constexpr (SF == RSM_BF16) {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(rsm::bf16lo(w[i]), rsm::bf16hi(w[i]));
  } else if constexpr (SF == RSM_F16) {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = rsm::f16x2_to_f32(w[i]);
  } else if constexpr (SF == RSM_I8) {
    // a code + 128 as the last byte of 2^23 + code + 128, exactly; then the offset goes
    const uint32_t w[2] = {r.v.x ^ 0x80808080u, r.v.y ^ 0x80808080u};
    const float2 off = make_float2(-8388736.0f, -8388736.0f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7440)),
                                        __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7441))), off);
      v[2 * i + 1] = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7442)),
                                            __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7443))), off);
    }
  } else {
    v[0] = rsm::e4m3x2_to_f32(r.v.x & 0xFFFFu);
    v[1] = rsm::e4m3x2_to_f32(r.v.x >> 16);
    v[2] = rsm::e4m3x2_to_f32(r.v.y & 0xFFFFu);
    v[3] = rsm::e4m3x2_to_f32(r.v.y >> 16);
  }
}

template <int SF>
__device__ __forceinline__ void store_eight(unsigned char* p, const float2 (&v)[4]) {
  if constexpr (SF == RSM_F32) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  } else if constexpr (SF == RSM_BF16) {
    *reinterpret_cast<uint4*>(p) = make_uint4(rsm::pack_bf16x2(v[0].x, v[0].y), rsm::pack_bf16x2(v[1].x, v[1].y),
                                              rsm::pack_bf16x2(v[2].x, v[2].y), rsm::pack_bf16x2(v[3].x, v[3].y));
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(rsm::pack_f16x2(v[0].x, v[0].y), rsm::pack_f16x2(v[1].x, v[1].y),
                                              rsm::pack_f16x2(v[2].x, v[2].y), rsm::pack_f16x2(v[3].x, v[3].y));
  }
}

// Eight rows' sums over the sixteen lanes that share them, but for the last
// exchange (lanes 2i and 2i + 1), which the caller's other terms can join.
__device__ __forceinline__ float fold8(float (&v)[8], int lane) {
#pragma unroll
  for (int w = 4; w >= 1; w >>= 1) {
    const bool up = (lane & (2 * w)) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float keep = up ? v[i + w] : v[i], give = up ? v[i] : v[i + w];
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 2 * w);
    }
  }
  return v[0];
}

// MODE: 0 the ring form, 1 one new token a request, state to state, 2 several.
template <typename IT, int SF, int MODE>
__global__ void __launch_bounds__(kTokThreads, MODE == 2 ? 2 : 3) ssm_token_kernel(const __grid_constant__ Params p) {
  constexpr int ES = SF == RSM_F32 ? 4 : (SF == RSM_BF16 || SF == RSM_F16) ? 2 : 1;
  constexpr int D = 64, N = 128;
  constexpr bool STEP = MODE != 0;
  __shared__ __align__(16) float sC[kTokMaxNew][N];
  __shared__ __align__(16) float sB[STEP ? kTokMaxNew : 1][N];
  __shared__ float sdot[STEP ? 1 : kTokMaxNew][kTokMaxAll];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hpg = p.H / p.G, per = p.heads_per_cta, parts = (hpg + per - 1) / per;
  const uint32_t bg = blockIdx.x / static_cast<uint32_t>(parts);
  const int part = static_cast<int>(blockIdx.x - bg * static_cast<uint32_t>(parts));
  const int b = static_cast<int>(bg / static_cast<uint32_t>(p.G)), g = static_cast<int>(bg - static_cast<uint32_t>(b) * p.G);
  const int h0 = g * hpg + part * per, h1 = min(h0 + per, (g + 1) * hpg);
  const int T = p.window;
  const bool say = g == 0 && part == 0 && tid == 0;

  const int src = slot_of(p, p.src, b, say);
  int dst = src, n_ring = 0, ring0 = 0;
  bool live = src >= 0;
  if constexpr (STEP) {
    if (p.dst != nullptr) dst = slot_of(p, p.dst, b, say);
  } else if (live) {
    ring0 = __ldg(p.ring_start + b);
    n_ring = __ldg(p.ring_len + b);
    uint32_t bad = 0;
    if (ring0 < 0 || ring0 >= p.R) bad |= RSM_STATUS_BAD_RING_START;
    if (n_ring < 0 || n_ring > p.R - T || n_ring > kTokMaxAll - T) bad |= RSM_STATUS_BAD_PREFIX_LEN;
    if (say) flag(p.status, bad);
    live = bad == 0;
  }
  IT* out = static_cast<IT*>(p.out) + static_cast<int64_t>(b) * p.out_bs;
  if (!live) {
    const int n = (h1 - h0) * D;
    for (int i = tid; i < T * n; i += kTokThreads) store_in(out + (i / n) * p.out_ts + h0 * D + i % n, 0.0f);
    return;
  }

  // this lane's eight columns of its warp's row pairs, in a head's tile
  const int row0 = kTokRows * (warp & 3) + (lane >> 4);
  const int64_t off = static_cast<int64_t>(row0 * N + 8 * (lane & 15)) * ES;
  const int64_t tile = static_cast<int64_t>(D) * N * ES;
  const unsigned char* from = static_cast<const unsigned char*>(p.state) + src * p.state_ss * ES + off;
  const int hfirst = h0 + (warp >> 2);
  Raw<SF> raw[kTokLoads];
  if (hfirst < h1) {
#pragma unroll
    for (int i = 0; i < kTokLoads; ++i) load_raw<SF>(raw[i], from + hfirst * tile + i * (2 * N * ES));
  }

  // the group's part: C (and B, or the dots B . C) of the tokens
  const IT* Bn = static_cast<const IT*>(p.B) + static_cast<int64_t>(b) * p.B_bs + static_cast<int64_t>(g) * N;
  const IT* Cn = static_cast<const IT*>(p.C) + static_cast<int64_t>(b) * p.C_bs + static_cast<int64_t>(g) * N;
  const IT* Bc = STEP ? nullptr : static_cast<const IT*>(p.B_cache) + src * p.Bc_ss + static_cast<int64_t>(g) * N;
  const int m = n_ring + T;
  for (int i = tid; i < T * N; i += kTokThreads) {
    const int t = i / N, n = i % N;
    sC[t][n] = load_in(Cn + t * p.C_ts + n);
    if constexpr (STEP) sB[t][n] = load_in(Bn + t * p.B_ts + n);
  }
  if constexpr (!STEP) {
    for (int s = warp; s < m; s += kTokThreads / 32) {
      const int64_t ring_row = (ring0 + s) % p.R;
      const IT* Bs = s < n_ring ? Bc + ring_row * p.G * N : Bn + static_cast<int64_t>(s - n_ring) * p.B_ts;
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = load_in(Bs + lane + 32 * k);
      if (s >= n_ring && part == 0) {  // a new token's B joins the ring, once for the group
        IT* to = static_cast<IT*>(p.B_cache) + src * p.Bc_ss + (ring_row * p.G + g) * N;
#pragma unroll
        for (int k = 0; k < 4; ++k) store_in(to + lane + 32 * k, v[k]);
      }
      for (int t = max(0, s - n_ring); t < T; ++t) {
        const IT* Ct = Cn + t * p.C_ts;
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) dot = fmaf(v[k], load_in(Ct + lane + 32 * k), dot);
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        if (lane == 0) sdot[t][s] = dot;
      }
    }
  }
  __syncthreads();

  const int r = 2 * ((lane >> 1) & 7) + (lane >> 4);      // the row this lane ends with
  const int d = kTokRows * (warp & 3) + r, odd = lane & 1;
  const IT* xn = static_cast<const IT*>(p.x) + static_cast<int64_t>(b) * p.x_bs;
  const float* dtn = p.dt + static_cast<int64_t>(b) * p.dt_bs;

  for (int h = hfirst; h < h1; h += 2) {
    const float A = __ldg(p.A + h);
    const float skip = p.D != nullptr ? __ldg(p.D + h) : 0.0f;
    const bool more = h + 2 < h1;
    auto load_next = [&] {
      if (more) {
#pragma unroll
        for (int i = 0; i < kTokLoads; ++i) load_raw<SF>(raw[i], from + (h + 2) * tile + i * (2 * N * ES));
      }
    };
    if constexpr (STEP) {
      unsigned char* to = static_cast<unsigned char*>(p.state) + dst * p.state_ss * ES + off + h * tile;
      constexpr int kHold = MODE == 2 ? kTokLoads : 1;  // row pairs held as fp32
      float2 S[kHold][4];
      if constexpr (MODE == 2) {
#pragma unroll
        for (int i = 0; i < kTokLoads; ++i) unpack<SF>(raw[i], S[i]);
        if constexpr (ES < 4) load_next();
      }
#pragma unroll 1
      for (int t = 0; t < T; ++t) {
        const float dt = __ldg(dtn + t * p.dt_ts + h), x = load_in(xn + t * p.x_ts + static_cast<int64_t>(h) * D + d);
        const float a = expf(dt * A), u = dt * x;
        const float4 b0 = *reinterpret_cast<const float4*>(&sB[t][8 * (lane & 15)]);
        const float4 b1 = *reinterpret_cast<const float4*>(&sB[t][8 * (lane & 15) + 4]);
        const float4 c0 = *reinterpret_cast<const float4*>(&sC[t][8 * (lane & 15)]);
        const float4 c1 = *reinterpret_cast<const float4*>(&sC[t][8 * (lane & 15) + 4]);
        const float2 B2[4] = {make_float2(b0.x, b0.y), make_float2(b0.z, b0.w), make_float2(b1.x, b1.y), make_float2(b1.z, b1.w)};
        const float2 C2[4] = {make_float2(c0.x, c0.y), make_float2(c0.z, c0.w), make_float2(c1.x, c1.y), make_float2(c1.z, c1.w)};
        const float2 a2 = make_float2(a, a);
        float acc[8];
#pragma unroll
        for (int i = 0; i < kTokLoads; ++i) {
          const int k = MODE == 2 ? i : 0;
          if constexpr (MODE == 1) unpack<SF>(raw[i], S[0]);
          const float ui = __shfl_sync(0xFFFFFFFFu, u, (lane & 16) | (i << 1));
          const float2 u2 = make_float2(ui, ui);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            S[k][q] = __ffma2_rn(a2, S[k][q], __fmul2_rn(u2, B2[q]));
            sum = __ffma2_rn(S[k][q], C2[q], sum);
          }
          acc[i] = sum.x + sum.y;
          if constexpr (MODE == 1)
            if (dst >= 0) store_eight<SF>(to + i * (2 * N * ES), S[0]);
        }
        if constexpr (MODE == 1) load_next();
        float y = fold8(acc, lane);
        y += __shfl_xor_sync(0xFFFFFFFFu, y, 1);
        if (!odd) store_in(out + t * p.out_ts + static_cast<int64_t>(h) * D + d, fmaf(skip, x, y));
      }
      if constexpr (MODE == 2) {
        if (dst >= 0) {
#pragma unroll
          for (int i = 0; i < kTokLoads; ++i) store_eight<SF>(to + i * (2 * N * ES), S[i]);
        }
        if constexpr (ES == 4) load_next();
      }
    } else {
      // the tokens' decays: token s in lane s % 32's word s / 32
      float dts[2], c[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int s = lane + 32 * k;
        dts[k] = 0.0f;
        if (s < m) {
          float* ring = p.dt_cache + src * p.dtc_ss + static_cast<int64_t>((ring0 + s) % p.R) * p.H + h;
          dts[k] = s < n_ring ? __ldg(ring) : __ldg(dtn + static_cast<int64_t>(s - n_ring) * p.dt_ts + h);
          if (s >= n_ring && (warp & 3) == 0) *ring = dts[k];
        }
        c[k] = dts[k] * A;
      }
      const float scale = (SF == RSM_I8 || SF == RSM_FP8_E4M3)
                              ? __ldg(p.scale + src * p.scale_ss + static_cast<int64_t>(h) * D + d) : 1.0f;
      // the first tokens' x of this lane's row; lanes 2i, 2i + 1 take every other token
      const IT* xr = static_cast<const IT*>(p.x_cache) + src * p.xc_ss + static_cast<int64_t>(h) * D + d;
      auto x_of = [&](int s) -> float {
        return s < n_ring ? load_in(xr + static_cast<int64_t>((ring0 + s) % p.R) * p.H * D)
                          : load_in(xn + static_cast<int64_t>(s - n_ring) * p.x_ts + static_cast<int64_t>(h) * D + d);
      };
      constexpr int kHeld = 4;  // tokens of a lane held in registers
      float x[kHeld];
#pragma unroll
      for (int k = 0; k < kHeld; ++k) x[k] = 2 * k + odd < m ? x_of(2 * k + odd) : 0.0f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float v = __shfl_up_sync(0xFFFFFFFFu, c[k], o);
          if (lane >= o) c[k] += v;
        }
      }
      c[1] += __shfl_sync(0xFFFFFFFFu, c[0], 31);

#pragma unroll 1
      for (int t = 0; t < T; ++t) {
        const int now = n_ring + t;
        const float4 c0 = *reinterpret_cast<const float4*>(&sC[t][8 * (lane & 15)]);
        const float4 c1 = *reinterpret_cast<const float4*>(&sC[t][8 * (lane & 15) + 4]);
        const float2 C2[4] = {make_float2(c0.x, c0.y), make_float2(c0.z, c0.w), make_float2(c1.x, c1.y), make_float2(c1.z, c1.w)};
        float acc[8];
#pragma unroll
        for (int i = 0; i < kTokLoads; ++i) {
          float2 S[4];
          unpack<SF>(raw[i], S);
          float2 sum = __fmul2_rn(S[0], C2[0]);
#pragma unroll
          for (int q = 1; q < 4; ++q) sum = __ffma2_rn(S[q], C2[q], sum);
          acc[i] = sum.x + sum.y;
        }
        if (t == T - 1) load_next();  // the rows have had their last use
        const float ct = __shfl_sync(0xFFFFFFFFu, now < 32 ? c[0] : c[1], now & 31);
        float y = fold8(acc, lane) * (expf(ct) * scale);
        float w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int s = lane + 32 * k;
          w[k] = s <= now ? expf(ct - c[k]) * dts[k] * sdot[t][s] : 0.0f;
          if (s == now) w[k] += skip;
        }
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
          const float ws = __shfl_sync(0xFFFFFFFFu, w[0], 2 * k + odd);
          y = 2 * k + odd <= now ? fmaf(ws, x[k], y) : y;
        }
        for (int k = kHeld; 2 * k <= now; ++k) {
          const int s = 2 * k + odd;
          const float ws = __shfl_sync(0xFFFFFFFFu, s < 32 ? w[0] : w[1], s & 31);
          if (s <= now) y = fmaf(ws, x_of(s), y);
        }
        y += __shfl_xor_sync(0xFFFFFFFFu, y, 1);
        if (!odd) store_in(out + t * p.out_ts + static_cast<int64_t>(h) * D + d, y);
        // the token's x joins the ring
        if (odd == (now & 1))
          store_in(const_cast<IT*>(xr) + static_cast<int64_t>((ring0 + now) % p.R) * p.H * D,
                   load_in(xn + t * p.x_ts + static_cast<int64_t>(h) * D + d));
      }
    }
  }
}

}  // namespace ssm
