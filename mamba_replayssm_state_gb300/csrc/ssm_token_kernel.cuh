// ssm_token_kernel.cuh -- new tokens of running requests, 64 x 128 states: the
// recurrent form (state slot to state slot) and the ring form (state only read).
//
// Ring form.  With tokens s = 0 .. m-1 (the ring's, then the T new ones), a_s =
// dt_s A and c_t = a_0 + .. + a_t, token t's output is
//   y_t = e^{c_t} S C_t + sum_{s<=t} (e^{c_t - c_s} dt_s (B_s . C_t) + [s = t] D) x_s,
// so the state is read once, whatever T and the ring's length, and the dots B_s .
// C_t belong to the group, not the head.
//
// Memory bounds both: the states' bytes, once (ring form) or once each way.  Measured on
// a GB300, 256 requests of 256 heads, bf16: one token to the state itself 343 us, 6.3
// TB/s; one token after a ring of 8 174 us, 6.4 TB/s; 64 requests: 4 tokens to the state
// 116 us, 4.6 TB/s, 4 after a ring of 16 52 us, 5.2 TB/s.  Instructions bound one-byte
// states (64 requests, 4 tokens, int8: 49 us, 3.7 TB/s).  A CTA
// takes heads of one request and group.  One round of loads stages what their
// tokens need; then four warps share a head, 16 dim rows each, and go through the
// CTA's heads two at a time, asking for the next head's rows as soon as the last's
// have had their use.
//
// With bf16 inputs the products are on the tensor cores (mma.sync m16n8k16: 16 rows, 8
// tokens), the state as bf16: exact for bf16, int8 and fp8, as hi + lo for fp16 (exact)
// and fp32 (within 2^-17).  The weights of the tokens, D in a token's own, are rounded to
// bf16.  Several tokens to the state itself are an empty ring's, and the update, of the state
// as it is, one product more, w x in it as hi + lo (within 2^-17).  A lane takes 16 bytes of a row at a time, k being numbered to suit.  (Rows through shared memory by
// bulk copies, two or three heads ahead, measured slower: what they take of it is CTAs,
// and with them the heads in whose time another CTA's staging passes.)
//
// Otherwise (fp32 inputs, one token to the state, one after a ring on fp16 states, more
// than eight to the state) a lane holds eight dstate columns of eight rows: sixteen lanes to a
// row, a 16-byte load (16-bit states) an instruction and two rows.  Sums over a
// row's sixteen lanes are taken for eight rows at once, halving the values at each
// exchange: eight shuffles, not 32; lane l then has row 2 ((l >> 1) & 7) + (l >> 4), the
// same in lanes 2i and 2i + 1, which split the ring's tokens by parity.
#pragma once
#include <cuda_runtime.h>

#include "rsm_ptx.cuh"
#include "ssm_seq_kernel.cuh"

namespace ssm {

constexpr int kTokThreads = kTokenThreads;
constexpr int kTokMaxNew = kTokenMaxNew;
constexpr int kTokMaxAll = kTokenMaxAll;
constexpr int kTokD = 64, kTokN = 128;
constexpr int kTokRows = 16;      // dim rows of a warp
constexpr int kTokMaxHeads = kTokenMaxHeads;  // of a CTA
constexpr int kTokLoads = 8;      // row pairs of a warp

// raw bytes of eight consecutive state elements
template <int SF> struct Raw { uint4 v; };
template <> struct Raw<RSM_F32> { float4 a, b; };
template <> struct Raw<RSM_I8> { uint2 v; };
template <> struct Raw<RSM_FP8_E4M3> { uint2 v; };

__device__ __forceinline__ uint4 ldg128_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg64_once(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
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

// Shared memory of a CTA, in bytes: what its heads' tokens need, staged by one
// round of loads; `all` is the most tokens a request can have (ring and new).
struct TokLayout {
  uint32_t C, B, x, dt, c, dot, w, e, bytes;
};
// elements between staged rows of B, and of x: on the tensor cores 16 bytes off a multiple of 128
__host__ __device__ constexpr int tok_B_row(int mode) { return kTokN + (mode >= 3 ? 8 : 0); }
__host__ __device__ constexpr int tok_x_row(int mode, int heads) { return heads * kTokD + (mode >= 3 ? 8 : 0); }
__host__ __device__ inline TokLayout tok_layout(int mode, int input_bytes, int heads, int fresh, int all) {
  const bool ring_form = mode == 0 || mode >= 3;
  TokLayout l{};
  uint32_t at = 0;
  auto take = [&](uint32_t n) {
    const uint32_t o = at;
    at += (n + 15u) & ~15u;
    return o;
  };
  const uint32_t all16 = (all + 15u) & ~15u, fresh8 = (fresh + 7u) & ~7u;
  // (ring form: B as stored, for the dots alone; tensor cores: C too)
  l.C = take(mode >= 3 ? fresh * tok_B_row(mode) * input_bytes : fresh * kTokN * 4);
  l.B = take((mode >= 3 ? all16 * tok_B_row(mode) : all * kTokN) * (ring_form ? input_bytes : 4));
  l.x = take(mode >= 3 ? all16 * tok_x_row(mode, heads) * input_bytes : all * heads * kTokD * input_bytes);
  l.dt = take(all * heads * 4);
  l.c = take(ring_form ? all * heads * 4 : 0);
  l.dot = take(ring_form ? fresh * all * 4 : 0);
  l.w = take(mode >= 3 ? heads * fresh8 * all16 * 2 : mode == 0 ? heads * fresh * all * 4 : 0);
  l.e = take(heads * fresh * 4);
  l.bytes = at;
  return l;
}

// Copies `rows` rows of `n` contiguous elements into shared memory, `stride` apart, a warp
// a row, row r from from(r): asynchronously, 16 bytes at a time, where every row allows it.
template <typename IT, typename From>
__device__ __forceinline__ void stage_rows(IT* to, int stride, int rows, int n, bool wide, From from) {
  constexpr int V = 16 / sizeof(IT);
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < rows; r += kTokThreads / 32) {
    const IT* f = from(r);
    IT* t = to + r * stride;
    if (wide) {
      for (int k = lane * V; k < n; k += 32 * V) rsm::cp_async_16(rsm::smem_addr(t + k), f + k);
    } else {
      for (int k = lane; k < n; k += 32) t[k] = f[k];
    }
  }
}
// ... and out of it, to to(r)
template <typename IT, typename To>
__device__ __forceinline__ void put_rows(const IT* from, int stride, int rows, int n, bool wide, To to) {
  constexpr int V = 16 / sizeof(IT);
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < rows; r += kTokThreads / 32) {
    const IT* f = from + r * stride;
    IT* t = to(r);
    if (wide) {
      for (int k = lane * V; k < n; k += 32 * V) *reinterpret_cast<uint4*>(t + k) = *reinterpret_cast<const uint4*>(f + k);
    } else {
      for (int k = lane; k < n; k += 32) t[k] = f[k];
    }
  }
}
__device__ __forceinline__ void staged() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// A lane's share of a row, 32 elements, as the bf16 pairs of eight k-steps, two a step:
// element pair_at(i, tq) and its neighbour (int8: the next but one) in pair i.
//
// An int8 code is 128 + its low seven bits, which is bf16 0x4300 with those for its
// mantissa, and -128, or -256 where it is negative: 3.5 instructions a pair against 5
// through fp32.  Its pairs are bytes 0 and 2, then 1 and 3, of each word.
template <int SF>
__device__ __forceinline__ constexpr int pair_at(int i, int tq) {
  return SF == RSM_F32 ? 16 * (i >> 1) + 4 * tq + 2 * (i & 1)
       : SF == RSM_BF16 || SF == RSM_F16 ? 32 * (i >> 2) + 8 * tq + 2 * (i & 3)
                        : 64 * (i >> 3) + 16 * tq + 4 * ((i >> 1) & 3) + (i & 1) * (SF == RSM_I8 ? 1 : 2);
}
template <int SF>
__device__ __forceinline__ void word_pairs(uint32_t w, uint32_t& a, uint32_t& b) {  // of one-byte states
  if constexpr (SF == RSM_I8) {
    const uint32_t u = w >> 8;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(a) : "r"((w & 0x007F007Fu) | 0x43004300u), "r"((w & 0x00800080u) | 0xC300C300u));
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(b) : "r"((u & 0x007F007Fu) | 0x43004300u), "r"((u & 0x00800080u) | 0xC300C300u));
  } else {
    const float2 lo = rsm::e4m3x2_to_f32(w & 0xFFFFu), hi = rsm::e4m3x2_to_f32(w >> 16);
    a = rsm::pack_bf16x2(lo.x, lo.y);
    b = rsm::pack_bf16x2(hi.x, hi.y);
  }
}

// Pair i of a lane's share of a row of a wider state, and as bf16 hi + lo: exact for
// fp16, within 2^-17 for fp32.
template <int SF, int P>
__device__ __forceinline__ float2 state_pair(const uint4 (&row)[P], int i) {
  if constexpr (SF == RSM_F32) {
    const uint4 u = row[i >> 1];
    return i & 1 ? make_float2(__uint_as_float(u.z), __uint_as_float(u.w)) : make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  } else {
    const uint4 u = row[i >> 2];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (SF == RSM_F16)
      return rsm::f16x2_to_f32(w[i & 3]);
    else
      return make_float2(rsm::bf16lo(w[i & 3]), rsm::bf16hi(w[i & 3]));
  }
}
__device__ __forceinline__ void split_pair(float2 v, uint32_t& hi, uint32_t& lo) {
  hi = rsm::pack_bf16x2(v.x, v.y);
  lo = bounded_lo(rsm::pack_bf16x2(v.x - rsm::bf16lo(hi), v.y - rsm::bf16hi(hi)));
}

// D += A B: 16 rows x 16 k, 16 k x 8 columns, bf16 in, fp32 sums
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// MODE: 0 the ring form, 1 one new token a request, state to state, 2 several; 3
// and 4 the ring form on the tensor cores, up to 8 and up to 16 new tokens; 5 up to 8
// new tokens, state to state, in the ring form with an empty ring.
template <typename IT, int SF, int MODE>
__global__ void __launch_bounds__(kTokThreads, SF == RSM_F32 || MODE == 1 || MODE == 2 || MODE >= 4 ? 2 : 3) ssm_token_kernel(const __grid_constant__ Params p) {
  constexpr int ES = SF == RSM_F32 ? 4 : (SF == RSM_BF16 || SF == RSM_F16) ? 2 : 1;
  constexpr int D = kTokD, N = kTokN;
  constexpr bool STEP = MODE == 1 || MODE == 2;
  constexpr bool MMA = MODE >= 3, KEEP = MODE == 5;  // on the tensor cores; whose states are stored
  constexpr int NT = MODE == 4 ? 2 : 1;  // eights of new tokens
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hpg = p.H / p.G, per = p.heads_per_cta, parts = (hpg + per - 1) / per;
  const uint32_t bg = blockIdx.x / static_cast<uint32_t>(parts);
  const int part = static_cast<int>(blockIdx.x - bg * static_cast<uint32_t>(parts));
  const int b = static_cast<int>(bg / static_cast<uint32_t>(p.G)), g = static_cast<int>(bg - static_cast<uint32_t>(b) * p.G);
  const int h0 = g * hpg + part * per, nh = min(per, (g + 1) * hpg - h0);
  const int T = p.window;
  const bool say = g == 0 && part == 0 && tid == 0;

  int n_ring = 0, ring0 = 0;
  if constexpr (!STEP && !KEEP) {
    ring0 = __ldg(p.ring_start + b);
    n_ring = __ldg(p.ring_len + b);
  }
  const int src = slot_of(p, p.src, b, say);
  int dst = src;
  bool live = src >= 0;
  if constexpr (STEP || KEEP) {
    if (p.dst != nullptr) dst = slot_of(p, p.dst, b, say);
  }
  // this lane's eight columns of its warp's row pairs, in a head's tile (tensor
  // cores: 16 bytes of row lane / 4, and of that + 8, and those 64 bytes on)
  const int row0 = kTokRows * (warp & 3) + (MMA ? lane >> 2 : lane >> 4);
  const int64_t off = static_cast<int64_t>(row0) * (N * ES) + (MMA ? 16 * (lane & 3) : 8 * ES * (lane & 15)) +
                      h0 * (static_cast<int64_t>(D) * N * ES);
  constexpr int64_t kTileBytes = static_cast<int64_t>(D) * N * ES;
  const unsigned char* from = static_cast<const unsigned char*>(p.state) + src * p.state_ss * ES + off;
  Raw<SF> raw[MMA ? 1 : kTokLoads];
  constexpr int kPieces = 2 * ES;
  uint4 rows[MMA ? 2 : 1][MMA ? kPieces : 1];
  auto load_head = [&](int hl) {
    if (hl < nh) {
      const unsigned char* at = from + hl * kTileBytes;
      if constexpr (MMA) {
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          rows[0][c] = ldg128_once(at + 64 * c);
          rows[1][c] = ldg128_once(at + 8 * N * ES + 64 * c);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kTokLoads; ++i) load_raw<SF>(raw[i], at + i * (2 * N * ES));
      }
    }
  };
  if (live) load_head(warp >> 2);
  if constexpr (!STEP && !KEEP) {
    if (live) {
      uint32_t bad = 0;
      if (ring0 < 0 || ring0 >= p.R) bad |= RSM_STATUS_BAD_RING_START;
      if (n_ring < 0 || n_ring > p.R - T || n_ring > kTokMaxAll - T) bad |= RSM_STATUS_BAD_PREFIX_LEN;
      if (say) flag(p.status, bad);
      live = bad == 0;
    }
  }
  IT* out = static_cast<IT*>(p.out) + static_cast<int64_t>(b) * p.out_bs + static_cast<int64_t>(h0) * D;
  if (!live) {
    const int n = nh * D;
    for (int i = tid; i < T * n; i += kTokThreads) store_in(out + (i / n) * p.out_ts + i % n, 0.0f);
    return;
  }

  // one round of loads for everything but the state
  const TokLayout l = tok_layout(MODE, sizeof(IT), per, T, p.tokens_max);
  const int xs = tok_x_row(MODE, nh);
  float* sC = reinterpret_cast<float*>(smem + l.C);
  IT* sx = reinterpret_cast<IT*>(smem + l.x);
  float* sdt = reinterpret_cast<float*>(smem + l.dt);
  float* se = reinterpret_cast<float*>(smem + l.e);
  const IT* xn = static_cast<const IT*>(p.x) + static_cast<int64_t>(b) * p.x_bs + static_cast<int64_t>(h0) * D;
  const IT* Bn = static_cast<const IT*>(p.B) + static_cast<int64_t>(b) * p.B_bs + static_cast<int64_t>(g) * N;
  const IT* Cn = static_cast<const IT*>(p.C) + static_cast<int64_t>(b) * p.C_bs + static_cast<int64_t>(g) * N;
  const float* dtn = p.dt + static_cast<int64_t>(b) * p.dt_bs + h0;
  const int m = n_ring + T;
  const bool wide = p.wide != 0;
  if constexpr (!MMA)
    for (int i = tid; i < T * N; i += kTokThreads) sC[i] = as_float(Cn[(i / N) * p.C_ts + i % N]);
  if constexpr (STEP) {
    float* sB = reinterpret_cast<float*>(smem + l.B);
    for (int i = tid; i < T * N; i += kTokThreads) sB[i] = as_float(Bn[(i / N) * p.B_ts + i % N]);
    stage_rows(sx, xs, T, nh * D, wide, [&](int r) { return xn + r * p.x_ts; });
    for (int t = tid >> 4; t < T; t += kTokThreads / 16)  // sixteen lanes a token, one a head
      if ((tid & 15) < nh) sdt[t * nh + (tid & 15)] = __ldg(dtn + t * p.dt_ts + (tid & 15));
    staged();
    __syncthreads();
  } else {
    constexpr int BS = tok_B_row(MODE);
    IT* sB = reinterpret_cast<IT*>(smem + l.B);
    float* sc = reinterpret_cast<float*>(smem + l.c);
    float* sdot = reinterpret_cast<float*>(smem + l.dot);
    const int T8 = (T + 7) & ~7, m16 = (m + 15) & ~15;
    auto ring_row = [&](int s) {
      const int r = ring0 + s;
      return static_cast<int64_t>(r < p.R ? r : r - p.R);  // ring0 < R, s < R
    };
    IT* xc = static_cast<IT*>(p.x_cache) + src * p.xc_ss + static_cast<int64_t>(h0) * D;
    IT* Bc = static_cast<IT*>(p.B_cache) + src * p.Bc_ss + static_cast<int64_t>(g) * N;
    float* dtc = p.dt_cache + src * p.dtc_ss + h0;
    const int64_t xrow = static_cast<int64_t>(p.H) * D, Brow = static_cast<int64_t>(p.G) * N;
    stage_rows(sx, xs, m, nh * D, wide,
               [&](int s) -> const IT* { return s < n_ring ? xc + ring_row(s) * xrow : xn + (s - n_ring) * p.x_ts; });
    stage_rows(sB, BS, m, N, wide,
               [&](int s) -> const IT* { return s < n_ring ? Bc + ring_row(s) * Brow : Bn + (s - n_ring) * p.B_ts; });
    if constexpr (MMA) stage_rows(reinterpret_cast<IT*>(smem + l.C), BS, T, N, wide, [&](int t) { return Cn + t * p.C_ts; });
    const int hq = tid & 15;  // sixteen lanes a token, one a head
    const float A = hq < nh ? __ldg(p.A + h0 + hq) : 0.0f;
    for (int s = tid >> 4; s < m; s += kTokThreads / 16)
      if (hq < nh)
        rsm::cp_async_4(rsm::smem_addr(sdt + s * nh + hq), s < n_ring ? dtc + ring_row(s) * p.H + hq : dtn + (s - n_ring) * p.dt_ts + hq);
    if constexpr (MMA)  // the rest of the last k-step: weight 0, and so finite
      for (int i = tid; i < (m16 - m) * xs; i += kTokThreads) sx[m * xs + i] = IT(0);
    static_assert(kTokMaxHeads <= 2 * (kTokThreads / 32), "a warp has two heads' weights at most");
    const bool has_skip = p.D != nullptr;
    const float skip0 = has_skip && warp < nh ? __ldg(p.D + h0 + warp) : 0.0f;
    const float skip1 = has_skip && warp + kTokThreads / 32 < nh ? __ldg(p.D + h0 + warp + kTokThreads / 32) : 0.0f;
    staged();
    __syncthreads();

    // the new tokens join the ring, B once for the group
    if constexpr (!KEEP) {
      put_rows(sx + n_ring * xs, xs, T, nh * D, wide, [&](int t) { return xc + ring_row(n_ring + t) * xrow; });
      if (part == 0) put_rows(sB + n_ring * BS, BS, T, N, wide, [&](int t) { return Bc + ring_row(n_ring + t) * Brow; });
      for (int t = tid >> 4; t < T; t += kTokThreads / 16)
        if (hq < nh) dtc[ring_row(n_ring + t) * p.H + hq] = sdt[(n_ring + t) * nh + hq];
    }

    // The decays (dt A summed) and the dots B_s . C_t.  With bf16 inputs the decays are those up
    // to and with each token, and a pair's is the difference of two: sums up to 2^14 leave the
    // weight within 2^-9, half its rounding.  With fp32 inputs a strong decay would take from the pairs after it,
    // so a ring token's is from it to the ring's end, a new one's from there up to and
    // with it, and a pair's their sum, of one sign, or for two new tokens that of the tokens between.
    // (For bf16 inputs too: 256 requests, rings of 8, 186 us for 175; 32 requests, rings of 64, 90 for 79.
    // With fp32 inputs it costs nothing: 32 requests of 256 heads, 4 tokens, rings of 16, 71 us; 8, rings of 64, 585.)
    // (bf16, few: each by itself; many: a warp scans.  256 heads, rings of 64, 32 requests, 4 tokens,
    // fp32 states: 76 us, 80 without the scan; rings of 8, 256 requests, bf16: 177 us with it, 175 without)
    constexpr bool BY_PARTS = sizeof(IT) == 4;
    if constexpr (BY_PARTS) {
      for (int hl = warp; hl < nh; hl += kTokThreads / 32) {
        const float Ah = __ldg(p.A + h0 + hl);
        auto scan = [&](float v) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float w = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += w;
          }
          return v;
        };
        float sum = 0.0f;  // of the ring's tokens after these 32
        for (int s0 = n_ring - 1; s0 >= 0; s0 -= 32) {
          const int s = s0 - lane;
          const float v = scan(s >= 0 && s + 1 < n_ring ? sdt[(s + 1) * nh + hl] : 0.0f) + sum;
          if (s >= 0) sc[s * nh + hl] = v * Ah;
          sum = __shfl_sync(0xFFFFFFFFu, v, 31);
        }
        const float v = scan(lane < T ? sdt[(n_ring + lane) * nh + hl] : 0.0f);  // (T <= 16)
        if (lane < T) sc[(n_ring + lane) * nh + hl] = v * Ah;
      }
    } else if (m <= 16) {
      if (hq < nh) {
        for (int s = tid >> 4; s < m; s += kTokThreads / 16) {
          float sum = 0.0f;
#pragma unroll 4
          for (int k = 0; k <= s; ++k) sum += sdt[k * nh + hq];
          sc[s * nh + hq] = sum * A;
        }
      }
    } else {
      for (int hl = warp; hl < nh; hl += kTokThreads / 32) {
        const float Ah = __ldg(p.A + h0 + hl);
        float sum = 0.0f;  // up to the 32 tokens before
        for (int s0 = 0; s0 < m; s0 += 32) {
          const int s = s0 + lane;
          float v = s < m ? sdt[s * nh + hl] : 0.0f;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float w = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += w;
          }
          v += sum;
          if (s < m) sc[s * nh + hl] = v * Ah;
          sum = __shfl_sync(0xFFFFFFFFu, v, 31);
        }
      }
    }
    if constexpr (MMA) {
      // sixteen tokens' B a warp against the new tokens' C (rows past m: whatever is there, for dots nobody takes)
      const IT* sCb = reinterpret_cast<const IT*>(smem + l.C);
      for (int s0 = 16 * (kTokThreads / 32 - 1 - warp); s0 < m; s0 += 16 * (kTokThreads / 32)) {
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[nt][q] = 0.0f;
        const uint32_t bm = rsm::smem_addr(sB) + 2u * ((s0 + (lane & 15)) * BS + 8 * (lane >> 4));
        const IT* ct[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ct[nt] = sCb + min(8 * nt + (lane >> 2), T - 1) * BS + 2 * (lane & 3);
#pragma unroll
        for (int k = 0; k < N; k += 16) {
          uint32_t a0, a1, a2, a3;
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                       : "r"(bm + 2u * k));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(acc[nt], a0, a1, a2, a3, *reinterpret_cast<const uint32_t*>(ct[nt] + k),
                     *reinterpret_cast<const uint32_t*>(ct[nt] + k + 8));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int s = s0 + (lane >> 2) + 8 * (q >> 1), t = 8 * nt + 2 * (lane & 3) + (q & 1);
            if (s < m && t < T) sdot[t * m + s] = acc[nt][q];
          }
      }
    } else {
      for (int i = tid >> 2; i < ((m * T + 7) & ~7); i += kTokThreads / 4) {  // four lanes a dot, whole warps
        const int s = i % m, t = i / m;
        float dot = 0.0f;
        if (t < T) {
#pragma unroll 8
          for (int k = 0; k < N / 4; ++k) dot = fmaf(as_float(sB[s * N + 4 * k + (tid & 3)]), sC[t * N + 4 * k + (tid & 3)], dot);
        }
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, 1);
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, 2);
        if ((tid & 3) == 0 && t < T) sdot[t * m + s] = dot;
      }
    }
    __syncthreads();

    // the tokens' weights, a warp per head
    for (int hl = warp; hl < nh; hl += kTokThreads / 32) {
      const float skip = hl == warp ? skip0 : skip1;
      const float Ah = BY_PARTS ? __ldg(p.A + h0 + hl) : 0.0f;
      auto weight = [&](int s, int t, float between) {  // between: dt of the tokens between two new ones (by parts)
        const int now = n_ring + t;
        if (s > now || t >= T) return 0.0f;
        const float decay = !BY_PARTS ? __expf(sc[now * nh + hl] - sc[s * nh + hl])
                                      : expf(s < n_ring ? sc[s * nh + hl] + sc[now * nh + hl] : between * Ah);
        return fmaf(decay * sdt[s * nh + hl], sdot[t * m + s], s == now ? skip : 0.0f);
      };
      if constexpr (BY_PARTS) {
        const float ring = n_ring > 0 ? fmaf(sdt[hl], Ah, sc[hl]) : 0.0f;
        for (int t = lane; t < T; t += 32) se[hl * T + t] = expf(ring + sc[(n_ring + t) * nh + hl]);
      } else {
        for (int t = lane; t < T; t += 32) se[hl * T + t] = __expf(sc[(n_ring + t) * nh + hl]);
      }
      if constexpr (MMA) {
        // pairs of tokens, eight lanes to sixteen of them
        const uint32_t q = m16 >> 4, inv = 65536u / q + 1u;
        uint32_t* w = reinterpret_cast<uint32_t*>(smem + l.w) + hl * T8 * (m16 >> 1);
        for (uint32_t i = lane; i < static_cast<uint32_t>(T8 * (m16 >> 1)); i += 32) {
          const uint32_t t = ((i >> 3) * inv) >> 16, s = 2 * (i - t * (m16 >> 1));
          w[i] = rsm::pack_bf16x2(weight(s, t, 0.0f), weight(s + 1, t, 0.0f));
        }
      } else {
        float* w = reinterpret_cast<float*>(smem + l.w) + hl * T * m;
        if constexpr (BY_PARTS) {
          for (int s = lane; s < m; s += 32) {
            float between = 0.0f;
            for (int t = 0; t < T; ++t) {
              if (s >= n_ring && n_ring + t > s) between += sdt[(n_ring + t) * nh + hl];
              w[t * m + s] = weight(s, t, between);
            }
          }
        } else {
          for (int t = 0; t < T; ++t)
            for (int s = lane; s < m; s += 32) w[t * m + s] = weight(s, t, 0.0f);
        }
      }
    }
    __syncthreads();
  }
  if constexpr (STEP) {
    for (int i = tid; i < nh * T; i += kTokThreads) se[i] = expf(sdt[(i % T) * nh + i / T] * __ldg(p.A + h0 + i / T));
    __syncthreads();
  }

  if constexpr (MMA) {
    const int gq = lane >> 2, tq = lane & 3, T8 = (T + 7) & ~7, m16 = (m + 15) & ~15;
    uint32_t cf[NT][16];  // tokens' C as the second operand
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int t = 8 * nt + gq;
      const uint32_t* ct = reinterpret_cast<const uint32_t*>(smem + l.C) + min(t, T - 1) * (tok_B_row(MODE) / 2);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        uint32_t v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) v[k] = ct[pair_at<SF>(i + (SF == RSM_I8 ? 0 : k), tq) / 2 + (SF == RSM_I8 ? k : 0)];
        if constexpr (SF == RSM_I8) {  // elements 0 and 2, 1 and 3 of four
          const uint32_t even = __byte_perm(v[0], v[1], 0x5410), other = __byte_perm(v[0], v[1], 0x7632);
          v[0] = even;
          v[1] = other;
        }
        cf[nt][i] = t < T ? v[0] : 0u;
        cf[nt][i + 1] = t < T ? v[1] : 0u;
      }
    }
    uint32_t bf[KEEP ? 16 : 1];  // tokens' B likewise, for the update: k is the token, twice
    if constexpr (KEEP) {
      const uint16_t* bt = reinterpret_cast<const uint16_t*>(smem + l.B) + 2 * tq * tok_B_row(MODE) + (gq & 1);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int el = pair_at<SF>(i, gq >> 1);
        const uint32_t lo = 2 * tq < T ? bt[el] : 0u, hi = 2 * tq + 1 < T ? bt[tok_B_row(MODE) + el] : 0u;
        bf[i] = lo | hi << 16;
      }
    }
    const uint16_t* sw = reinterpret_cast<const uint16_t*>(smem + l.w);
    // rows of x for ldmatrix: lanes 0-7 tokens 0-7, columns 0-7; 8-15 columns 8-15; 16-31 tokens 8-15
    const uint32_t xm = rsm::smem_addr(sx) + 2u * (((lane & 7) + ((lane >> 4) << 3)) * xs + kTokRows * (warp & 3) + 8 * ((lane >> 3) & 1));
#pragma unroll 1
    for (int hl = warp >> 2; hl < nh; hl += 2) {
      float acc[NT][4], ring[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[nt][q] = ring[nt][q] = 0.0f;
      float scale[2] = {1.0f, 1.0f};
      if constexpr (ES == 1) {
        const float* sc = p.scale + src * p.scale_ss + static_cast<int64_t>(h0 + hl) * D + kTokRows * (warp & 3) + gq;
        scale[0] = __ldg(sc);
        scale[1] = __ldg(sc + 8);
      }
      if constexpr (SF == RSM_F32 || SF == RSM_F16) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) split_pair(state_pair<SF>(rows[q & 1], i + (q >> 1)), hi[q], lo[q]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(acc[nt], hi[0], hi[1], hi[2], hi[3], cf[nt][i], cf[nt][i + 1]);
            mma16816(acc[nt], lo[0], lo[1], lo[2], lo[3], cf[nt][i], cf[nt][i + 1]);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const uint4 r0 = rows[0][c], r1 = rows[1][c];
          const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
          if constexpr (ES == 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(acc[nt], w0[2 * k], w1[2 * k], w0[2 * k + 1], w1[2 * k + 1], cf[nt][4 * c + 2 * k], cf[nt][4 * c + 2 * k + 1]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t a0, a1, a2, a3;
              word_pairs<SF>(w0[k], a0, a2);
              word_pairs<SF>(w1[k], a1, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(acc[nt], a0, a1, a2, a3, cf[nt][8 * c + 2 * k], cf[nt][8 * c + 2 * k + 1]);
            }
          }
        }
      }
      if constexpr (KEEP) {
        // S <- e^{c_last} S + sum_s (e^{c_last - c_s} dt_s x_s) (x) B_s, a product over the tokens: w x as
        // bf16 hi in k = 0..7 and lo in 8..15 (16 bits), the decays after a token summed from the end
        const float A = __ldg(p.A + h0 + hl), e = se[hl * T + T - 1];
        float after = 0.0f, w0 = 0.0f, w1 = 0.0f;
        for (int s = T - 1; s >= 0; --s) {
          const float d = sdt[s * nh + hl];
          if (s == 2 * tq) w0 = expf(after * A) * d;
          if (s == 2 * tq + 1) w1 = expf(after * A) * d;
          after += d;
        }
        const IT* xr = sx + 2 * tq * xs + hl * D + kTokRows * (warp & 3) + gq;  // (past T: zeros)
        uint32_t a[4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          split_pair(make_float2(w0 * as_float(xr[8 * q]), w1 * as_float(xr[xs + 8 * q])), a[q], a[q + 2]);
        unsigned char* to = static_cast<unsigned char*>(p.state) + dst * p.state_ss * ES + off + hl * kTileBytes;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          uint32_t out0[4], out1[4];
#pragma unroll
          for (int q = 0; q < 8 / ES; ++q) {
            const int i = (8 / ES) * c + q;
            const float2 r0 = state_pair<SF>(rows[0], i), r1 = state_pair<SF>(rows[1], i);
            float v[4] = {e * r0.x, e * r0.y, e * r1.x, e * r1.y};
            mma16816(v, a[0], a[1], a[2], a[3], bf[i], bf[i]);
            if constexpr (SF == RSM_F32) {
              out0[2 * q] = __float_as_uint(v[0]), out0[2 * q + 1] = __float_as_uint(v[1]);
              out1[2 * q] = __float_as_uint(v[2]), out1[2 * q + 1] = __float_as_uint(v[3]);
            } else {
              out0[q] = SF == RSM_F16 ? rsm::pack_f16x2(v[0], v[1]) : rsm::pack_bf16x2(v[0], v[1]);
              out1[q] = SF == RSM_F16 ? rsm::pack_f16x2(v[2], v[3]) : rsm::pack_bf16x2(v[2], v[3]);
            }
          }
          if (dst >= 0) {
            *reinterpret_cast<uint4*>(to + 64 * c) = make_uint4(out0[0], out0[1], out0[2], out0[3]);
            *reinterpret_cast<uint4*>(to + 8 * N * ES + 64 * c) = make_uint4(out1[0], out1[1], out1[2], out1[3]);
          }
        }
      }
      load_head(hl + 2);  // the rows have had their use
#pragma unroll 1
      for (int s0 = 0; s0 < m; s0 += 16) {
        uint32_t a0, a1, a2, a3;
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                     : "r"(xm + 2u * (s0 * xs + hl * D)));
        const uint16_t* wt = sw + (hl * T8 + gq) * m16 + s0 + 2 * tq;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816(ring[nt], a0, a1, a2, a3, *reinterpret_cast<const uint32_t*>(wt + nt * 8 * m16),
                   *reinterpret_cast<const uint32_t*>(wt + nt * 8 * m16 + 8));
      }
      IT* outh = out + hl * D + kTokRows * (warp & 3) + gq;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int t = 8 * nt + 2 * tq + (q & 1);
          if (t < T) store_in(outh + t * p.out_ts + 8 * (q >> 1), fmaf(acc[nt][q], se[hl * T + t] * scale[q >> 1], ring[nt][q]));
        }
    }
    return;
  }
  const int r = 2 * ((lane >> 1) & 7) + (lane >> 4);      // the row this lane ends with
  const int d = kTokRows * (warp & 3) + r, odd = lane & 1;
#pragma unroll 1
  for (int hl = warp >> 2; hl < nh; hl += 2) {
    IT* outh = out + hl * D + d;
    const IT* xh = sx + hl * D + d;
    if constexpr (STEP) {
      const float* sB = reinterpret_cast<const float*>(smem + l.B);
      const float skip = p.D != nullptr ? __ldg(p.D + h0 + hl) : 0.0f;
      unsigned char* to = static_cast<unsigned char*>(p.state) + dst * p.state_ss * ES + off + hl * kTileBytes;
      constexpr int kHold = MODE == 2 ? kTokLoads : 1;  // row pairs held as fp32
      float2 S[kHold][4];
      if constexpr (MODE == 2) {
#pragma unroll
        for (int i = 0; i < kTokLoads; ++i) unpack<SF>(raw[i], S[i]);
      }
#pragma unroll 1
      for (int t = 0; t < T; ++t) {
        const float a = se[hl * T + t], x = as_float(xh[t * xs]), u = sdt[t * nh + hl] * x;
        const float4* Bt = reinterpret_cast<const float4*>(sB + t * N + 8 * (lane & 15));
        const float4* Ct = reinterpret_cast<const float4*>(sC + t * N + 8 * (lane & 15));
        const float4 b0 = Bt[0], b1 = Bt[1], c0 = Ct[0], c1 = Ct[1];
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
        if constexpr (MODE == 1) load_head(hl + 2);
        float y = fold8(acc, lane);
        y += __shfl_xor_sync(0xFFFFFFFFu, y, 1);
        if (!odd) store_in(outh + t * p.out_ts, fmaf(skip, x, y));
      }
      if constexpr (MODE == 2) {
        if (dst >= 0) {
#pragma unroll
          for (int i = 0; i < kTokLoads; ++i) store_eight<SF>(to + i * (2 * N * ES), S[i]);
        }
        load_head(hl + 2);
      }
    } else if constexpr (MODE == 0) {
      const float* sw = reinterpret_cast<const float*>(smem + l.w);
      const float scale = (SF == RSM_I8 || SF == RSM_FP8_E4M3)
                              ? __ldg(p.scale + src * p.scale_ss + static_cast<int64_t>(h0 + hl) * D + d) : 1.0f;
#pragma unroll 1
      for (int t = 0; t < T; ++t) {
        const float4* Ct = reinterpret_cast<const float4*>(sC + t * N + 8 * (lane & 15));
        const float4 c0 = Ct[0], c1 = Ct[1];
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
        if (t == T - 1) load_head(hl + 2);  // the rows have had their last use
        float y = fold8(acc, lane) * (se[hl * T + t] * scale);
        const float* wt = sw + (hl * T + t) * m;
        for (int s = odd; s <= n_ring + t; s += 2) y = fmaf(wt[s], as_float(xh[s * xs]), y);
        y += __shfl_xor_sync(0xFFFFFFFFu, y, 1);
        if (!odd) store_in(outh + t * p.out_ts, y);
      }
    }
  }
}

}  // namespace ssm
