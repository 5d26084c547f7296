// ssm_tc_kernel.cuh -- prompts on the tensor cores: the chunked form of linear
// attention with a decay for each head (bf16 inputs, 64 x 128 states).
//
// With a_t = dt_t A, a chunk of 128 tokens that starts from state S gives
//   y_i = e^{a_0+..+a_i} S C_i + sum_{j<=i} (C_i . B_j) e^{a_{j+1}+..+a_i} dt_j x_j,
//   S  <- e^{a_0+..+a_127} S + sum_j w_j x_j (x) B_j,    w_j = e^{a_{j+1}+..+a_127} dt_j,
// four matrix products, all tcgen05.mma with M = 128:
//   G  = C B^T           [i, j]       once for the CTA's heads, which share B and C
//   Y1 = C S^T           [i, (h, d)]
//   Y2 = P X             [i, d]       P = G o decay o dt, masked, in tensor memory as bf16
//   U  = B^T (w X)       [n, (h, d)]  w X as bf16 hi + lo (16 bits), or hi alone for bf16 states
// and y = e^{..} Y1 + Y2.  The skip term D x is a D on P's diagonal.
//
// Decays are products of factors that are all at most 1: a chunk is four blocks of
// 32 tokens, and a pair (i, j) of blocks k > b decays by e^{sum over i's block up
// to i} e^{blocks between} e^{rest of j's block}; only pairs of one block take an
// exponential of their own.  Sums run inside a block, so their rounding does
// not grow with the chunk, and nothing overflows or is divided.
//
// One persistent CTA per SM takes units (sequence, segment, two heads of one
// group; one head where a group has an odd number), all chunks of a unit in order:
//   warp 0       loads C, B and x (two stages each) with tensor-map copies
//   warp 1       issues the MMAs; warps 2, 3 stage dt, a head each
//   warps 4-11   four a head: P; a thread holds row i; G from tensor memory, P back into it
//   warps 12-15  w X: a thread holds token t's row; x becomes w x in place
//   warps 16-23  four a head: y out of Y1 and Y2; the state in registers as
//                fp32, a thread per dstate column, and its bf16 copy for Y1
// A sequence's last chunk may be partial: dt counts as 0 there, and the rows of
// x and B past its end, which are a neighbour's or nobody's, are cleared
// before an MMA multiplies them by 0.
//
// Every wait is bounded; one that runs out flags RSM_STATUS_WAIT_TIMEOUT, and
// all roles leave, drain the copies in flight and free the tensor memory.
#pragma once
#include <cuda_runtime.h>

#include "rsm_formats.cuh"
#include "rsm_ptx.cuh"
#include "rsm_tc.cuh"
#include "ssm_seq_kernel.cuh"
#include "ssm_tc_params.h"

namespace ssm {

using rsm::fence_proxy_async_smem;
using rsm::mbar_arrive;
using rsm::mbar_init;
using rsm::tc_commit;
using rsm::tc_fence_after;
using rsm::tc_fence_before;

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// Shared-memory descriptors with the 128-byte swizzle, as (low, high) words:
// the low word holds the start address and the first stride, both in 16 bytes,
// so that moving along K adds to it alone.  K-major: groups of 8 rows 1024
// bytes apart, 16 elements of K 32 bytes inside the swizzle atom.  MN-major:
// 64 elements of M or N to an atom, atoms a tile apart along M or N and 1024
// bytes (8 rows of K) along K.
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr) { return (saddr >> 4) | ((kTile >> 4) << 16); }

// D[tmem] (+)= A * B^T, A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// The same with A in tensor memory: 128 lanes, two bf16 of K to a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}

// 16 columns of this thread's lane, as they are.  Whole warp.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 16 columns of this thread's lane from each of two places.  Whole warp.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, float (&a)[16], float (&b)[16]) {
  uint32_t r[16], s[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
        "=&r"(s[0]), "=&r"(s[1]), "=&r"(s[2]), "=&r"(s[3]), "=&r"(s[4]), "=&r"(s[5]), "=&r"(s[6]), "=&r"(s[7]),
        "=&r"(s[8]), "=&r"(s[9]), "=&r"(s[10]), "=&r"(s[11]), "=&r"(s[12]), "=&r"(s[13]), "=&r"(s[14]), "=&r"(s[15])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(s[i]);
  }
}

// 32 bytes of a row, streaming past L1
__device__ __forceinline__ void stg256(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lds(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 lds4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// ---------------------------------------------------------------------------
// the units of this CTA, walked alike by every role
// ---------------------------------------------------------------------------
struct Unit {
  int64_t t0;           // first token
  int len;              // tokens
  int seq, seg, group;  // sequence, segment among all sequences', heads' group
  bool last;            // last segment of the sequence
  bool split;           // its state comes from the segment states
};

struct Walk {
  const TcParams& tp;
  uint32_t u;         // next unit
  int seq = 0;        // sequence under the cursor
  uint32_t base = 0;  // segments before it
  int64_t t0 = 0;
  uint32_t len = 0, nseg = 0;
  bool flagger;       // the one thread of the CTA that reports

  __device__ Walk(const TcParams& tp_, bool flagger_) : tp(tp_), u(blockIdx.x), flagger(flagger_) { look(); }

  __device__ void look() {
    if (seq >= tp.p.units) return;
    t0 = __ldg(tp.p.cu_seqlens + seq);
    const int64_t t1 = __ldg(tp.p.cu_seqlens + seq + 1);
    len = static_cast<uint32_t>(t1 - t0);
    if (t0 < 0 || t1 < t0 || t1 > tp.p.tokens) {
      if (flagger) flag(tp.p.status, RSM_STATUS_BAD_SEQUENCE);
      len = 0;
      nseg = 0;  // no unit at all
    } else {
      nseg = len <= tp.seg ? 1 : (len + tp.seg - 1) / tp.seg;
    }
  }
  __device__ bool next(Unit& w) {
    for (;;) {
      const uint32_t sg = u / static_cast<uint32_t>(tp.pairs);
      while (seq < tp.p.units && sg >= base + nseg) {
        base += nseg;
        ++seq;
        look();
      }
      if (seq >= tp.p.units) return false;
      const uint32_t s = sg - base;
      w.group = static_cast<int>(u - sg * static_cast<uint32_t>(tp.pairs));
      u += gridDim.x;
      w.last = s == nseg - 1;
      w.split = nseg > 1;
      if (tp.states_only && w.last) continue;  // nothing follows its state
      w.seq = seq;
      w.seg = static_cast<int>(sg);
      w.t0 = t0 + static_cast<int64_t>(s) * tp.seg;
      w.len = static_cast<int>(min(tp.seg, len - s * tp.seg));
      return true;
    }
  }
};

// ---------------------------------------------------------------------------
// decays of a chunk's tokens, in units of log2
// ---------------------------------------------------------------------------
struct Scan {
  float dt;     // this thread's token (block `warp`, place `lane`)
  float upto;   // its block's sum up to and with it
  float after;  // its block's sum after it
  float t[4];   // the blocks' sums
};

__device__ __forceinline__ Scan scan_chunk(uint32_t dt_addr, float A2, int block, int lane) {
  Scan s;
  float a_own = 0.0f;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float d = lds(dt_addr + static_cast<uint32_t>(b * 32 + lane) * 4u);
    const float a = d * A2;
    float t = a;
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    s.t[b] = t;
    if (b == block) {
      s.dt = d;
      a_own = a;
    }
  }
  float up = a_own, down = a_own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_up_sync(0xFFFFFFFFu, up, o);
    const float y = __shfl_down_sync(0xFFFFFFFFu, down, o);
    if (lane >= o) up += x;
    if (lane + o < 32) down += y;
  }
  s.upto = up;
  down = __shfl_down_sync(0xFFFFFFFFu, down, 1);
  s.after = lane == 31 ? 0.0f : down;
  return s;
}

// ---------------------------------------------------------------------------
struct Cta {
  const TcParams& tp;
  unsigned char* smem;
  uint32_t base;
  uint32_t tmem;
  int warp, lane;
  volatile int* abort_flag;

  __device__ uint32_t bar(uint32_t b) const { return base + kOffBar + 8u * b; }
  // The phase of `parity` of a barrier has completed; false when the wait ran
  // out or another role has given up.
  __device__ __forceinline__ bool wait(uint32_t b, uint32_t parity) const {
    const uint32_t at = bar(b);
    if (rsm::mbar_try_wait(at, parity & 1u)) return true;
    const uint64_t t0 = rsm::global_timer_ns();
    for (uint32_t it = 1;; ++it) {
      if (rsm::mbar_try_wait(at, parity & 1u)) return true;
      if ((it & 255u) == 0u && (*abort_flag != 0 || rsm::global_timer_ns() - t0 > kTcTimeoutNs)) return false;
    }
  }
  __device__ bool wait_warp(uint32_t b, uint32_t parity) const {
    return __all_sync(0xFFFFFFFFu, wait(b, parity)) != 0;
  }
  __device__ void arrive_warp(uint32_t b) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  }
};

template <int NH, bool LO>
__device__ __forceinline__ bool run_loader(const Cta& c) {
  const TcParams& tp = c.tp;
  const bool state_in_x = LO && !tp.states_only;
  Walk walk(tp, c.lane == 0);
  Unit w;
  uint32_t j = 0, n_bc = 0, n_x = 0;  // chunk; copies issued so far
  const uint32_t per_group = static_cast<uint32_t>(tp.p.H / tp.p.G);
  const bool one = elect_one();
  bool ok = true;
  while (ok && walk.next(w)) {
    const int h0 = w.group * NH, g = static_cast<int>(static_cast<uint32_t>(h0) / per_group);
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u;
      const int row = static_cast<int>(w.t0 + c0);
      if (j >= 2 && !(ok = c.wait_warp(kEmptyBC + st, (j >> 1) - 1u))) break;
      if (one) {
        const uint32_t bc = c.bar(kFullBC + st);
        mbar_arrive_expect(bc, tp.states_only ? 2 * kTile : 4 * kTile);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!tp.states_only)
            tma_load_2d(c.base + kOffC + (2 * st + half) * kTile, &tp.C_map, g * kState + 64 * half, row, bc);
          tma_load_2d(c.base + kOffB + (2 * st + half) * kTile, &tp.B_map, g * kState + 64 * half, row, bc);
        }
      }
      ++n_bc;
      // the stage is free after the update two chunks ago, or, where that chunk's
      // state took it, after the Y1 of the last one
      if (state_in_x ? j >= 1 : j >= 2)
        if (!(ok = c.wait_warp(kEmptyX + st, state_in_x ? (j - 1u) >> 1 : (j >> 1) - 1u))) break;
      if (one) {
        const uint32_t xb = c.bar(kFullX + st);
        mbar_arrive_expect(xb, NH * kTile);
#pragma unroll
        for (int h = 0; h < NH; ++h)
          tma_load_2d(c.base + kOffX + (2 * st + h) * kTile, &tp.x_map, (h0 + h) * kDim, row, xb);
      }
      ++n_x;
    }
  }
  // no copy may land after the CTA has gone, whichever way the roles end
  for (uint32_t k = n_bc >= 2 ? n_bc - 2 : 0; k < n_bc; ++k)
    (void)rsm::mbar_wait(c.bar(kFullBC + (k & 1u)), (k >> 1) & 1u, kTcTimeoutNs);
  for (uint32_t k = n_x >= 2 ? n_x - 2 : 0; k < n_x; ++k)
    (void)rsm::mbar_wait(c.bar(kFullX + (k & 1u)), (k >> 1) & 1u, kTcTimeoutNs);
  return ok;
}

template <int NH>
__device__ __forceinline__ bool run_dt(const Cta& c, int h) {
  const TcParams& tp = c.tp;
  Walk walk(tp, false);
  Unit w;
  uint32_t j = 0;
  while (walk.next(w)) {
    const float* dt = tp.p.dt + w.t0 * tp.p.dt_ts + (w.group * NH + h);
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      float v[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int t = c0 + 32 * b + c.lane;
        v[b] = t < w.len ? __ldg(dt + static_cast<int64_t>(t) * tp.p.dt_ts) : 0.0f;
      }
      const uint32_t st = j & 1u;
      if (j >= 2 && !c.wait_warp(kEmptyDt + st, (j >> 1) - 1u)) return false;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        sts(c.base + kOffDt + ((st * 2 + h) * kChunk + 32 * b + c.lane) * 4u, v[b]);
      c.arrive_warp(kFullDt + st);
    }
  }
  return true;
}

// The whole warp walks and waits, so that addresses stay uniform; one thread issues.
template <int NH, bool LO>
__device__ __forceinline__ bool run_mma(const Cta& c) {
  const TcParams& tp = c.tp;
  Walk walk(tp, false);
  Unit w;
  uint32_t j = 0;
  constexpr uint32_t kIdG = rsm::idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t kIdY1 = rsm::idesc_bf16_f32(128, 64 * NH, false, true);
  constexpr uint32_t kIdPx = rsm::idesc_bf16_f32(128, 64, false, true);
  constexpr uint32_t kIdU = rsm::idesc_bf16_f32(128, 64 * NH, true, true);
  constexpr uint32_t kStepMn = 2048 / 16;  // 16 rows of K
  const uint32_t tm = c.tmem;
  const bool one = elect_one();

  auto issue_G = [&](uint32_t st) {
    tc_fence_after();
    if (one) {
      const uint32_t a = desc_k(c.base + kOffC + 2 * st * kTile), b = desc_k(c.base + kOffB + 2 * st * kTile);
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {  // 16 dstate columns each: 32 bytes, four to a 64-column tile
        const uint32_t o = (k >> 2) * (kTile / 16) + (k & 3) * 2;
        mma_ss(tm + kColG, a + o, b + o, kIdG, k > 0);
      }
      tc_commit(c.bar(kGFull));
    }
    __syncwarp();
  };

  while (walk.next(w)) {
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u;
      if (!tp.states_only) {
        // (the last chunk's P has been read out of G: its P barriers were waited for below)
        if (c0 == 0) {
          if (!c.wait_warp(kFullBC + st, j >> 1)) return false;
          issue_G(st);
        }
        // Y2 = P X
        if (!c.wait_warp(kFullX + st, j >> 1) || !c.wait_warp(kClean, j)) return false;
#pragma unroll 1
        for (uint32_t h = 0; h < NH; ++h) {
          if (!c.wait_warp(kPFull + h, j)) return false;
          if (j >= 1 && !c.wait_warp(kY2Empty + h, j - 1u)) return false;
          tc_fence_after();
          if (one) {
            const uint32_t b = desc_mn(c.base + kOffX + (2 * st + h) * kTile);
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k)
              mma_ts(tm + kColY2 + 64 * h, tm + kColP + 64 * h + 8 * k, b + k * kStepMn, kIdPx, k > 0);
            tc_commit(c.bar(kPxDone + h));
          }
          __syncwarp();
        }
        // Y1 = C S^T
        if (!c.wait_warp(kSFull, j)) return false;
        tc_fence_after();
        if (one) {
          const uint32_t a = desc_k(c.base + kOffC + 2 * st * kTile);
          const uint32_t b = desc_mn(c.base + (LO ? kOffX + 2 * (st ^ 1u) * kTile : kOffMore));
#pragma unroll
          for (uint32_t k = 0; k < 8; ++k)
            mma_ss(tm + kColV, a + (k >> 2) * (kTile / 16) + (k & 3) * 2, b + k * kStepMn, kIdY1, k > 0);
          tc_commit(c.bar(kY1Full));
          if (LO) tc_commit(c.bar(kEmptyX + (st ^ 1u)));
        }
        __syncwarp();
        // the next chunk's G while this one's w X is made
        if (c0 + kChunk < w.len) {
          if (!c.wait_warp(kFullBC + (st ^ 1u), (j + 1u) >> 1)) return false;
          issue_G(st ^ 1u);
        }
      } else if (!c.wait_warp(kFullBC + st, j >> 1)) {
        return false;
      }
      // U = B^T (w X), where Y1 was
      if (!c.wait_warp(kWFull, j)) return false;
      if (!tp.states_only || j >= 1)
        if (!c.wait_warp(kVRead, tp.states_only ? j - 1u : j)) return false;
      tc_fence_after();
      if (one) {
        const uint32_t a = desc_mn(c.base + kOffB + 2 * st * kTile), hi = desc_mn(c.base + kOffX + 2 * st * kTile);
        const uint32_t lo = desc_mn(c.base + kOffMore);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
          mma_ss(tm + kColV, a + k * kStepMn, hi + k * kStepMn, kIdU, k > 0);
          if constexpr (LO)
            mma_ss(tm + kColV, a + k * kStepMn, lo + k * kStepMn, kIdU, 1u);
        }
        tc_commit(c.bar(kUFull));
        tc_commit(c.bar(kEmptyBC + st));
        if (!LO || tp.states_only) tc_commit(c.bar(kEmptyX + st));
      }
      __syncwarp();
    }
  }
  return true;
}

// P = G o decay o dt (+ D on the diagonal) of one head, a thread per row.
template <int NH>
__device__ __forceinline__ bool run_p(const Cta& c, int h) {
  const TcParams& tp = c.tp;
  if (tp.states_only) return true;
  const int k = c.warp & 3, lane = c.lane;
  const uint32_t trow = c.tmem + (static_cast<uint32_t>(32 * k) << 16);
  const uint32_t prow = trow + kColP + 64 * h;
  const uint32_t va = c.base + kOffV + h * (96 * 4u);
  // the blocks above the diagonal are zero for good
  {
    uint32_t zero[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) zero[i] = 0u;
#pragma unroll 1
    for (int b = k + 1; b < 4; ++b) tmem_st16(prow + 16 * b, zero);
    rsm::tmem_st_wait();
  }
  Walk walk(tp, false);
  Unit w;
  uint32_t j = 0;
  while (walk.next(w)) {
    const float A2 = __ldg(tp.p.A + w.group * NH + h) * kLog2e;
    const float skip = tp.p.D != nullptr ? __ldg(tp.p.D + w.group * NH + h) : 0.0f;
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u;
      const uint32_t dta = c.base + kOffDt + (st * 2 + h) * (kChunk * 4u);
      if (!c.wait_warp(kFullDt + st, j >> 1)) return false;
      const Scan s = scan_chunk(dta, A2, k, lane);
      // the last P has been multiplied: every warp is done with it and with the v it was made of
      if (j >= 1 && !c.wait_warp(kPxDone + h, j - 1u)) return false;
      if (k < 3) sts(va + static_cast<uint32_t>(32 * k + lane) * 4u, s.dt * exp2_approx(s.after));
      c.arrive_warp(kVSync + h);
      if (!c.wait_warp(kVSync + h, j)) return false;
      if (!c.wait_warp(kGFull, j)) return false;
      tc_fence_after();
      float between = s.upto;  // row i back to the end of block b
#pragma unroll 1
      for (int b = k - 1; b >= 0; --b) {
        float g[32];
        rsm::tmem_ld32(trow + kColG + 32 * b, g);
        const float f = exp2_approx(between);
        between += b == 2 ? s.t[2] : s.t[1];
        uint32_t r[16];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 v = lds4(va + static_cast<uint32_t>(32 * b + 4 * q) * 4u);
          const float2 ff = make_float2(f, f);
          const float2 lo = __fmul2_rn(__fmul2_rn(make_float2(g[4 * q], g[4 * q + 1]), make_float2(v.x, v.y)), ff);
          const float2 hi = __fmul2_rn(__fmul2_rn(make_float2(g[4 * q + 2], g[4 * q + 3]), make_float2(v.z, v.w)), ff);
          r[2 * q] = rsm::pack_bf16x2(lo.x, lo.y);
          r[2 * q + 1] = rsm::pack_bf16x2(hi.x, hi.y);
        }
        tmem_st16(prow + 16 * b, r);
      }
      {
        float g[32];
        rsm::tmem_ld32(trow + kColG + 32 * k, g);
        uint32_t r[16];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 d4 = lds4(dta + static_cast<uint32_t>(32 * k + 4 * q) * 4u);
          const float dd[4] = {d4.x, d4.y, d4.z, d4.w};
          float e[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int jj = 4 * q + m;
            const float pj = __shfl_sync(0xFFFFFFFFu, s.upto, jj);
            const float v = g[jj] * (exp2_approx(s.upto - pj) * dd[m]);
            // the diagonal: no decay, and the skip term
            e[m] = jj < lane ? v : jj == lane ? v + skip : 0.0f;
          }
          r[2 * q] = rsm::pack_bf16x2(e[0], e[1]);
          r[2 * q + 1] = rsm::pack_bf16x2(e[2], e[3]);
        }
        tmem_st16(prow + 16 * k, r);
      }
      rsm::tmem_st_wait();
      tc_fence_before();
      c.arrive_warp(kPFull + h);
      c.arrive_warp(kEmptyDt + st);
    }
  }
  return true;
}

// w X, a thread per token row; hi over x, lo beside it.
template <int NH, bool LO>
__device__ __forceinline__ bool run_w(const Cta& c) {
  const TcParams& tp = c.tp;
  Walk walk(tp, false);
  Unit w;
  uint32_t j = 0;
  const int k = c.warp & 3, lane = c.lane, t = 32 * k + lane;
  const uint32_t row = static_cast<uint32_t>(t) * 128u;
  const uint32_t swz = static_cast<uint32_t>(t & 7) << 4;
  while (walk.next(w)) {
    const float A0 = __ldg(tp.p.A + w.group * NH) * kLog2e, A1 = __ldg(tp.p.A + w.group * NH + NH - 1) * kLog2e;
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u;
      const bool live = c0 + t < w.len;
      if (!c.wait_warp(kFullDt + st, j >> 1)) return false;
      float w0 = 0.0f, w1 = 0.0f;
#pragma unroll 1
      for (int h = 0; h < NH; ++h) {
        const Scan s = scan_chunk(c.base + kOffDt + (st * 2 + h) * (kChunk * 4u), h ? A1 : A0, k, lane);
        float rest = s.after;
#pragma unroll
        for (int b = 1; b < 4; ++b) rest += b > k ? s.t[b] : 0.0f;
        w0 = w1;
        w1 = s.dt * exp2_approx(rest);
      }
      if (NH == 1) w0 = w1;
      c.arrive_warp(kEmptyDt + st);
      if (w.len - c0 < kChunk) {
        if (!c.wait_warp(kFullX + st, j >> 1) || !c.wait_warp(kFullBC + st, j >> 1)) return false;
        if (!live) {
#pragma unroll 1
          for (uint32_t q = 0; q < 8; ++q) {
#pragma unroll
            for (int h = 0; h < NH; ++h) sts128(c.base + kOffX + (2 * st + h) * kTile + row + 16u * q, 0u, 0u, 0u, 0u);
            sts128(c.base + kOffB + (2 * st) * kTile + row + 16u * q, 0u, 0u, 0u, 0u);
            sts128(c.base + kOffB + (2 * st + 1) * kTile + row + 16u * q, 0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
      }
      if (!tp.states_only) c.arrive_warp(kClean);
      if (!c.wait_warp(kFullX + st, j >> 1)) return false;
      if (LO && j >= 1 && !c.wait_warp(kUFull, j - 1u)) return false;  // the lo tiles have been multiplied
#pragma unroll 1
      for (int h = 0; h < NH; ++h) {
        if (!tp.states_only && !c.wait_warp(kPxDone + h, j)) return false;
        const uint32_t xa = c.base + kOffX + (2 * st + h) * kTile + row;
        const uint32_t la = c.base + kOffMore + h * kTile + row;
        const float wt = h ? w1 : w0;
        const float2 w2 = make_float2(wt, wt);
#pragma unroll 1
        for (uint32_t q0 = 0; q0 < 8; q0 += 4) {
          uint4 v[4];
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q) v[q] = rsm::lds128(xa + (((q0 + q) << 4) ^ swz));
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q) {
            const uint32_t at = ((q0 + q) << 4) ^ swz;
            const uint32_t in[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float2 u = __fmul2_rn(make_float2(rsm::bf16lo(in[m]), rsm::bf16hi(in[m])), w2);
              hw[m] = rsm::pack_bf16x2(u.x, u.y);
              if constexpr (LO) {
                // u - hi is exact; rounded to bf16, hi + lo is within 2^-17 of u
                const float2 l = __ffma2_rn(make_float2(rsm::bf16lo(hw[m]), rsm::bf16hi(hw[m])), make_float2(-1.0f, -1.0f), u);
                lw[m] = rsm::pack_bf16x2(l.x, l.y);
              }
              hw[m] = live ? hw[m] : 0u;
              if constexpr (LO) lw[m] = live ? lw[m] : 0u;
            }
            sts128(xa + at, hw[0], hw[1], hw[2], hw[3]);
            if constexpr (LO) sts128(la + at, lw[0], lw[1], lw[2], lw[3]);
          }
        }
      }
      fence_proxy_async_smem();
      c.arrive_warp(kWFull);
    }
  }
  return true;
}

// A dstate column of a slot's head: 64 elements kState apart.
__device__ __forceinline__ void load_column(float (&S)[kDim], const Params& p, int slot, int64_t tile) {
  if (slot < 0) {
#pragma unroll
    for (int d = 0; d < kDim; ++d) S[d] = 0.0f;
    return;
  }
  const int64_t at = slot * p.state_ss + tile;
  if (p.state_dtype == RSM_F32) {
    const float* s = static_cast<const float*>(p.state) + at;
#pragma unroll
    for (int d = 0; d < kDim; ++d) S[d] = s[d * kState];
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(p.state) + at;
    uint16_t raw[kDim];
#pragma unroll
    for (int d = 0; d < kDim; ++d) raw[d] = s[d * kState];
    if (p.state_dtype == RSM_BF16) {
#pragma unroll
      for (int d = 0; d < kDim; ++d) S[d] = __uint_as_float(static_cast<uint32_t>(raw[d]) << 16);
    } else {
#pragma unroll
      for (int d = 0; d < kDim; ++d) S[d] = __half2float(__ushort_as_half(raw[d]));
    }
  }
}
__device__ __forceinline__ void store_column(const float (&S)[kDim], const Params& p, int slot, int64_t tile) {
  const int64_t at = slot * p.state_ss + tile;
  if (p.state_dtype == RSM_F32) {
    float* s = static_cast<float*>(p.state) + at;
#pragma unroll
    for (int d = 0; d < kDim; ++d) s[d * kState] = S[d];
  } else if (p.state_dtype == RSM_BF16) {
    uint16_t* s = static_cast<uint16_t*>(p.state) + at;
#pragma unroll
    for (int d = 0; d < kDim; ++d) s[d * kState] = static_cast<uint16_t>(rsm::pack_bf16x2(S[d], 0.0f));
  } else {
    __half* s = static_cast<__half*>(p.state) + at;
#pragma unroll
    for (int d = 0; d < kDim; ++d) s[d * kState] = __float2half_rn(S[d]);
  }
}

// One head's outputs and state.
template <int NH, bool LO>
__device__ __forceinline__ bool run_head(const Cta& c, int h) {
  const TcParams& tp = c.tp;
  const Params& p = tp.p;
  Walk walk(tp, false);
  Unit w;
  uint32_t j = 0;
  const int k = c.warp & 3, lane = c.lane, r = 32 * k + lane;  // output row, and dstate column
  const uint32_t trow = c.tmem + (static_cast<uint32_t>(32 * k) << 16);
  const uint32_t srow = c.base + (LO ? kOffX : kOffMore) + h * kTile + static_cast<uint32_t>(r) * 128u;
  const uint32_t swz = static_cast<uint32_t>(r & 7) << 4;
  while (walk.next(w)) {
    const int head = w.group * NH + h;
    const float A2 = __ldg(p.A + head) * kLog2e;
    const int64_t tile = static_cast<int64_t>(head) * (kDim * kState) + r;
    float S[kDim];
    const bool say = w.group == 0 && h == 0 && r == 0 && !tp.states_only;
    if (w.split && !tp.states_only) {
      const float* at = tp.seg_state + static_cast<int64_t>(w.seg) * p.H * (kDim * kState) + tile;
#pragma unroll
      for (int d = 0; d < kDim; ++d) S[d] = at[d * kState];
    } else {
      const int src = tp.states_only ? -1 : slot_of(p, p.src, w.seq, say);
      load_column(S, p, src, tile);
    }
    float decay = 0.0f;  // of the segment, log2
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u;
      if (!tp.states_only) {
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q)
          sts128(srow + (LO ? 2 * (st ^ 1u) * kTile : 0u) + ((q << 4) ^ swz), rsm::pack_bf16x2(S[8 * q], S[8 * q + 1]),
                 rsm::pack_bf16x2(S[8 * q + 2], S[8 * q + 3]), rsm::pack_bf16x2(S[8 * q + 4], S[8 * q + 5]),
                 rsm::pack_bf16x2(S[8 * q + 6], S[8 * q + 7]));
        fence_proxy_async_smem();
        tc_fence_before();
        c.arrive_warp(kSFull);
      }
      if (!c.wait_warp(kFullDt + st, j >> 1)) return false;
      const Scan s = scan_chunk(c.base + kOffDt + (st * 2 + h) * (kChunk * 4u), A2, k, lane);
      c.arrive_warp(kEmptyDt + st);
      const float total = (s.t[0] + s.t[1]) + (s.t[2] + s.t[3]);
      decay += total;
      if (!tp.states_only) {
        float up = s.upto;
#pragma unroll
        for (int b = 0; b < 3; ++b) up += b < k ? s.t[b] : 0.0f;
        const float e = exp2_approx(up);
        if (!c.wait_warp(kY1Full, j) || !c.wait_warp(kPxDone + h, j)) return false;
        tc_fence_after();
        unsigned char* out = static_cast<unsigned char*>(p.out) + ((w.t0 + c0 + r) * p.out_ts + head * kDim) * 2;
        const bool live = c0 + r < w.len;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float y1[16], y2[16];
          tmem_ld16x2(trow + kColV + 64 * h + 16 * q, trow + kColY2 + 64 * h + 16 * q, y1, y2);
          uint32_t v[8];
#pragma unroll
          for (int m = 0; m < 8; ++m)
            v[m] = rsm::pack_bf16x2(fmaf(e, y1[2 * m], y2[2 * m]), fmaf(e, y1[2 * m + 1], y2[2 * m + 1]));
          if (live) stg256(out + 32 * q, v);
        }
        tc_fence_before();
        c.arrive_warp(kVRead);
        if (c.lane == 0) mbar_arrive(c.bar(kY2Empty + h));
      }
      if (!c.wait_warp(kUFull, j)) return false;
      tc_fence_after();
      const float a = exp2_approx(total);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float u[32];
        rsm::tmem_ld32(trow + kColV + 64 * h + 32 * q, u);
#pragma unroll
        for (int m = 0; m < 32; ++m) S[32 * q + m] = fmaf(a, S[32 * q + m], u[m]);
      }
      if (tp.states_only) {
        tc_fence_before();
        c.arrive_warp(kVRead);
      }
    }
    if (tp.states_only) {
      float* at = tp.seg_state + static_cast<int64_t>(w.seg) * p.H * (kDim * kState) + tile;
#pragma unroll
      for (int d = 0; d < kDim; ++d) at[d * kState] = S[d];
      if (r == 0) tp.seg_decay[static_cast<int64_t>(w.seg) * p.H + head] = decay;
    } else if (w.last) {
      const int dst = slot_of(p, p.dst, w.seq, say);
      if (dst >= 0) store_column(S, p, dst, tile);
    }
  }
  return true;
}

template <int NH, bool LO>
__global__ void __launch_bounds__(kTcThreads, 1) ssm_tc_kernel(const __grid_constant__ TcParams tp) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = rsm::smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((base & 1023u) != 0u) {  // the swizzled tiles need it (never seen otherwise)
    if (threadIdx.x == 0) flag(tp.p.status, RSM_STATUS_WAIT_TIMEOUT);
    return;
  }
  if (warp == 1) {
    rsm::tmem_alloc(base + kOffTmem, 512u);
    rsm::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    const uint32_t bars = base + kOffBar;
    auto init = [&](uint32_t b, uint32_t n, int how_many = 1) {
      for (int i = 0; i < how_many; ++i) mbar_init(bars + 8u * (b + i), n);
    };
    init(kFullBC, 1, 2);
    init(kEmptyBC, 1, 2);
    init(kFullX, 1, 2);
    init(kEmptyX, 1, 2);
    init(kFullDt, NH, 2);
    init(kEmptyDt, (tp.states_only ? 4 : 4 + 4 * NH) + 4 * NH, 2);
    init(kGFull, 1);
    init(kPFull, 4, 2);
    init(kPxDone, 1, 2);
    init(kY2Empty, 4, 2);
    init(kSFull, 4 * NH);
    init(kY1Full, 1);
    init(kVRead, 4 * NH);
    init(kWFull, 4);
    init(kClean, 4);
    init(kUFull, 1);
    init(kVSync, 4, 2);
    init(kExit, 1);
    *reinterpret_cast<volatile int*>(smem + kOffAbort) = 0;
    rsm::fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Cta c{tp, smem, base, *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem), warp, lane,
              reinterpret_cast<volatile int*>(smem + kOffAbort)};
  // Registers: the launch's 6 x 80 a thread of each warpgroup, shared out anew
  // (56 + 2 x 72 + 56 + 2 x 112 = 480): a head warp holds a column of 64 state values.
  bool ok = true;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      ok = run_loader<NH, LO>(c);
    } else if (warp == 1) {
      ok = run_mma<NH, LO>(c);
      // no MMA may be in flight when the tensor memory is freed, whichever way the role ended
      __syncwarp();
      if (elect_one()) tc_commit(c.bar(kExit));
      __syncwarp();
      (void)rsm::mbar_wait(c.bar(kExit), 0u, kTcTimeoutNs);
    } else if (warp - 2 < NH) {
      ok = run_dt<NH>(c, warp - 2);
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if ((warp - 4) / 4 < NH) ok = run_p<NH>(c, (warp - 4) / 4);
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    ok = run_w<NH, LO>(c);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    if ((warp - 16) / 4 < NH) ok = run_head<NH, LO>(c, (warp - 16) / 4);
  }
  if (!ok) {
    *c.abort_flag = 1;
    flag(tp.p.status, RSM_STATUS_WAIT_TIMEOUT);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) rsm::tmem_dealloc(c.tmem, 512u);
}

// R = the sequence's initial state; for each of its segments: the segment
// starts from R, and R = its decay R + its own state.  One CTA per (sequence,
// head); the same elements belong to the same thread throughout.
__global__ void __launch_bounds__(256) ssm_join_kernel(const __grid_constant__ TcParams tp) {
  const Params& p = tp.p;
  const int seq = static_cast<int>(blockIdx.x / static_cast<uint32_t>(p.H));
  const int h = static_cast<int>(blockIdx.x % static_cast<uint32_t>(p.H));
  auto segs_of = [&](int s) -> uint32_t {
    const int64_t a = __ldg(p.cu_seqlens + s), b = __ldg(p.cu_seqlens + s + 1);
    if (a < 0 || b < a || b > p.tokens) return 0;
    const uint32_t len = static_cast<uint32_t>(b - a);
    return len <= tp.seg ? 1 : (len + tp.seg - 1) / tp.seg;
  };
  const uint32_t n = segs_of(seq);
  if (n <= 1) return;
  int64_t sg = 0;  // segments before the sequence's
  for (int s = 0; s < seq; ++s) sg += segs_of(s);
  const int src = slot_of(p, p.src, seq, false);
  constexpr int kPer = kDim * kState / 256;
  float R[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    R[i] = src >= 0 ? load_state(p.state, src * p.state_ss + static_cast<int64_t>(h) * (kDim * kState) + threadIdx.x + 256 * i,
                                 p.state_dtype)
                    : 0.0f;
  for (uint32_t s = 0; s < n; ++s) {
    float* at = tp.seg_state + ((sg + s) * p.H + h) * (kDim * kState) + threadIdx.x;
    const float a = s + 1 < n ? exp2f(tp.seg_decay[(sg + s) * p.H + h]) : 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float own = s + 1 < n ? at[256 * i] : 0.0f;
      at[256 * i] = R[i];
      R[i] = fmaf(a, R[i], own);
    }
  }
}

}  // namespace ssm
