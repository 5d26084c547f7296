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
// The skip term D x is a D on P's diagonal, rounded to bf16 with it.  P, the state's copy
// and w x are what is rounded on the way: each term of an output once, within 2^-8, as the output
// itself is; what a state sums keeps 16 bits unless it is stored in 8.
//
// Decays.  With p_i the sum of a from the start of i's half of the chunk, a pair
// (i, j) of one half decays by e^{p_i} e^{-p_j}: the column factor goes into P (one
// product an element, no exponential), the row factor onto Y2 when y = m1 Y1 + m2
// Y2 leaves.  A pair across the halves is e^{p_i} e^{rest of the first half}.  Where a half
// decays by more than 2^-32 both factors are taken from its middle, e^{mid - p_j} and e^{p_i -
// mid}: none is beyond 2^50 then, and G, x and their sums have 2^77 left either way.  A half
// that decays by more than 2^-100 ("steep", a mean dt A above 1.08) takes an exponential of p_i -
// p_j an element.  (From the middle always: weights near 1 then round differently from those of
// new tokens, and a prompt differs more from the same tokens in pieces, 1.1e-2 -> 1.35e-2.)  The
// weights towards a chunk's end are summed from there, so that small decays near it
// keep their precision next to large ones before them.
//
// One persistent CTA per SM takes units (sequence, segment, two heads of one group; one
// head where a group has an odd number or SMs would idle), all chunks of a unit in order:
//   warp 0       loads C, B and x (two stages each) with tensor-map copies
//   warp 1       issues the MMAs but G; warps 2, 3 make the decay tables, a head each
//   warps 4-7    P below the diagonal: a thread holds row i, and puts the heads' P where
//                it read G; warp 4 has no such block and issues G
//   warps 8-11   P's blocks on the diagonal
//   warps 12-19  w X, a head each four: a thread holds token t's row; x becomes w x in place
//   warps 20-27  a head each four: the state in registers as fp32, a thread per dstate
//                column, and its bf16 copy for Y1; between the two, y out of Y1 and Y2
// What bounds it is latency, the way round of a chunk: Y2 and Y1 to y and the next Y2 (bf16
// states), and S to Y1 to lo to U to S (others).  Measured on a GB300: a chunk and pair of
// heads takes 2.5 us with bf16 states and 3.0 with fp32 ones (4900 and 5800 cycles), of
// which the four products are 2050 and 2560 cycles; 4 sequences of 8192 tokens in all, 256
// heads, bf16 states: 170 to 180 us, 390 TFLOP/s.
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

// into L2
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* at, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
               "r"(y), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// this thread's stores have read shared memory
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
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

// 8 columns of this thread's lane.  Whole warp.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// 8 columns of this thread's lane from each of two places.  Whole warp.
__device__ __forceinline__ void tmem_ld8x2(uint32_t ta, uint32_t tb, float (&a)[8], float (&b)[8]) {
  uint32_t r[8], s[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(s[0]), "=&r"(s[1]), "=&r"(s[2]), "=&r"(s[3]), "=&r"(s[4]), "=&r"(s[5]), "=&r"(s[6]), "=&r"(s[7])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(s[i]);
  }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSteep = 100.0f;  // decay of a half chunk, log2, past which 2^(mid - p) is not formed
constexpr float kMild = 32.0f;    // ... and up to which mid is 0

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
__device__ __forceinline__ void sts4(uint32_t addr, const float (&v)[4]) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// ---------------------------------------------------------------------------
// the units of this CTA, walked alike by every role
// ---------------------------------------------------------------------------
struct Unit {
  int t0;               // first token
  int len;              // tokens
  int seq, seg, group;  // sequence, segment among all sequences', heads' group
  bool last;            // last segment of the sequence
  bool split;           // its state comes from the segment states
};

// Sequences that are few and not split are taken longest first, so that the last units
// are short: the prompts of a batch differ, and a CTA has few units.  (16 of 8192 tokens
// in all, the longest 2011, 128 heads: 159 us in their own order, 144 us like this.)
__device__ __forceinline__ bool in_order(const TcParams& tp) { return tp.p.units > kSorted || tp.seg_state != nullptr; }
// Where they go back ends the walk: it and those after it come last, it before them.
__device__ __forceinline__ void sort_sequences(const TcParams& tp, uint32_t order, int lane) {  // one warp
  const int n = tp.p.units;
  const int t0 = lane < n ? __ldg(tp.p.cu_seqlens + lane) : 0, t1 = lane < n ? __ldg(tp.p.cu_seqlens + lane + 1) : 0;
  const uint32_t back = __ballot_sync(0xFFFFFFFFu, goes_back(t0, t1));
  const bool before = (back & (2u * (1u << lane) - 1u)) == 0u;  // none at it or before it
  const int len = before ? static_cast<int>(min(static_cast<uint32_t>(t1) - static_cast<uint32_t>(t0), 0x7FFFFFFFu)) : -1;
  uint32_t longer = 0;
  for (int i = 0; i < n; ++i) {
    const int other = __shfl_sync(0xFFFFFFFFu, len, i);
    longer += other > len || (other == len && i < lane) ? 1u : 0u;
  }
  if (lane < n) asm volatile("st.shared.u32 [%0], %1;" ::"r"(order + 4u * longer), "r"(lane) : "memory");
}

// A role's walk: a CTA's units are every gridDim.x-th, to and fro.
struct Walk {
  const TcParams& tp;
  uint32_t order;     // the sequences' order, in shared memory
  uint32_t u;         // next unit
  int at = 0;         // sequence under the cursor, counted in the order taken
  uint32_t base = 0;  // segments before it
  bool flagger;       // the one thread of the CTA that reports

  __device__ Walk(const TcParams& tp_, uint32_t order_, bool flagger_) : tp(tp_), order(order_), u(blockIdx.x), flagger(flagger_) {}

  // Little is kept from unit to unit: a role's registers are few.
  __device__ bool next(Unit& w) {
    for (;; ++at) {
      if (at >= tp.p.units) return false;
      int seq = at;
      if (!in_order(tp)) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(seq) : "r"(order + 4u * at));
      const int t0 = __ldg(tp.p.cu_seqlens + seq), t1 = __ldg(tp.p.cu_seqlens + seq + 1);
      if (!within(t0, t1, tp.p.tokens)) {
        if (flagger) flag(tp.p.status, RSM_STATUS_BAD_SEQUENCE);
        if (goes_back(t0, t1)) return false;  // nor any after it
        continue;                             // no unit at all
      }
      const uint32_t len = static_cast<uint32_t>(t1 - t0);
      const uint32_t nseg = segments_of(len, tp.seg);
      for (uint32_t sg; (sg = u / static_cast<uint32_t>(tp.pairs)) < base + nseg;) {
        const uint32_t s = sg - base;
        w.group = static_cast<int>(u - sg * static_cast<uint32_t>(tp.pairs));
        const uint32_t round = u / gridDim.x + 1;
        u = round * gridDim.x + (round & 1u ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        w.last = s == nseg - 1;
        w.split = nseg > 1;
        if (tp.states_only && w.last) continue;  // nothing follows its state
        w.seq = seq;
        w.seg = static_cast<int>(sg);
        w.t0 = t0 + static_cast<int>(s * tp.seg);
        w.len = static_cast<int>(min(tp.seg, len - s * tp.seg));
        return true;
      }
      base += nseg;
    }
  }
};

// ---------------------------------------------------------------------------
// A few instructions, since every role's code shares the instruction cache.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, %3;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra AGAIN;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "n"(kTcTries)
      : "memory");
  return ok != 0;
}

struct Cta {
  const TcParams& tp;
  unsigned char* smem;
  uint32_t base;
  uint32_t tmem;
  int warp, lane;

  __device__ uint32_t bar(uint32_t b) const { return base + kOffBar + 8u * b; }
  __device__ uint32_t table(uint32_t stage, int h) const { return base + kOffTab + (2 * stage + h) * kTabBytes; }
  // The phase of `parity` of a barrier has completed; false when the tries ran out.
  __device__ __forceinline__ bool wait(uint32_t b, uint32_t parity) const { return wait_bounded(bar(b), parity & 1u); }
  __device__ bool wait_warp(uint32_t b, uint32_t parity) const {
    return __all_sync(0xFFFFFFFFu, wait(b, parity)) != 0;
  }
  __device__ void arrive_warp(uint32_t b) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  }
};

template <int NH>
__device__ __forceinline__ bool run_loader(const Cta& c) {
  const TcParams& tp = c.tp;
  Walk walk(tp, c.base + kOffOrder, c.lane == 0);
  Unit w;
  uint32_t j = 0, n_bc = 0, n_x = 0;  // chunk; copies issued so far
  const uint32_t per_group = static_cast<uint32_t>(tp.p.H / tp.p.G);
  const bool one = elect_one();
  bool ok = true;
  while (ok && walk.next(w)) {
    const int h0 = w.group * NH, g = static_cast<int>(static_cast<uint32_t>(h0) / per_group);
    if (one && !tp.states_only && !w.split) {  // the state it starts from is wanted in a chunk or two
      const int src = slot_of(tp.p, tp.p.src, w.seq, false);
      if (src >= 0) {
        const uint32_t size = tp.p.state_dtype == RSM_F32 ? 4u : 2u;
        const char* at = static_cast<const char*>(tp.p.state) +
                         (src * tp.p.state_ss + static_cast<int64_t>(h0) * (kDim * kState)) * static_cast<int64_t>(size);
        if (reinterpret_cast<uintptr_t>(at) % 16 == 0) prefetch_l2(at, NH * kDim * kState * size);
      }
    }
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u;
      const int row = w.t0 + c0;
      if (one) {  // the stages are taken yet, but x can come nearer
        for (int h = 0; h < NH; ++h) tma_prefetch_2d(&tp.x_map, (h0 + h) * kDim, row);
      }
      const uint32_t bc = c.bar(kFullBC + st);
      if (!tp.states_only) {  // C's place is free before B's, but for lo, which is there until the update
        if (j >= 2 && !(ok = c.wait_warp(kEmptyC + st, (j >> 1) - 1u))) break;
        if (one) {
          mbar_expect(bc, 2 * kTile);
#pragma unroll
          for (int half = 0; half < 2; ++half)
            tma_load_2d(c.base + kOffC + (2 * st + half) * kTile, &tp.C_map, g * kState + 64 * half, row, bc);
        }
      }
      if (j >= 2 && !(ok = c.wait_warp(kEmptyB + st, (j >> 1) - 1u))) {
        if (!tp.states_only) {  // C is on its way, and to be waited for
          if (one) mbar_arrive(bc);
          ++n_bc;
        }
        break;
      }
      if (one) {
        mbar_arrive_expect(bc, 2 * kTile);
#pragma unroll
        for (int half = 0; half < 2; ++half)
          tma_load_2d(c.base + kOffB + (2 * st + half) * kTile, &tp.B_map, g * kState + 64 * half, row, bc);
      }
      ++n_bc;
      // the stage is free once the last chunk's Y1 has read the state that took it
      // (without a Y1: after the update two chunks ago)
      if (tp.states_only ? j >= 2 : j >= 1)
        if (!(ok = c.wait_warp(kEmptyX + st, tp.states_only ? (j >> 1) - 1u : (j - 1u) >> 1))) break;
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
    (void)c.wait(kFullBC + (k & 1u), k >> 1);
  for (uint32_t k = n_x >= 2 ? n_x - 2 : 0; k < n_x; ++k)
    (void)c.wait(kFullX + (k & 1u), k >> 1);
  return ok;
}

// The decay tables of a head's chunks; a lane has four tokens in a row, half a warp a half chunk.
template <int NH>
__device__ __forceinline__ bool run_tables(const Cta& c, int h) {
  const TcParams& tp = c.tp;
  Walk walk(tp, c.base + kOffOrder, false);
  Unit w;
  uint32_t j = 0;
  const int lane = c.lane;
  const bool second = lane >= 16;
  while (walk.next(w)) {
    const int head = w.group * NH + h;
    const float* dt = tp.p.dt + static_cast<int64_t>(w.t0) * tp.p.dt_ts + head;
    const float A2 = __ldg(tp.p.A + head) * kLog2e;
    const float skip = tp.p.D != nullptr ? __ldg(tp.p.D + head) : 0.0f;
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      float d[4], upto[4], after[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int i = c0 + 4 * lane + m;
        d[m] = i < w.len ? __ldg(dt + static_cast<int64_t>(i) * tp.p.dt_ts) : 0.0f;
      }
      // sums over the lane's tokens, then over the half's lanes from either end
      upto[0] = d[0] * A2;
#pragma unroll
      for (int m = 1; m < 4; ++m) upto[m] = fmaf(d[m], A2, upto[m - 1]);
      after[3] = 0.0f;
#pragma unroll
      for (int m = 2; m >= 0; --m) after[m] = fmaf(d[m + 1], A2, after[m + 1]);
      float before = upto[3], beyond = upto[3];
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        const float x = __shfl_up_sync(0xFFFFFFFFu, before, o, 16);
        const float y = __shfl_down_sync(0xFFFFFFFFu, beyond, o, 16);
        if ((lane & 15) >= o) before += x;
        if ((lane & 15) + o < 16) beyond += y;
      }
      const float half0 = __shfl_sync(0xFFFFFFFFu, before, 15), half1 = __shfl_sync(0xFFFFFFFFu, before, 31);
      const float bx = __shfl_up_sync(0xFFFFFFFFu, before, 1, 16), by = __shfl_down_sync(0xFFFFFFFFu, beyond, 1, 16);
      before = (lane & 15) == 0 ? 0.0f : bx;
      beyond = (lane & 15) == 15 ? 0.0f : by;
      const bool steep = !(fabsf(second ? half1 : half0) <= kSteep);
      const float mid = steep || fabsf(second ? half1 : half0) <= kMild ? 0.0f : 0.5f * (second ? half1 : half0);
      const float mid1 = __shfl_sync(0xFFFFFFFFu, mid, 31);
      const float start = second ? half0 + mid : mid, rest1 = second ? 0.0f : half1;
      before -= mid;
      const uint32_t st = j & 1u;
      if (j >= 2 && !c.wait_warp(kEmptyTab + st, (j >> 1) - 1u)) return false;
      const uint32_t at = c.table(st, h) + 16u * lane;
      float col[4], v[4], ww[4], m1[4], m2[4], sk[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float p = before + upto[m], rest = after[m] + beyond;  // (p less mid)
        const float inv = exp2_approx(-p);
        col[m] = steep ? p : d[m] * inv;
        v[m] = d[m] * exp2_approx(rest + mid1);
        ww[m] = d[m] * exp2_approx(rest + rest1);
        m1[m] = exp2_approx(start + p);
        m2[m] = steep ? 1.0f : exp2_approx(p);
        sk[m] = steep ? skip : skip * inv;
      }
      sts4(at + kTabCol, col);
      sts4(at + kTabDt, d);
      if (!second) sts4(at + kTabV, v);
      sts4(at + kTabW, ww);
      sts4(at + kTabM1, m1);
      sts4(at + kTabM2, m2);
      sts4(at + kTabSkip, sk);
      const float flagged = steep ? 1.0f : 0.0f;
      const float steep0 = __shfl_sync(0xFFFFFFFFu, flagged, 0), steep1 = __shfl_sync(0xFFFFFFFFu, flagged, 31);
      if (lane == 0) {
        const float misc[4] = {exp2_approx(half0 + half1), half0 + half1, steep0, steep1};
        sts4(at + kTabMisc, misc);
      }
      c.arrive_warp(kFullTab + st);
    }
  }
  return true;
}

// The whole warp walks and waits, so that addresses stay uniform; one thread issues.
template <int NH, bool LO>
__device__ __forceinline__ bool run_mma(const Cta& c) {
  const TcParams& tp = c.tp;
  Walk walk(tp, c.base + kOffOrder, false);
  Unit w;
  uint32_t j = 0;
  constexpr uint32_t kIdY1 = rsm::idesc_bf16_f32(128, 64 * NH, false, true);
  constexpr uint32_t kIdPx = rsm::idesc_bf16_f32(128, 64, false, true);
  constexpr uint32_t kIdU = rsm::idesc_bf16_f32(128, 64 * NH, true, true);
  constexpr uint32_t kStepMn = 2048 / 16;  // 16 rows of K
  const uint32_t tm = c.tmem;
  const bool one = elect_one();

  while (walk.next(w)) {
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u;
      if (!tp.states_only) {
        // Y2 = P X (x has come, or W would not have looked at it)
        if (!c.wait_warp(kClean, j) || !c.wait_warp(kPFull + st, j >> 1)) return false;
        if (j >= 1 && !c.wait_warp(kYRead, j - 1u)) return false;
        tc_fence_after();
        if (one) {
          const uint32_t P = tm + kColG + 128 * st;
#pragma unroll 1
          for (uint32_t h = 0; h < NH; ++h) {
            const uint32_t b = desc_mn(c.base + kOffX + (2 * st + h) * kTile);
#pragma unroll 4
            for (uint32_t k = 0; k < 8; ++k)  // 16 tokens each, two to a block
              mma_ts(tm + kColY2 + 64 * h, P + 32 * (k >> 1) + 16 * h + 8 * (k & 1), b + k * kStepMn, kIdPx, k > 0);
          }
          tc_commit(c.bar(kPxDone));
        }
        __syncwarp();
        // Y1 = C S^T
        if (!c.wait_warp(kSFull, j)) return false;
        tc_fence_after();
        if (one) {
          const uint32_t a = desc_k(c.base + kOffC + 2 * st * kTile);
          const uint32_t b = desc_mn(c.base + kOffX + 2 * (st ^ 1u) * kTile);
#pragma unroll 4
          for (uint32_t k = 0; k < 8; ++k)
            mma_ss(tm + kColY1, a + (k >> 2) * (kTile / 16) + (k & 3) * 2, b + k * kStepMn, kIdY1, k > 0);
          tc_commit(c.bar(kY1Full));
          if constexpr (!LO) tc_commit(c.bar(kEmptyC + st));
          tc_commit(c.bar(kEmptyX + (st ^ 1u)));
        }
        __syncwarp();
      } else if (!c.wait_warp(kFullBC + st, j >> 1)) {
        return false;
      }
      // U = B^T (w X); P, where it goes, has been multiplied
      if (!c.wait_warp(kWFull + st, j >> 1)) return false;
      if (tp.states_only && j >= 2 && !c.wait_warp(kURead + st, (j >> 1) - 1u)) return false;
      tc_fence_after();
      const uint32_t ua = desc_mn(c.base + kOffB + 2 * st * kTile);
      if (one) {
        const uint32_t hi = desc_mn(c.base + kOffX + 2 * st * kTile);
#pragma unroll 4
        for (uint32_t k = 0; k < 8; ++k) mma_ss(tm + kColG + 128 * st, ua + k * kStepMn, hi + k * kStepMn, kIdU, k > 0);
      }
      __syncwarp();
      if constexpr (LO) {
        if (!c.wait_warp(kLoFull + st, j >> 1)) return false;
        tc_fence_after();
        if (one) {
          const uint32_t lo = desc_mn(c.base + kOffC + 2 * st * kTile);
#pragma unroll 4
          for (uint32_t k = 0; k < 8; ++k) mma_ss(tm + kColG + 128 * st, ua + k * kStepMn, lo + k * kStepMn, kIdU, 1u);
        }
      }
      if (one) {
        tc_commit(c.bar(kUFull + st));
        tc_commit(c.bar(kEmptyB + st));
        if constexpr (LO) tc_commit(c.bar(kEmptyC + st));
        if (tp.states_only) tc_commit(c.bar(kEmptyX + st));
      }
      __syncwarp();
    }
  }
  return true;
}

// G = C B^T of a stage.  One thread.
__device__ __forceinline__ void issue_G(const Cta& c, uint32_t st) {
  constexpr uint32_t kIdG = rsm::idesc_bf16_f32(128, 128, false, false);
  const uint32_t a = desc_k(c.base + kOffC + 2 * st * kTile), b = desc_k(c.base + kOffB + 2 * st * kTile);
#pragma unroll 4
  for (uint32_t k = 0; k < 8; ++k) {  // 16 dstate columns each: 32 bytes, four to a 64-column tile
    const uint32_t o = (k >> 2) * (kTile / 16) + (k & 3) * 2;
    mma_ss(c.tmem + kColG + 128 * st, a + o, b + o, kIdG, k > 0);
  }
  tc_commit(c.bar(kGFull + st));
}

// 32 columns of a row by their factors.
__device__ __forceinline__ void scale_block(const float (&g)[32], uint32_t col, uint32_t (&r)[16]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 v = lds4(col + 16u * q);
    const float2 lo = __fmul2_rn(make_float2(g[4 * q], g[4 * q + 1]), make_float2(v.x, v.y));
    const float2 hi = __fmul2_rn(make_float2(g[4 * q + 2], g[4 * q + 3]), make_float2(v.z, v.w));
    r[2 * q] = rsm::pack_bf16x2(lo.x, lo.y);
    r[2 * q + 1] = rsm::pack_bf16x2(hi.x, hi.y);
  }
}

// A row's blocks (the one on the diagonal, or those below it) where a head's decay is
// steep; the other head may be as usual.
template <int NH, bool DIAG>
__device__ __forceinline__ void steep_rows(uint32_t tab0, uint32_t trow, int k, int lane) {
#pragma unroll 1
  for (int b = DIAG ? k : 0; b < (DIAG ? k + 1 : k); ++b) {
    float g[32];
    rsm::tmem_ld32(trow + 32 * b, g);
    const bool same = (b >> 1) == (k >> 1);
#pragma unroll 1
    for (int h = 0; h < NH; ++h) {
      const uint32_t tab = tab0 + h * kTabBytes;
      const bool steep = lds(tab + kTabMisc + 8u + 4u * (k >> 1)) != 0.0f;
      const float pi = lds(tab + kTabCol + 4u * (32 * k + lane)), skip = lds(tab + kTabSkip + 4u * (32 * k + lane));
      const float ui = steep ? exp2_approx(pi) : 1.0f;
      uint32_t r[16];
#pragma unroll
      for (int q = 0; q < 32; q += 2) {
        float e[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint32_t o = 128u * b + 4u * (q + m);
          const bool in = !DIAG || q + m <= lane;
          float f;
          if (!same)
            f = ui * lds(tab + kTabV + o);
          else if (steep)
            f = exp2_approx(pi - lds(tab + kTabCol + o)) * lds(tab + kTabDt + o);
          else
            f = lds(tab + kTabCol + o);
          const float y = fmaf(g[q + m], f, DIAG && q + m == lane ? skip : 0.0f);
          e[m] = in ? y : 0.0f;
        }
        r[q / 2] = rsm::pack_bf16x2(e[0], e[1]);
      }
      tmem_st16(trow + 32 * b + 16 * h, r);
    }
  }
}

// P of the heads, a thread per row; the row factor 2^(p - mid) is left to the output.  A row's
// warp has one block of 32 columns on the diagonal, which is one warpgroup's work
// (DIAG), and 0 to 3 below it, which with zeros above are the other's.  The warp with
// zeros alone has the time to issue G.
template <int NH, bool DIAG>
__device__ __forceinline__ bool run_p(const Cta& c) {
  const TcParams& tp = c.tp;
  if (tp.states_only) return true;
  const int k = c.warp & 3, lane = c.lane;
  const uint32_t trow0 = c.tmem + (static_cast<uint32_t>(32 * k) << 16) + kColG;
  const bool issuer = !DIAG && k == 0, one = elect_one();
  Walk walk(tp, c.base + kOffOrder, false);
  Unit w;
  uint32_t j = 0;
  while (walk.next(w)) {
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u, tab0 = c.table(st, 0), trow = trow0 + 128 * st;
      if (issuer) {
        if (j >= 2 && !c.wait_warp(kURead + st, (j >> 1) - 1u)) return false;
        if (!c.wait_warp(kFullBC + st, j >> 1)) return false;
        tc_fence_after();
        if (one) issue_G(c, st);
        __syncwarp();
      }
      if (!c.wait_warp(kFullTab + st, j >> 1) || !c.wait_warp(kGFull + st, j >> 1)) return false;
      tc_fence_after();
      // whether the rows' half is steep for either head
      const bool steep = lds(tab0 + kTabMisc + 8u + 4u * (k >> 1)) + lds(c.table(st, NH - 1) + kTabMisc + 8u + 4u * (k >> 1)) != 0.0f;
      if (steep) {
        steep_rows<NH, DIAG>(tab0, trow, k, lane);
      } else if constexpr (DIAG) {
        float g[32], gd = 0.0f;
        rsm::tmem_ld32(trow + 32 * k, g);
#pragma unroll
        for (int i = 0; i < 32; ++i) {  // once for the heads: what is below the diagonal, and what is on it
          gd = i == lane ? g[i] : gd;
          g[i] = i < lane ? g[i] : 0.0f;
        }
#pragma unroll 1
        for (int h = 0; h < NH; ++h) {
          const uint32_t tab = tab0 + h * kTabBytes;
          uint32_t r[16];
          scale_block(g, tab + kTabCol + 128u * k, r);
          const float on = fmaf(gd, lds(tab + kTabCol + 4u * (32 * k + lane)), lds(tab + kTabSkip + 4u * (32 * k + lane)));
          const uint32_t bits = rsm::pack_bf16x2(lane & 1 ? 0.0f : on, lane & 1 ? on : 0.0f);
#pragma unroll
          for (int q = 0; q < 16; ++q) r[q] |= lane >> 1 == q ? bits : 0u;
          tmem_st16(trow + 32 * k + 16 * h, r);
        }
      } else {
#pragma unroll 1
        for (int b = 0; b < k; ++b) {
          float g[32];
          rsm::tmem_ld32(trow + 32 * b, g);
#pragma unroll 1
          for (int h = 0; h < NH; ++h) {
            uint32_t r[16];
            scale_block(g, tab0 + h * kTabBytes + (k >= 2 && b < 2 ? kTabV : kTabCol) + 128u * b, r);
            tmem_st16(trow + 32 * b + 16 * h, r);
          }
        }
      }
      if constexpr (!DIAG) {
        uint32_t zero[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) zero[i] = 0u;
#pragma unroll 1
        for (int b = k + 1; b < 4; ++b) {
          tmem_st16(trow + 32 * b, zero);
          if (NH == 2) tmem_st16(trow + 32 * b + 16, zero);
        }
      }
      rsm::tmem_st_wait();
      tc_fence_before();
      c.arrive_warp(kPFull + st);
      if (lane == 0) mbar_arrive(c.bar(kEmptyTab + st));
    }
  }
  return true;
}

// w X of a head, a thread per token row; hi over x, lo in C's place.
template <int NH, bool LO>
__device__ __forceinline__ bool run_w(const Cta& c, int h) {
  const TcParams& tp = c.tp;
  Walk walk(tp, c.base + kOffOrder, false);
  Unit w;
  uint32_t j = 0;
  const int k = c.warp & 3, lane = c.lane, t = 32 * k + lane;
  const uint32_t row = static_cast<uint32_t>(t) * 128u;
  const uint32_t swz = static_cast<uint32_t>(t & 7) << 4;
  while (walk.next(w)) {
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u;
      if (!c.wait_warp(kFullTab + st, j >> 1)) return false;
      const float wt = lds(c.table(st, h) + kTabW + 4u * t);
      c.arrive_warp(kEmptyTab + st);
      if (!c.wait_warp(kFullX + st, j >> 1)) return false;
      const uint32_t xa = c.base + kOffX + (2 * st + h) * kTile + row;
      const uint32_t la = c.base + kOffC + (2 * st + h) * kTile + row;
      if (w.len - c0 < kChunk) {  // rows past the end: zero, whatever is there
        if (!c.wait_warp(kFullBC + st, j >> 1)) return false;
        if (c0 + t >= w.len) {
#pragma unroll 1
          for (uint32_t q = 0; q < 8; ++q) {
            sts128(xa + 16u * q, 0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = h; i < 2; i += NH) sts128(c.base + kOffB + (2 * st + i) * kTile + row + 16u * q, 0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
      }
      if (!tp.states_only) c.arrive_warp(kClean);
      if (!tp.states_only && !c.wait_warp(kPxDone, j)) return false;
      const float2 w2 = make_float2(wt, wt);
      uint32_t lw[LO ? 32 : 1];
#pragma unroll(LO ? 8 : 2)
      for (uint32_t q = 0; q < 8; ++q) {
        const uint32_t at = (xa + swz) ^ (q << 4);  // a row is 128 bytes
        const uint4 v = rsm::lds128(at);
        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
        uint32_t hw[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 u = __fmul2_rn(make_float2(rsm::bf16lo(in[m]), rsm::bf16hi(in[m])), w2);
          hw[m] = rsm::pack_bf16x2(u.x, u.y);
          if constexpr (LO) {
            // u - hi is exact; rounded to bf16, hi + lo is within 2^-17 of u
            const float2 l = __ffma2_rn(make_float2(rsm::bf16lo(hw[m]), rsm::bf16hi(hw[m])), make_float2(-1.0f, -1.0f), u);
            lw[4 * q + m] = bounded_lo(rsm::pack_bf16x2(l.x, l.y));
          }
        }
        if constexpr (LO)  // here and now: two registers a pair until then are too many
          asm volatile("" : "+r"(lw[4 * q]), "+r"(lw[4 * q + 1]), "+r"(lw[4 * q + 2]), "+r"(lw[4 * q + 3]));
        sts128(at, hw[0], hw[1], hw[2], hw[3]);
      }
      fence_proxy_async_smem();
      c.arrive_warp(kWFull + st);
      if constexpr (LO) {
        if (!tp.states_only && !c.wait_warp(kY1Full, j)) return false;  // the last to read C
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q)
          sts128((la + swz) ^ (q << 4), lw[4 * q], lw[4 * q + 1], lw[4 * q + 2], lw[4 * q + 3]);
        fence_proxy_async_smem();
        c.arrive_warp(kLoFull + st);
      }
    }
  }
  return true;
}

// A dstate column of a slot's head: 64 elements kState apart.
__device__ __forceinline__ void load_column(float2 (&S)[kDim / 2], const Params& p, int slot, int64_t tile) {
  if (slot < 0) {
#pragma unroll
    for (int d = 0; d < kDim / 2; ++d) S[d] = make_float2(0.0f, 0.0f);
    return;
  }
  const int64_t at = slot * p.state_ss + tile;
  if (p.state_dtype == RSM_F32) {
    const float* s = static_cast<const float*>(p.state) + at;
#pragma unroll
    for (int d = 0; d < kDim / 2; ++d) S[d] = make_float2(s[2 * d * kState], s[(2 * d + 1) * kState]);
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(p.state) + at;
    uint16_t raw[kDim];
#pragma unroll
    for (int d = 0; d < kDim; ++d) raw[d] = s[d * kState];
    const bool bf = p.state_dtype == RSM_BF16;
#pragma unroll
    for (int d = 0; d < kDim; ++d) {
      const float v = bf ? __uint_as_float(static_cast<uint32_t>(raw[d]) << 16) : __half2float(__ushort_as_half(raw[d]));
      if (d & 1)
        S[d / 2].y = v;
      else
        S[d / 2].x = v;
    }
  }
}
__device__ __forceinline__ void store_column(const float2 (&S)[kDim / 2], const Params& p, int slot, int64_t tile) {
  const int64_t at = slot * p.state_ss + tile;
  if (p.state_dtype == RSM_F32) {
    float* s = static_cast<float*>(p.state) + at;
#pragma unroll
    for (int d = 0; d < kDim; ++d) s[d * kState] = d & 1 ? S[d / 2].y : S[d / 2].x;
  } else {
    uint16_t* s = static_cast<uint16_t*>(p.state) + at;
    const bool bf = p.state_dtype == RSM_BF16;
#pragma unroll
    for (int d = 0; d < kDim / 2; ++d) {
      const uint32_t v = bf ? rsm::pack_bf16x2(S[d].x, S[d].y) : rsm::pack_f16x2(S[d].x, S[d].y);
      s[2 * d * kState] = static_cast<uint16_t>(v);
      s[(2 * d + 1) * kState] = static_cast<uint16_t>(v >> 16);
    }
  }
}

// One head's state, a thread per dstate column, and between its two uses the head's
// outputs, a thread per row.
template <int NH>
__device__ __forceinline__ bool run_state(const Cta& c, int h) {
  const TcParams& tp = c.tp;
  const Params& p = tp.p;
  Walk walk(tp, c.base + kOffOrder, false);
  Unit w;
  uint32_t j = 0;
  const int k = c.warp & 3, lane = c.lane, r = 32 * k + lane;
  const uint32_t lanes = c.tmem + (static_cast<uint32_t>(32 * k) << 16) + 64 * h;
  const uint32_t srow = c.base + kOffX + h * kTile + static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>(r & 7) << 4);
  // A warp's rows leave 32 columns at a time, by a tensor-map store from shared
  // memory: rows stored by their threads take its pipe 32 lines an instruction.
  // 16-byte pieces of a row change places by its number / 2.
  const uint32_t ywarp = c.base + kOffY + (4 * h + k) * kYBytes;
  const uint32_t yput = ywarp + 64u * lane + (static_cast<uint32_t>((lane >> 1) & 3) << 4);
  while (walk.next(w)) {
    const int64_t tile = (static_cast<int64_t>(w.group) * NH + h) * (kDim * kState) + r;
    float2 S[kDim / 2];
    const bool say = w.group == 0 && h == 0 && r == 0 && !tp.states_only;
    if (w.split && !tp.states_only) {
      const float* at = tp.seg_state + static_cast<int64_t>(w.seg) * p.H * (kDim * kState) + tile;
#pragma unroll
      for (int d = 0; d < kDim / 2; ++d) S[d] = make_float2(at[2 * d * kState], at[(2 * d + 1) * kState]);
    } else {
      load_column(S, p, tp.states_only ? -1 : slot_of(p, p.src, w.seq, say), tile);
    }
    float decay = 0.0f;  // of the segment, log2
    const int col = (w.group * NH + h) * kDim;
#pragma unroll 1
    for (int c0 = 0; c0 < w.len; c0 += kChunk, ++j) {
      const uint32_t st = j & 1u, tab = c.table(st, h);
      if (!tp.states_only) {
        const uint32_t at = srow + 2 * (st ^ 1u) * kTile;
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q)
          sts128(at ^ (q << 4), rsm::pack_bf16x2(S[4 * q].x, S[4 * q].y), rsm::pack_bf16x2(S[4 * q + 1].x, S[4 * q + 1].y),
                 rsm::pack_bf16x2(S[4 * q + 2].x, S[4 * q + 2].y), rsm::pack_bf16x2(S[4 * q + 3].x, S[4 * q + 3].y));
        fence_proxy_async_smem();
        c.arrive_warp(kSFull);
      }
      if (!c.wait_warp(kFullTab + st, j >> 1)) return false;
      const float a = lds(tab + kTabMisc), m1 = lds(tab + kTabM1 + 4u * r), m2 = lds(tab + kTabM2 + 4u * r);
      decay += lds(tab + kTabMisc + 4u);
      c.arrive_warp(kEmptyTab + st);
      if (!tp.states_only) {
        const float2 f1 = make_float2(m1, m1), f2 = make_float2(m2, m2);
        if (!c.wait_warp(kPxDone, j) || !c.wait_warp(kY1Full, j)) return false;
        tc_fence_after();
        const int rows = w.len - c0 - 32 * k;  // of this warp's that exist
#pragma unroll 1
        for (uint32_t part = 0; part < 2; ++part) {
          if (lane == 0) tma_store_wait_read();  // the last store from here
          __syncwarp();
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q) {
            float y1[8], y2[8];
            tmem_ld8x2(lanes + kColY1 + 32 * part + 8 * q, lanes + kColY2 + 32 * part + 8 * q, y1, y2);
            uint32_t v[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float2 y = __ffma2_rn(f1, make_float2(y1[2 * m], y1[2 * m + 1]), __fmul2_rn(f2, make_float2(y2[2 * m], y2[2 * m + 1])));
              v[m] = rsm::pack_bf16x2(y.x, y.y);
            }
            sts128(yput ^ (16u * q), v[0], v[1], v[2], v[3]);
          }
          if (part == 1) {
            tc_fence_before();
            c.arrive_warp(kYRead);
          }
          if (rows >= 32) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tma_store_2d(&tp.y_map, col + 32 * part, w.t0 + c0 + 32 * k, ywarp);
          } else if (lane < rows) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + static_cast<int64_t>(w.t0 + c0 + r) * p.out_ts + col + 32 * part);
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) out[q] = rsm::lds128(yput ^ (16u * q));
          }
        }
      }
      if (!c.wait_warp(kUFull + st, j >> 1)) return false;
      tc_fence_after();
      const float2 a2 = make_float2(a, a);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float u[16];
        rsm::tmem_ld16(lanes + kColG + 128 * st + 16 * q, u);
#pragma unroll
        for (int m = 0; m < 8; ++m) S[8 * q + m] = __ffma2_rn(a2, S[8 * q + m], make_float2(u[2 * m], u[2 * m + 1]));
      }
      tc_fence_before();
      c.arrive_warp(kURead + st);
    }
    if (tp.states_only) {
      float* at = tp.seg_state + static_cast<int64_t>(w.seg) * p.H * (kDim * kState) + tile;
#pragma unroll
      for (int d = 0; d < kDim / 2; ++d) {
        at[2 * d * kState] = S[d].x;
        at[(2 * d + 1) * kState] = S[d].y;
      }
      if (r == 0) tp.seg_decay[static_cast<int64_t>(w.seg) * p.H + w.group * NH + h] = decay;
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
  if (warp == 2 && !in_order(tp)) sort_sequences(tp, base + kOffOrder, lane);
  if (threadIdx.x == 0) {
    const uint32_t bars = base + kOffBar;
    auto init = [&](uint32_t b, uint32_t n, int how_many = 1) {
      for (int i = 0; i < how_many; ++i) mbar_init(bars + 8u * (b + i), n);
    };
    init(kFullBC, 1, 2);
    init(kEmptyB, 1, 2);
    init(kEmptyC, 1, 2);
    init(kFullX, 1, 2);
    init(kEmptyX, 1, 2);
    init(kFullTab, NH, 2);
    init(kEmptyTab, 8 * NH + (tp.states_only ? 0 : 8), 2);  // W and S; P
    init(kGFull, 1, 2);
    init(kPFull, 8, 2);
    init(kPxDone, 1);
    init(kSFull, 4 * NH);
    init(kY1Full, 1);
    init(kYRead, 4 * NH);
    init(kWFull, 4 * NH, 2);
    init(kLoFull, 4 * NH, 2);
    init(kClean, 4 * NH);
    init(kUFull, 1, 2);
    init(kURead, 4 * NH, 2);
    init(kExit, 1, 2);
    rsm::fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Cta c{tp, smem, base, *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem), warp, lane};
  // Registers: the launch's 7 x 72 a thread of each warpgroup, shared out anew (40 + 2 x
  // 72 + 2 x 56 + 2 x 104 = 504; without lo w X needs 48 and the states have 112): P has to
  // fit (64 a thread: 92 -> 98 us, 304 heads of 4096 tokens), a state warp holds columns of 64 values.
  bool ok = true;
  // no MMA may be in flight when the tensor memory is freed, whichever way its issuer ended
  auto drain = [&](uint32_t bar) {
    __syncwarp();
    if (elect_one()) tc_commit(c.bar(bar));
    __syncwarp();
    (void)c.wait(bar, 0u);
  };
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      ok = run_loader<NH>(c);
    } else if (warp == 1) {
      ok = run_mma<NH, LO>(c);
      drain(kExit);
    } else if (warp - 2 < NH) {
      ok = run_tables<NH>(c, warp - 2);
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    ok = warp < 8 ? run_p<NH, false>(c) : run_p<NH, true>(c);
    if (warp == 4) drain(kExit + 1);
  } else if (warp < 20) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LO ? 56 : 48));
    if ((warp - 12) / 4 < NH) ok = run_w<NH, LO>(c, (warp - 12) / 4);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LO ? 104 : 112));
    if ((warp - 20) / 4 < NH) {
      ok = run_state<NH>(c, (warp - 20) / 4);
      if (lane == 0) tma_store_wait_read();  // shared memory outlives the stores that read it
    }
  }
  if (!ok) flag(tp.p.status, RSM_STATUS_WAIT_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) rsm::tmem_dealloc(c.tmem, 512u);
}

// R = the sequence's initial state; for each of its segments: the segment
// starts from R, and R = its decay R + its own state.  One CTA per (sequence,
// head, part of the state); a thread keeps four elements throughout and asks for
// eight segments' at a time, which no store of its own comes before.
__global__ void __launch_bounds__(kJoinThreads) ssm_join_kernel(const __grid_constant__ TcParams tp) {
  const Params& p = tp.p;
  constexpr uint32_t kParts = kDim * kState / (4 * kJoinThreads);
  const uint32_t part = blockIdx.x % kParts, unit = blockIdx.x / kParts;
  const int seq = static_cast<int>(unit / static_cast<uint32_t>(p.H));
  const int h = static_cast<int>(unit % static_cast<uint32_t>(p.H));
  int64_t sg = 0;  // segments before the sequence's
  uint32_t n = 0;  // its own
  for (int s = 0; s <= seq; ++s) {
    const int a = __ldg(p.cu_seqlens + s), b = __ldg(p.cu_seqlens + s + 1);
    if (goes_back(a, b)) return;
    sg += n;
    n = within(a, b, p.tokens) ? segments_of(static_cast<uint32_t>(b - a), tp.seg) : 0;
  }
  if (n <= 1) return;
  const int src = slot_of(p, p.src, seq, h == 0 && part == 0 && threadIdx.x == 0);  // (the segments do not look at it)
  const uint32_t e = 4 * (part * kJoinThreads + threadIdx.x);
  float R[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (src >= 0) {
    const int64_t at = src * p.state_ss + static_cast<int64_t>(h) * (kDim * kState) + e;
    for (int i = 0; i < 4; ++i) R[i] = load_state(p.state, at + i, p.state_dtype);
  }
  const int64_t step = static_cast<int64_t>(p.H) * (kDim * kState);
  float* at = tp.seg_state + (sg * p.H + h) * (kDim * kState) + e;
  const float* decay = tp.seg_decay + sg * p.H + h;
  constexpr uint32_t kAhead = 8;
  for (uint32_t s0 = 0; s0 < n; s0 += kAhead) {
    float4 own[kAhead];
    float a[kAhead];
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i) {
      const bool have = s0 + i + 1 < n;  // nothing follows the last
      own[i] = have ? *reinterpret_cast<const float4*>(at + (s0 + i) * step) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      a[i] = have ? exp2f(decay[static_cast<int64_t>(s0 + i) * p.H]) : 0.0f;
    }
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i) {
      if (s0 + i >= n) break;
      *reinterpret_cast<float4*>(at + (s0 + i) * step) = make_float4(R[0], R[1], R[2], R[3]);
      R[0] = fmaf(a[i], R[0], own[i].x);
      R[1] = fmaf(a[i], R[1], own[i].y);
      R[2] = fmaf(a[i], R[2], own[i].z);
      R[3] = fmaf(a[i], R[3], own[i].w);
    }
  }
}

}  // namespace ssm
