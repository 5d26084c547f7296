// attn_tile_kernel.cuh -- attention of new tokens over pages, on the tensor cores.
//
// For a key head the queries of its `per` heads and of all new tokens are the rows
// of one matrix Q: S = Q K^T, P = 2^(scale S - m), O = P V, with a running maximum m
// and sum l a row, so the cache is gone through once.
//
// Memory bounds it: 8 rows of 128 columns make 8 multiplications of a byte of keys and
// values.  So the cache is what is organised.  A CTA has four warps, and
// each streams a step of 8 to 32 tokens (4 to 16 KB of keys and values) at a time through shared memory of its
// own, two or three stages of it (TMA boxes of up to 16 tokens where pages are whole boxes; else gathers of
// four rows, a lane each, where the pages make one matrix of rows; else cp.async.  100000 tokens, 8
// key heads of 128, bf16, in pages of 16, 7 and 1 take 69, 74 and 80 us by boxes and gathers, 104 and
// 109 by cp.async of pages of 7 and 1): no barrier of the CTA holds a load back, and warps are joined
// only at the end of a request's part.  Weights are taken against a bound of the running maximum: where a score passes
// it, that row's bound becomes 2^8 times its maximum, and its sum and outputs are scaled anew, which takes a few steps of
// a request instead of all.  So a weight is at most one, and sums of large values do not overflow before their row's
// quotient would; the largest weight of a row is at least 2^-8, far from where fp32 and bf16 end.
//
// The bf16 products are m16n8k16 instructions on registers, taken the other way round, S^T = K Q^T and
// O^T = V^T P^T, so that rows come in eights, with P^T turned between them by
// movmatrix, as two bf16 parts up to 24 rows (attn_low()).  Up to 16 rows memory hides them.  (tcgen05 takes this form too, 128
// tokens or columns by rows in eights, with sums in tensor memory; that has not been built, so what it would give
// where products bind, from 24 rows on, is not known.)  The fp32 products run on the CUDA cores, in pairs (fma.rn.f32x2): three tf32
// products each would take three times the instructions, most of them to split the operands.
//
// Head sizes between the compiled ones (64, 128, 256) are padded with zeros on the chip; the
// padding is not read from memory.
//
// Measured on a GB300 (graphs of calls on changing caches): 200000 tokens in 64 requests, 8 key heads of 128, bf16,
// 126 to 129 us, 6.4 TB/s; one request of 131072 tokens, 2 key heads, 30 us, 4.5 TB/s (a call's start,
// seven microseconds of lookups and first loads, and the join are a third of it); drafts of 4
// tokens, 20 rows, 80000 tokens, 67 us, 4.9 TB/s; 50000 tokens, 8 heads of 128 in fp32, 70 us, 5.8
// TB/s.  From 32 rows on the products bind it: 8 new tokens of 4 heads a key head take 86 us where
// 4 take 76, and more go at 190 TFLOP/s.
//
// The work of a call is its (request, key head, group of rows) units' tiles of four steps,
// one after the other, and with each unit two to four tiles more for what its end takes; every CTA
// takes the same number of them, wherever they begin and end, so that lengths (which only
// the device knows) may differ as they like.  A unit that a CTA has to itself is finished
// by it; pieces of others go to the workspace, two a CTA at most, and attn_join_kernel puts
// them together.
#pragma once
#include <type_traits>
#include <utility>

#include "attn_plain_kernel.cuh"
#include "rsm_ptx.cuh"

namespace hybrid {

__device__ __forceinline__ int tiles_of(const AttnParams& p, int64_t len) {
  return static_cast<int>((len + (1 << p.tile_shift) - 1) >> p.tile_shift);
}

// What a unit of that many tiles counts.
__device__ __forceinline__ int64_t counts(const AttnParams& p, int tiles) { return tiles == 0 ? 0 : tiles + p.unit_end; }

// a / b; mostly of numbers of 32 bits, which take a fourth of the time.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (static_cast<uint64_t>(a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// How a call's tiles are dealt out, the same in both kernels: `more` CTAs have each + 1 of them, the others each.
struct AttnDeal {
  int64_t total;  // tiles, the units' ends among them
  int64_t ctas;   // that have any
  int64_t each, more;
  __device__ __forceinline__ AttnDeal(int64_t tiles, int64_t most_ctas) : total(tiles), ctas(min(most_ctas, tiles)) {
    each = ctas == 0 ? 0 : quotient(total, ctas);
    more = total - each * ctas;
  }
  __device__ __forceinline__ int64_t begin(int64_t c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int64_t owner(int64_t tile) const {
    const int64_t firsts = more * (each + 1);
    return tile < firsts ? quotient(tile, each + 1) : more + quotient(tile - firsts, each);
  }
};

struct Place {
  int b;          // a request
  int64_t first;  // its first tile
};

// The requests' tiles, in order; every function by the whole CTA.
template <int THREADS>
struct Deal {
  int64_t own, total;  // own: of request threadIdx.x
  __device__ __forceinline__ static int64_t of(const AttnParams& p, int b, bool report) {
    if (b >= p.pages.requests) return 0;
    return counts(p, tiles_of(p, request_tokens(p.pages, b, p.window, p.status, report))) * (p.G * p.row_tiles);
  }
  // (One use for each WHICH: its place is written once.)
  template <int WHICH>
  __device__ __forceinline__ static int64_t sum(int64_t n) {
    __shared__ int64_t sums[THREADS / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) n += sums[i];
    return n;
  }
  __device__ __forceinline__ Deal(const AttnParams& p, bool report) {
    own = of(p, threadIdx.x, report);
    int64_t n = own;
    for (int b = threadIdx.x + THREADS; b < p.pages.requests; b += THREADS) n += of(p, b, report);
    total = sum<0>(n);
  }
  // Tiles of the requests before b.
  __device__ __forceinline__ int64_t before(const AttnParams& p, int b) const {
    int64_t n = static_cast<int>(threadIdx.x) < b ? own : 0;
    for (int i = threadIdx.x + THREADS; i < b; i += THREADS) n += of(p, i, false);
    return sum<1>(n);
  }
  // The request that has tile number `tile` (below the total).
  __device__ __forceinline__ Place find(const AttnParams& p, int64_t tile) const {
    __shared__ int64_t sums[THREADS / 32];
    __shared__ Place place;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t before = 0;
    for (int base = 0;; base += THREADS) {
      const int b = base + static_cast<int>(threadIdx.x);
      const int64_t n = base == 0 ? own : of(p, b, false);
      int64_t upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
      }
      if (lane == 31) sums[warp] = upto;
      __syncthreads();
      int64_t all = before;
#pragma unroll
      for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) upto += sums[i];
        all += sums[i];
      }
      upto += before;
      if (tile < upto && tile >= upto - n) place = Place{b, upto - n};
      __syncthreads();
      if (tile < all || base + THREADS >= p.pages.requests) return place;
      before = all;
    }
  }
};

__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool yes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(yes ? 16 : 0) : "memory");
}

// The box of attn_box() tokens and 128 bytes at (column, head, row, page).
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, int column, int head, int row, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(column), "r"(head), "r"(row), "r"(page), "r"(bar)
      : "memory");
}

// 128 bytes of each of four rows.
__device__ __forceinline__ void gather_load(uint32_t dst, const CUtensorMap* map, int column, const int (&row)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(column), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar)
      : "memory");
}

template <int OFFSET>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at), "n"(OFFSET));
}
template <int OFFSET>
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at), "n"(OFFSET));
}
// f(0), f(1), ... f(N - 1), each with a constant of its own.
template <typename F, int... I>
__device__ __forceinline__ void each(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  each(f, std::make_integer_sequence<int, N>{});
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first of a sum.
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// Lane 4 i + j's values (i, 2 j) and (i, 2 j + 1) of an 8 x 8 matrix become (2 j, i) and (2 j + 1, i).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Where a 16-byte chunk of a token's row lies: boxes of a step's rows of 128 bytes, the chunks
// of a row in the order of the boxes' 128-byte swizzle, so that what the lanes of an
// instruction read lies in different banks.
template <int STEP>
__device__ __forceinline__ int chunk_at(int token, int chunk) {
  return (chunk >> 3) * (STEP * 128) + token * 128 + ((chunk & 7) ^ (token & 7)) * 16;
}

constexpr float kAttnRoom = 8.0f;  // log2 of how far the bound is above the maximum that it is taken of
constexpr float kAttnLowest = -3.402823466e38f;  // a maximum of nothing: no difference with it is NaN
constexpr uint64_t kAttnTimeoutNs = 2000000000ull;  // of a wait that takes microseconds

template <typename IT, int DIM, bool THREE>
struct AttnShape {
  static constexpr int kStep = attn_step(sizeof(IT), DIM, THREE);          // a warp's tokens of a stage
  static constexpr int kChunks = DIM * static_cast<int>(sizeof(IT)) / 16;  // of a row
  static constexpr int kHalf = kStep * DIM * static_cast<int>(sizeof(IT));  // a warp's keys of a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = attn_stages(sizeof(IT), DIM, THREE);
  static constexpr uint32_t kAll = kStep == 32 ? 0xFFFFFFFFu : (1u << kStep) - 1u;
};

// A place among the tiles, as one walks along them: request, key head, rows, tile.
struct AttnCursor {
  int b, g, rt, tile, tiles, len;
  __device__ __forceinline__ void at_request(const AttnParams& p) {
    len = static_cast<int>(request_tokens(p.pages, b, p.window, nullptr, false));
    tiles = tiles_of(p, len);
  }
  __device__ __forceinline__ void next_unit(const AttnParams& p) {
    tile = 0;
    if (++rt < p.row_tiles) return;
    rt = 0;
    if (++g < p.G) return;
    g = 0;
    do {
      if (++b >= p.pages.requests) {  // (behind the last: nothing more is looked at)
        len = tiles = 0;
        return;
      }
      at_request(p);
    } while (len == 0);
  }
  __device__ __forceinline__ void next(const AttnParams& p) {
    if (++tile == tiles) next_unit(p);
  }
  // Row r of the unit: its queries (null: there is none) and the last token that it sees.
  template <typename IT>
  __device__ __forceinline__ const IT* query(const AttnParams& p, int rows, int row, int& last) const {
    const int r = rt * rows + row, t = r / p.per;
    last = len - p.window + t;
    if (r >= p.per * p.window || len == 0) return nullptr;
    return static_cast<const IT*>(p.q) + b * p.q_bs + t * p.q_ts + static_cast<int64_t>(g * p.per + r - t * p.per) * p.dim;
  }
};

// A stage of a warp as its products take it: the tokens from `row`, the first of which is the
// request's token0; those of the bits `seen` (from bit 0 on) are there.
struct AttnStep {
  uint32_t keys, values;  // shared memory
  char* held;             // the values, to change them
  uint32_t seen;
  int row, token0;
  bool differ;            // rows differ in what they see
  int first_new;          // of these tokens, the first that is not seen by all rows
};

// New tokens' values that are not finite go to the rows that see them, by add(token), and not
// into the product, where a weight of zero would not keep them from the others.  TOKENS from a.row on.
template <typename IT, int DIM, int STEP, int TOKENS, typename F>
__device__ __forceinline__ void odd_values(const AttnStep& a, int lane, F add) {
  constexpr int kChunks = DIM * static_cast<int>(sizeof(IT)) / 16;
  bool odd = false;
  for (int c = lane; c < TOKENS * kChunks; c += 32) {
    const int j = c / kChunks;
    if (j < a.first_new) continue;
    const uint4 v = rsm::lds128(a.values + chunk_at<STEP>(a.row + j, c % kChunks));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      odd |= (w[k] & 0x7F800000u) == 0x7F800000u;
      if (sizeof(IT) == 2) odd |= (w[k] & 0x7F80u) == 0x7F80u;
    }
  }
  if (!__any_sync(0xFFFFFFFFu, odd)) return;
  for (int j = a.first_new; j < TOKENS; ++j)
    if (a.seen >> j & 1u) add(j);
  __syncwarp();
  for (int c = lane; c < TOKENS * kChunks; c += 32) {
    const int j = c / kChunks;
    if (j < a.first_new) continue;
    IT* v = reinterpret_cast<IT*>(a.held + chunk_at<STEP>(a.row + j, c % kChunks));
#pragma unroll
    for (int k = 0; k < 16 / static_cast<int>(sizeof(IT)); ++k)
      if (!isfinite(get(v + k))) v[k] = IT(0);
  }
  rsm::fence_proxy_async_smem();
  __syncwarp();
}

template <typename IT, int STEP>
__device__ __forceinline__ float held_value(const AttnStep& a, int token, int column) {
  const int c = column * static_cast<int>(sizeof(IT));
  return get(reinterpret_cast<const IT*>(a.held + chunk_at<STEP>(a.row + token, c / 16) + c % 16));
}

// A warp's part of a unit, bf16: 8 N rows.  Lane (quad, four) holds of S^T tokens quad and quad
// + 8, rows 8 n + 2 four + {0, 1}; of O^T columns 16 i + quad and + 8, the same rows.  Queries stay in
// registers where outputs leave room for them (attn_shared_queries()), else in shared memory.
// LOW: weights meet the values as sums of two bf16 values, 16 bits of them, else rounded to 8.
template <int DIM, int N, bool THREE, bool LOW>
struct AttnBf16 {
  using IT = uint16_t;
  using Shape = AttnShape<IT, DIM, THREE>;
  static constexpr bool kThree = THREE;
  static constexpr int kRows = 8 * N, kSteps = DIM / 16, kTokens = 16, kStep = Shape::kStep;
  static constexpr bool kShared = attn_shared_queries(DIM, kRows);
  static constexpr int kQuery = attn_query(2, DIM, kRows);
  static constexpr int kChains = N == 1 ? 4 : N == 2 ? 2 : 1;  // sums that do not wait for one another
  static constexpr int kOwn = kShared ? (kRows * DIM / 8 + kAttnThreads - 1) / kAttnThreads : 1;  // a thread's chunks of the queries
  // The next unit's queries are asked for before this one's last products, where they come to shared memory
  // (32 rows, 100000 tokens: 106 -> 99 us; in registers, which that takes more of, no difference).
  static constexpr bool kEarly = kShared;
  uint32_t q[kShared ? 1 : N][kShared ? 1 : kSteps][2];
  uint4 next[kOwn];
  int limit[N][2];
  float o[kSteps][N][4], m[N][2], l[N][2];

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
      m[n][0] = m[n][1] = kAttnLowest;
      l[n][0] = l[n][1] = 0.0f;
    }
  }
  // A unit's queries: asked for by fetch(), there after commit().
  __device__ __forceinline__ void fetch(const AttnParams& p, const AttnCursor& at, int lane) {
    if constexpr (kShared) {
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        const int c = threadIdx.x + k * kAttnThreads, row = c / (DIM / 8), col = c % (DIM / 8) * 8;
        next[k] = make_uint4(0, 0, 0, 0);
        if (c >= kRows * DIM / 8 || col >= p.dim) continue;
        int last;
        const IT* from = at.query<IT>(p, kRows, row, last);
        if (from == nullptr) continue;
        if (p.q_wide) {
          next[k] = *reinterpret_cast<const uint4*>(from + col);
        } else {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = static_cast<uint32_t>(from[col + 2 * e]) | static_cast<uint32_t>(from[col + 2 * e + 1]) << 16;
          next[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    } else {
      const int quad = lane >> 2, four = lane & 3;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        int last;
        const IT* from = at.query<IT>(p, kRows, 8 * n + quad, last);
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t v = 0;
            const int c = 16 * ks + 8 * e + 2 * four;
            if (from != nullptr && c < p.dim)
              v = p.q_pairs ? *reinterpret_cast<const uint32_t*>(from + c) : static_cast<uint32_t>(from[c]) | static_cast<uint32_t>(from[c + 1]) << 16;
            q[n][ks][e] = v;
          }
      }
    }
  }
  __device__ __forceinline__ void commit(const AttnParams& p, const AttnCursor& at, int lane, char* smem) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) (void)at.query<IT>(p, kRows, 8 * n + 2 * (lane & 3) + e, limit[n][e]);
    if constexpr (kShared) {
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        const int c = threadIdx.x + k * kAttnThreads, row = c / (DIM / 8), chunk = c % (DIM / 8);
        if (c < kRows * DIM / 8) *reinterpret_cast<uint4*>(smem + row * (2 * DIM) + ((chunk & ~7) | ((chunk ^ row) & 7)) * 16) = next[k];
      }
      __syncthreads();
    }
  }
  // What is left of weight w, bits b, behind its upper 16 bits.  Not zero where the weight is not: an infinite
  // value times either part is infinite.
  __device__ __forceinline__ static float rest(float w, uint32_t b) {
    return fmaxf(w - __uint_as_float(b & 0xFFFF0000u), fminf(w, 1.17549435e-38f));
  }
  __device__ __forceinline__ void step(const AttnParams& p, const AttnStep& a, const AttnCursor&, int lane, const char* smem) {
    const int quad = lane >> 2, four = lane & 3;
    float part[kChains][N][4], s[N][4];
    [[maybe_unused]] uint32_t pair[kShared ? N : 1][4];  // queries' chunks for two steps
    {
      // Chunks 2 ks and 2 ks + 1 of a token's row: the swizzle turns a chunk's number's lowest three bits by the
      // token's, so that beside the lane's own bits a step is one more turn, or an offset.
      const int token = a.row + (lane & 15), odd = lane >> 4;
      const uint32_t keys = a.keys + token * 128 + ((odd ^ token) & 7) * 16;
      const uint32_t queries = rsm::smem_addr(smem) + (lane & 7) * (2 * DIM) + (((lane >> 3) ^ lane) & 7) * 16;
      each<kSteps>([&](auto index) {
        constexpr int ks = decltype(index)::value;
        uint32_t ka[4];
        ldmatrix4<(ks / 4) * (kStep * 128)>(ka, keys ^ (ks % 4 * 32));
        each<N>([&](auto which) {
          constexpr int n = decltype(which)::value;
          uint32_t b0, b1;
          if constexpr (kShared) {
            if constexpr (ks % 2 == 0) ldmatrix4<n * (16 * DIM) + (ks / 4) * 128>(pair[n], queries ^ (ks / 2 % 2 * 64));
            b0 = pair[n][ks % 2 * 2], b1 = pair[n][ks % 2 * 2 + 1];
          } else {
            b0 = q[n][ks][0], b1 = q[n][ks][1];
          }
          if constexpr (ks < kChains)
            mma_bf16_first(part[ks][n], ka, b0, b1);
          else
            mma_bf16(part[ks % kChains][n], ka, b0, b1);
        });
      });
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = part[0][n][e];
#pragma unroll
        for (int c = 1; c < kChains; ++c) s[n][e] += part[c][n][e];
      }
    if (a.differ || (a.seen & 0xFFFFu) != 0xFFFFu) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = quad + 8 * (e >> 1);
          if (!(a.seen >> j & 1u) || a.token0 + j > limit[n][e & 1]) s[n][e] = p.hidden;
        }
    }
    // t = log2 of the weights
    bool above = false;
    float t[N][4];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[n][e] = fmaf(s[n][e], p.scale_log2, -m[n][e & 1]);
        above |= t[n][e] > 0.0f;
      }
    if (__any_sync(0xFFFFFFFFu, above)) {  // some row's bound moves
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(s[n][e] * p.scale_log2, s[n][e + 2] * p.scale_log2);
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
          const float next = top > m[n][e] ? top + kAttnRoom : m[n][e], keep = exp2_fast(m[n][e] - next);
          m[n][e] = next;
          l[n][e] *= keep;
          t[n][e] = fmaf(s[n][e], p.scale_log2, -next);
          t[n][e + 2] = fmaf(s[n][e + 2], p.scale_log2, -next);
#pragma unroll
          for (int i = 0; i < kSteps; ++i) o[i][n][e] *= keep, o[i][n][e + 2] *= keep;
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = exp2_fast(t[n][e]);
        l[n][e & 1] += s[n][e];
      }
    if (a.differ && p.window > 1)
      odd_values<IT, DIM, kStep, kTokens>(a, lane, [&](int j) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w = __shfl_sync(0xFFFFFFFFu, j & 8 ? s[n][e + 2] : s[n][e], (j & 7) * 4 + four);
            if (a.token0 + j > limit[n][e]) continue;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float v = held_value<IT, kStep>(a, j, 16 * i + 8 * h + quad);
                if (!isfinite(v)) o[i][n][2 * h + e] += w * v;
              }
          }
      });
    uint32_t pb[N][2];
    [[maybe_unused]] uint32_t low[LOW ? N : 1][2];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float w0 = s[n][2 * h], w1 = s[n][2 * h + 1];
        if constexpr (LOW) {
          const uint32_t b0 = __float_as_uint(w0), b1 = __float_as_uint(w1);
          pb[n][h] = transpose8(__byte_perm(b0, b1, 0x7632));
          low[n][h] = transpose8(rsm::pack_bf16x2(rest(w0, b0), rest(w1, b1)));
        } else {
          pb[n][h] = transpose8(rsm::pack_bf16x2(w0, w1));
        }
      }
    const int token = a.row + (lane >> 4) * 8 + (lane & 7), odd = lane >> 3 & 1;
    const uint32_t values = a.values + token * 128 + ((odd ^ token) & 7) * 16;
    each<kSteps>([&](auto index) {
      constexpr int i = decltype(index)::value;
      uint32_t va[4];
      ldmatrix4_trans<(i / 4) * (kStep * 128)>(va, values ^ (i % 4 * 32));
#pragma unroll
      for (int n = 0; n < N; ++n) {
        mma_bf16(o[i][n], va, pb[n][0], pb[n][1]);
        if constexpr (LOW) mma_bf16(o[i][n], va, low[n][0], low[n][1]);
      }
    });
  }
  __device__ __forceinline__ void stats(float* ms, float* ls, int lane) const {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
        if (lane < 4) ms[8 * n + 2 * lane + e] = m[n][e], ls[8 * n + 2 * lane + e] = sum;
      }
  }
  // Rows 16 pass and up, 16 of them at most, as own[row][DIM]: columns in the order of place().
  __device__ __forceinline__ static int place(int row, int column) { return row * DIM + (column ^ (row >> 1 & 3) << 3); }
  template <int PASS>
  __device__ __forceinline__ void outputs(float* own, int lane) const {
    const int quad = lane >> 2, four = lane & 3;
#pragma unroll
    for (int n = 2 * PASS; n < (2 * PASS + 2 < N ? 2 * PASS + 2 : N); ++n)
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) own[place(8 * (n & 1) + 2 * four + (e & 1), 16 * i + 8 * (e >> 1) + quad)] = o[i][n][e];
  }
};

// The same for fp32, R rows (1, 2, 4 or 8), all tokens of a stage.  For the scores lane (slice, group) = (lane & 7,
// lane >> 3) sums over the 16-byte chunks slice + 8 j of a quarter of the tokens, `group`'s, and
// the slices are then added up in halves, so that each lane ends with a token and half of the rows;
// the weights go through shared memory, and a lane adds its columns' values for all rows.
template <int DIM, int R>
struct AttnF32 {
  using IT = float;
  using Shape = AttnShape<IT, DIM, false>;
  static constexpr bool kThree = false;
  static constexpr int kRows = R, kStep = Shape::kStep, kTokens = kStep, kQuery = attn_query(4, DIM, R);
  static constexpr int kTake = kStep / 4;             // a group's tokens
  static constexpr int kChunks = DIM / 32;            // a slice's
  static constexpr int kHalf = R > 1 ? R / 2 : 1;     // rows that a lane ends with
  static constexpr int kCols = DIM / 32;              // columns of a lane
  static_assert(kTake == 2 || kTake == 4);
  uint64_t q[R][kChunks][2];
  int limit[kHalf];
  uint64_t o[R][kCols / 2];
  float m[kHalf], l[kHalf];

  __device__ __forceinline__ static uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ static float2 both(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
  }
  __device__ __forceinline__ static uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
  }
  __device__ __forceinline__ static void lds_pairs(uint32_t at, uint64_t& a, uint64_t& b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(at));
  }
  // The token of the stage and the first row that lane ends with.
  __device__ __forceinline__ static int own_token(int lane) {
    return kTake == 4 ? (lane >> 3) * 4 + (lane & 1) * 2 + (lane >> 1 & 1) : (lane >> 3) * 2 + (lane & 1);
  }
  // (Two tokens a group: the second bit takes a half of the rows too.)
  __device__ __forceinline__ static int own_row(int lane) {
    if (kTake == 4) return R > 1 ? (lane >> 2 & 1) * kHalf : 0;
    return R > 2 ? (lane >> 1 & 1) * (R / 2) + (lane >> 2 & 1) * (R / 4) : R > 1 ? (lane >> 1 & 1) : 0;
  }
  static constexpr bool kEarly = false;
  static constexpr int kKept = kTake == 4 ? kHalf : R > 2 ? R / 4 : 1;  // rows that a lane ends with, kHalf or fewer

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) o[r][c] = 0;
#pragma unroll
    for (int h = 0; h < kKept; ++h) m[h] = kAttnLowest, l[h] = 0.0f;
  }
  __device__ __forceinline__ void fetch(const AttnParams& p, const AttnCursor& at, int lane) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int last;
      const IT* from = at.query<IT>(p, R, r, last);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int c = 4 * ((lane & 7) + 8 * j);
        q[r][j][0] = q[r][j][1] = 0;
        if (from == nullptr || c >= p.dim) continue;
        if (p.q_wide) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(from + c);
          q[r][j][0] = v.x, q[r][j][1] = v.y;
        } else {
          q[r][j][0] = pair(from[c], from[c + 1]), q[r][j][1] = pair(from[c + 2], from[c + 3]);
        }
      }
    }
  }
  __device__ __forceinline__ void commit(const AttnParams& p, const AttnCursor& at, int lane, char*) {
#pragma unroll
    for (int h = 0; h < kKept; ++h) (void)at.query<IT>(p, R, own_row(lane) + h, limit[h]);
  }
  __device__ __forceinline__ void step(const AttnParams& p, const AttnStep& a, const AttnCursor& at, int lane, char* smem) {
    const int slice = lane & 7, group = lane >> 3;
    float v[kTake * R];
#pragma unroll
    for (int t = 0; t < kTake; ++t) {
      const int token = group * kTake + t;
      uint64_t acc[R];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = 0;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        uint64_t k0, k1;
        lds_pairs(a.keys + chunk_at<kStep>(token, slice + 8 * j), k0, k1);
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = fma2(k1, q[r][j][1], fma2(k0, q[r][j][0], acc[r]));
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 x = both(acc[r]);
        v[t * R + r] = x.x + x.y;
      }
    }
    // the slices' sums: each exchange adds and halves what a lane has, while it has more than one
    int have = kTake * R;
#pragma unroll
    for (int bit = 1; bit < 8; bit <<= 1) {
      const bool upper = lane & bit;
      if (have > 1) {
        have /= 2;
#pragma unroll
        for (int i = 0; i < kTake * R / 2; ++i)
          if (i < have) {
            const float send = upper ? v[i] : v[i + have], keep = upper ? v[i + have] : v[i];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, bit);
          }
      } else {
        v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], bit);
      }
    }
    const int j = own_token(lane);
    if (a.differ || a.seen != Shape::kAll) {
#pragma unroll
      for (int h = 0; h < kKept; ++h)
        if (!(a.seen >> j & 1u) || a.token0 + j > limit[h]) v[h] = p.hidden;
    }
    bool above = false;
#pragma unroll
    for (int h = 0; h < kKept; ++h) above |= fmaf(v[h], p.scale_log2, -m[h]) > 0.0f;
    if (__any_sync(0xFFFFFFFFu, above)) {  // some row's bound moves
      float keep[kKept];
#pragma unroll
      for (int h = 0; h < kKept; ++h) {
        float top = v[h] * p.scale_log2;
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        if (kTake == 4) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
        const float next = top > m[h] ? top + kAttnRoom : m[h];
        keep[h] = exp2_fast(m[h] - next);
        m[h] = next;
        l[h] *= keep[h];
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {  // from a lane that has row r
        const int from = kTake == 4 ? (R > 1 ? r / kHalf * 4 : 0) : R > 2 ? r / (R / 2) * 2 + r / (R / 4) % 2 * 4 : R > 1 ? r * 2 : 0;
        const float f = __shfl_sync(0xFFFFFFFFu, keep[r % kKept], from);
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) {
          const float2 x = both(o[r][c]);
          o[r][c] = pair(x.x * f, x.y * f);
        }
      }
    }
    // weights, each twice, [token][row]
    const uint32_t weights = rsm::smem_addr(smem) + (threadIdx.x >> 5) * (kStep * R * 8);
#pragma unroll
    for (int h = 0; h < kKept; ++h) {
      const float w = exp2_fast(fmaf(v[h], p.scale_log2, -m[h]));
      // (a token and row that two lanes end with counts once)
      l[h] += kTake == 4 ? (R > 1 || !(lane & 4) ? w : 0.0f) : (R > 2 || !(lane & 4)) && (R > 1 || !(lane & 2)) ? w : 0.0f;
      asm volatile("st.shared.v2.f32 [%0], {%1, %1};" ::"r"(weights + (j * R + own_row(lane) + h) * 8), "f"(w) : "memory");
    }
    __syncwarp();
    if (a.differ && p.window > 1)
      odd_values<IT, DIM, kStep, kTokens>(a, lane, [&](int t) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          int last;
          (void)at.query<IT>(p, R, r, last);
          float w;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w) : "r"(weights + (t * R + r) * 8));
          if (a.token0 + t > last) continue;
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {
            float2 x = both(o[r][c]);
            const float v0 = held_value<IT, kStep>(a, t, column(lane, 2 * c)), v1 = held_value<IT, kStep>(a, t, column(lane, 2 * c + 1));
            if (!isfinite(v0)) x.x += w * v0;
            if (!isfinite(v1)) x.y += w * v1;
            o[r][c] = pair(x.x, x.y);
          }
        }
      });
#pragma unroll
    for (int t = 0; t < kStep; ++t) {
      uint64_t x[kCols / 2];
#pragma unroll
      for (int c = 0; c < kCols / 4; ++c) lds_pairs(a.values + chunk_at<kStep>(t, lane + 32 * c), x[2 * c], x[2 * c + 1]);
      if constexpr (kCols == 2) asm volatile("ld.shared.b64 %0, [%1];" : "=l"(x[0]) : "r"(a.values + chunk_at<kStep>(t, lane >> 1) + (lane & 1) * 8));
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        uint64_t w0, w1 = 0;
        if constexpr (R > 1)
          lds_pairs(weights + (t * R + r) * 8, w0, w1);
        else
          asm volatile("ld.shared.b64 %0, [%1];" : "=l"(w0) : "r"(weights + t * 8));
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) {
          o[r][c] = fma2(w0, x[c], o[r][c]);
          if (R > 1) o[r + (R > 1)][c] = fma2(w1, x[c], o[r + (R > 1)][c]);
        }
      }
    }
  }
  // The column of a lane's c-th.
  __device__ __forceinline__ static int column(int lane, int c) { return kCols == 2 ? 2 * lane + c : 4 * (lane + 32 * (c / 4)) + c % 4; }
  __device__ __forceinline__ void stats(float* ms, float* ls, int lane) const {
#pragma unroll
    for (int h = 0; h < kKept; ++h) {
      float sum = l[h];
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      if (kTake == 4 || R == 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      if ((kTake == 4 && R == 1) || (kTake == 2 && R <= 2)) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
      if ((lane & 25) == 0) ms[own_row(lane) + h] = m[h], ls[own_row(lane) + h] = sum;
    }
  }
  __device__ __forceinline__ static int place(int row, int column) { return row * DIM + column; }
  template <int PASS>
  __device__ __forceinline__ void outputs(float* own, int lane) const {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) *reinterpret_cast<float2*>(own + place(r, column(lane, 2 * c))) = both(o[r][c]);
  }
};

// LOADS: by TMA in boxes of attn_box() rows, where the pages are whole boxes, or four rows at a time from
// anywhere; or by cp.async.
template <typename Math, int DIM, AttnLoads LOADS>
__global__ void __launch_bounds__(kAttnThreads, attn_ctas_per_sm(sizeof(typename Math::IT), DIM, Math::kThree))
    attn_tile_kernel(const __grid_constant__ AttnTileParams tp) {
  using IT = typename Math::IT;
  using Shape = typename Math::Shape;
  constexpr int kWarps = kAttnThreads / 32, kRows = Math::kRows, S = Shape::kStages, kChunks = Shape::kChunks;
  constexpr int kStep = Shape::kStep, kTile = 4 * kStep, kTokens = Math::kTokens, kBox = 128 / static_cast<int>(sizeof(IT));  // columns of a box
  constexpr bool BOXES = LOADS == AttnLoads::kBoxes, GATHER = LOADS == AttnLoads::kGather, TMA = BOXES || GATHER;
  constexpr int kBoxRows = attn_box(sizeof(IT), DIM), kParts = BOXES ? kStep / kBoxRows : 1;  // a step's boxes of rows
  constexpr uint32_t kAll = Shape::kAll;
  extern __shared__ __align__(1024) char smem[];
  __shared__ float m_s[kWarps][kRows], l_s[kWarps][kRows];
  __shared__ uint32_t seen_s[kWarps][S];
  __shared__ __align__(8) uint64_t full_s[kWarps][S];  // TMA: a stage's loads
  const AttnParams& p = tp.p;
  const rsm_pages& pg = p.pages;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (TMA) {
    if (lane == 0) {
      for (int i = 0; i < S; ++i) rsm::mbar_init(rsm::smem_addr(&full_s[warp][i]), 1);
      rsm::fence_mbar_init();
      asm volatile("prefetch.tensormap [%0];" ::"l"(&tp.k_map) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(&tp.v_map) : "memory");
    }
    __syncwarp();
  }

  auto skipped = [&]() {  // rows of skipped requests
    for (int b = blockIdx.x; b < pg.requests; b += gridDim.x)
      if (request_tokens(pg, b, p.window, nullptr, false) == 0) {
        const int64_t n = static_cast<int64_t>(p.window) * p.H * p.dim;
        IT* out = static_cast<IT*>(p.out) + b * n;
        for (int64_t i = threadIdx.x; i < n; i += kAttnThreads) out[i] = IT(0);
      }
  };
  const Deal<kAttnThreads> requests(p, blockIdx.x == 0);
  const AttnDeal deal(requests.total, gridDim.x);
  if (blockIdx.x >= deal.ctas) return skipped();
  const int64_t begin = deal.begin(blockIdx.x);
  const Place place = requests.find(p, begin);
  // `room` is what is left of this CTA's share where `at` stands.
  int64_t room = deal.begin(blockIdx.x + 1) - begin;
  AttnCursor at;
  at.b = place.b;
  at.at_request(p);
  {
    const int64_t into = begin - place.first;
    const int unit = static_cast<int>(quotient(into, counts(p, at.tiles))), tile = static_cast<int>(into - unit * counts(p, at.tiles));
    at.g = unit / p.row_tiles;
    at.rt = unit - at.g * p.row_tiles;
    at.tile = tile;
    if (tile >= at.tiles) {  // the share begins in what a unit's end counts
      room -= counts(p, at.tiles) - tile;
      if (room <= 0) return skipped();
      at.next_unit(p);
    }
  }
  AttnCursor ask = at;
  int64_t ask_room = room;

  // ---- loads: a warp's step of a tile ----
  const uint32_t ring = rsm::smem_addr(smem) + Math::kQuery + warp * (S * Shape::kStage);
  const uint32_t full = rsm::smem_addr(&full_s[warp][0]);
  const bool one_page = BOXES || (!GATHER && pg.page_size % kStep == 0);  // a step, or a box, lies in one page
  auto first_bits = [](int n) { return n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };
  auto page_at = [&](int64_t token) {
    if (token >= ask.len) return -1;  // no token
    const int i = p.page_shift >= 0 ? static_cast<int>(token) >> p.page_shift : static_cast<int>(token) / pg.page_size;
    return __ldg(pg.page_table + ask.b * pg.table_stride + i);
  };
  // One page a step (or box): a lane looks up that of a tile's, 32 at once; else a lane a token, a step ahead.
  constexpr int kLook = 32 / kParts;  // tiles
  int looked = -1, pages = -1;
  auto look_up = [&](bool request) {
    if (one_page) {
      const int group = ask.tile / kLook;
      if (!request && group == looked) return;
      looked = group;
      pages = page_at((static_cast<int64_t>(group) * kLook + lane / kParts) * kTile + warp * kStep + lane % kParts * kBoxRows);
    } else {
      pages = page_at(static_cast<int64_t>(ask.tile) * kTile + warp * kStep + lane % kStep);
    }
  };
  look_up(true);
  auto load = [&](int stage) {
    if (ask_room <= 0) {
      if constexpr (!TMA) cp_async_commit();
      return;
    }
    const int g = ask.g, token0 = ask.tile * kTile + warp * kStep;
    const uint32_t base = ring + stage * Shape::kStage;
    uint32_t seen = 0;
    if constexpr (BOXES) {
      int page[kParts];
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        const int token = token0 + h * kBoxRows;
        page[h] = __shfl_sync(0xFFFFFFFFu, pages, ask.tile % kLook * kParts + h);
        if (page[h] >= 0 && page[h] < pg.num_pages) {
          seen |= first_bits(min(kBoxRows, ask.len - token)) << (h * kBoxRows);
        } else {
          page[h] = -1;
          if (token < ask.len) flag(p.status, RSM_STATUS_BAD_PAGE);
        }
      }
      if (lane == 0) {
        const uint32_t bar = full + stage * 8;
        uint32_t bytes = 0;
#pragma unroll
        for (int h = 0; h < kParts; ++h) bytes += page[h] >= 0 ? Shape::kStage / kParts : 0;
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          if (page[h] < 0) continue;
          const int token = token0 + h * kBoxRows, row = p.page_shift >= 0 ? token & (pg.page_size - 1) : token % pg.page_size;
#pragma unroll
          for (int c = 0; c < DIM / kBox; ++c) {
            const uint32_t to = base + c * (kStep * 128) + h * (kBoxRows * 128);
            box_load(to, &tp.k_map, kBox * c, g, row, page[h], bar);
            box_load(to + Shape::kHalf, &tp.v_map, kBox * c, g, row, page[h], bar);
          }
        }
      }
    } else if constexpr (GATHER) {
      // a lane a token's row, then a lane four rows' 128 bytes of keys or of values
      const bool good = pages >= 0 && pages < pg.num_pages;
      const int token = token0 + lane % kStep;
      if (!good && token < ask.len) flag(p.status, RSM_STATUS_BAD_PAGE);
      const int row = p.page_shift >= 0 ? token & (pg.page_size - 1) : token % pg.page_size;
      const int index = good ? pages * p.page_rows + row + g * p.head_rows : 0;  // (the first row stands in for none)
      seen = __ballot_sync(0xFFFFFFFFu, good) & kAll;
      constexpr int kGroups = kStep / 4, kColumns = DIM / kBox;
      static_assert(2 * kGroups * kColumns <= 32);
      const int group = lane % kGroups, column = lane / kGroups % kColumns, value = lane / (kGroups * kColumns);
      const uint32_t bar = full + stage * 8;
      if (lane == 0) mbar_arrive_expect_tx(bar, __popc((seen | seen >> 1 | seen >> 2 | seen >> 3) & 0x11111111u) * (Shape::kStage / kGroups));
      int rows[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) rows[k] = __shfl_sync(0xFFFFFFFFu, index, 4 * group + k);
      __syncwarp();
      if (value < 2 && (seen >> (4 * group) & 15u) != 0)
        gather_load(base + value * Shape::kHalf + column * (kStep * 128) + group * 512, value == 0 ? &tp.k_map : &tp.v_map,
                    g * p.head_columns + kBox * column, rows, bar);
    } else {
      const int page = one_page ? __shfl_sync(0xFFFFFFFFu, pages, ask.tile % kLook) : pages;
      const bool good = page >= 0 && page < pg.num_pages;
      if (!good && token0 + (one_page ? 0 : lane % kStep) < ask.len) flag(p.status, RSM_STATUS_BAD_PAGE);
      const int token = token0 + (one_page ? 0 : lane % kStep), chunks = p.dim * static_cast<int>(sizeof(IT)) / 16;
      const int row = p.page_shift >= 0 ? token & (pg.page_size - 1) : token % pg.page_size;
      seen = one_page ? (good ? first_bits(min(kStep, ask.len - token0)) : 0u) : __ballot_sync(0xFFFFFFFFu, good) & kAll;
#pragma unroll 4
      for (int i = 0; i < kStep * kChunks / 32; ++i) {
        const int f = i * 32 + lane, r = f / kChunks, chunk = f % kChunks;
        int pr = page, rr = row + r;
        if (!one_page) pr = __shfl_sync(0xFFFFFFFFu, page, r), rr = __shfl_sync(0xFFFFFFFFu, row, r);
        const bool yes = (seen >> r & 1u) && chunk < chunks;
        const IT* kr = static_cast<const IT*>(pg.k) + (yes ? pr * pg.k_page_stride + rr * pg.k_row_stride + g * pg.k_head_stride : 0);
        const IT* vr = static_cast<const IT*>(pg.v) + (yes ? pr * pg.v_page_stride + rr * pg.v_row_stride + g * pg.v_head_stride : 0);
        cp_async_16_or_zero(base + chunk_at<kStep>(r, chunk), reinterpret_cast<const char*>(kr) + (yes ? chunk * 16 : 0), yes);
        cp_async_16_or_zero(base + Shape::kHalf + chunk_at<kStep>(r, chunk), reinterpret_cast<const char*>(vr) + (yes ? chunk * 16 : 0), yes);
      }
      cp_async_commit();
    }
    if (lane == 0) seen_s[warp][stage] = seen;
    ask_room -= ask.tile + 1 == ask.tiles ? 1 + p.unit_end : 1;
    if (ask_room > 0) {
      const int b = ask.b;
      ask.next(p);
      look_up(ask.b != b);
    }
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) load(s);

  Math math;
  math.fetch(p, at, lane);
  skipped();
  math.commit(p, at, lane, smem);
  math.reset();
  int from = at.tile;  // the piece's first tile
  uint32_t phase = 0;
  for (int stage = 0;;) {
    AttnCursor then = at;  // the unit after this one
    if constexpr (Math::kEarly) {
      if (at.tile + 1 == at.tiles && room > 1 + p.unit_end) {
        then.next_unit(p);
        math.fetch(p, then, lane);
      }
    }
    if constexpr (TMA) {
      if (!rsm::mbar_wait(full + stage * 8, phase, kAttnTimeoutNs)) {  // (never expected)
        flag(p.status, RSM_STATUS_WAIT_TIMEOUT);
        for (int k = 0; k < S; ++k) (void)rsm::mbar_wait(full + k * 8, k < stage ? phase ^ 1u : phase, 1000000ull);  // copies on the way
        return;
      }
    } else {
      cp_async_wait<S - 2>();
    }
    __syncwarp();
    load(stage == 0 ? S - 1 : stage - 1);
    AttnStep a;
    a.seen = seen_s[warp][stage];
    if (a.seen != 0) {
      a.keys = ring + stage * Shape::kStage;
      a.values = a.keys + Shape::kHalf;
      a.held = smem + (a.values - rsm::smem_addr(smem));
      if constexpr (TMA) {  // rows behind the last token came with the others
        if (a.seen != kAll) {
          for (int c = lane; c < kStep * kChunks; c += 32)
            if (!(a.seen >> ((c >> 3) % kStep) & 1u)) *reinterpret_cast<uint4*>(a.held + c * 16) = make_uint4(0, 0, 0, 0);
          rsm::fence_proxy_async_smem();
          __syncwarp();
        }
      }
      const uint32_t all_seen = a.seen;
#pragma unroll
      for (int sub = 0; sub < kStep / kTokens; ++sub) {
        a.row = sub * kTokens;
        a.seen = all_seen >> a.row;
        if (sub > 0 && a.seen == 0) break;
        a.token0 = at.tile * kTile + warp * kStep + a.row;
        a.differ = a.token0 + kTokens - 1 > at.len - p.window;
        a.first_new = max(at.len - p.window + 1 - a.token0, 0);
        math.step(p, a, at, lane, smem);
      }
    }

    // ---- the end of a unit, or of this CTA's part of it ----
    const bool last_tile = at.tile + 1 == at.tiles;
    room -= last_tile ? 1 + p.unit_end : 1;
    const bool over = room <= 0;
    if (last_tile || over) {
      const AttnCursor was = at;
      const bool whole = from == 0 && last_tile;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (from == 0 ? 1 : 0);
      math.stats(m_s[warp], l_s[warp], lane);
      if (!over) {  // the next unit's queries are on their way meanwhile
        if constexpr (Math::kEarly) {
          at = then;
        } else {
          at.next(p);
          math.fetch(p, at, lane);
        }
      }
      // the warps' outputs pass through the stages just read, 16 rows at a time
      char* const pass_at = smem + Math::kQuery + stage * Shape::kStage;
      auto pass = [&](auto index) {
        constexpr int kPass = decltype(index)::value, kHere = kRows - 16 * kPass < 16 ? kRows - 16 * kPass : 16;
        math.template outputs<kPass>(reinterpret_cast<float*>(pass_at + warp * (S * Shape::kStage)), lane);
        __syncthreads();
        for (int c = threadIdx.x; c < kHere * DIM / 4; c += kAttnThreads) {
          const int row = c / (DIM / 4), col = (c - row * (DIM / 4)) * 4, r = 16 * kPass + row, all = was.rt * kRows + r;
          if (all >= p.per * p.window || col >= p.dim) continue;
          float top = -INFINITY, sum = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w][r]);
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_fast(m_s[w][r] - top);
            const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(pass_at + w * (S * Shape::kStage)) + Math::place(row, col));
            y.x = fmaf(v.x, f, y.x), y.y = fmaf(v.y, f, y.y), y.z = fmaf(v.z, f, y.z), y.w = fmaf(v.w, f, y.w);
            sum = fmaf(l_s[w][r], f, sum);
          }
          if (whole) {
            const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
            const int t = all / p.per;
            IT* out = static_cast<IT*>(p.out) + ((static_cast<int64_t>(was.b) * p.window + t) * p.H + was.g * p.per + all - t * p.per) * p.dim + col;
            if (!p.out_wide)
              put(out, y.x * f), put(out + 1, y.y * f), put(out + 2, y.z * f), put(out + 3, y.w * f);
            else if constexpr (sizeof(IT) == 4)
              *reinterpret_cast<float4*>(out) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
            else
              *reinterpret_cast<uint2*>(out) = make_uint2(rsm::pack_bf16x2(y.x * f, y.y * f), rsm::pack_bf16x2(y.z * f, y.w * f));
          } else {
            *reinterpret_cast<float4*>(p.part + (slot * kRows + r) * DIM + col) = y;
            if (col == 0)
              *reinterpret_cast<float2*>(p.part + 2 * static_cast<int64_t>(p.ctas) * kRows * DIM + (slot * kRows + r) * 2) = make_float2(top, sum);
          }
        }
        if constexpr (TMA) rsm::fence_proxy_async_smem();  // the loads to come write here too
        __syncthreads();
      };
      pass(std::integral_constant<int, 0>{});
      if constexpr (kRows > 16) pass(std::integral_constant<int, 1>{});
      if (over) break;
      math.commit(p, at, lane, smem);
      math.reset();
      from = 0;
    } else {
      ++at.tile;
    }
    if (++stage == S) stage = 0, phase ^= 1u;
  }
  if constexpr (!TMA) cp_async_wait<0>();
}

// Units in pieces, `parts` CTAs each, which share the rows out.  By unit, where there
// are no more of them than CTAs of the first kernel; else by such a CTA: it has at most one
// unit's first piece.  A warp joins a row of up to 32 pieces by itself, a CTA one of more.
template <typename Math, int DIM>
__global__ void __launch_bounds__(kAttnJoinThreads) attn_join_kernel(const __grid_constant__ AttnParams p, int parts, int by_unit) {
  using IT = typename Math::IT;
  constexpr int kRows = Math::kRows, kLanes = DIM / 4, kGroups = kAttnJoinThreads / kLanes;  // kLanes threads take a row's columns, four each
  constexpr int kU = 8;  // rows asked for at a time
  __shared__ float4 acc_s[kGroups][kLanes];
  __shared__ float red_s[kAttnJoinThreads / 32];
  extern __shared__ float weight_s[];  // a piece's
  const int index = blockIdx.x / parts, part = blockIdx.x - index * parts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units = p.G * p.row_tiles;
  const Deal<kAttnJoinThreads> d(p, false);
  const AttnDeal deal(d.total, p.ctas);
  int64_t first = 0;
  int b = 0, u = 0, tiles = 0;
  if (by_unit) {
    b = index / units;
    u = index - b * units;
    tiles = tiles_of(p, request_tokens(p.pages, b, p.window, nullptr, false));
    first = d.before(p, b) + u * counts(p, tiles);
  } else if (index < deal.ctas) {
    const Place place = d.find(p, deal.begin(index + 1) - 1);
    b = place.b;
    tiles = tiles_of(p, request_tokens(p.pages, b, p.window, nullptr, false));
    u = static_cast<int>(quotient(deal.begin(index + 1) - 1 - place.first, counts(p, tiles)));
    first = place.first + u * counts(p, tiles);
    if (first < deal.begin(index)) tiles = 0;  // it began before
  }
  int c0 = 0, pieces = 1;
  if (tiles > 0) {
    c0 = static_cast<int>(deal.owner(first));
    pieces = static_cast<int>(deal.owner(first + tiles - 1)) - c0 + 1;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // by every CTA: the call is over when this kernel is
  if (pieces == 1) return;
  const int g = u / p.row_tiles, rt = u - g * p.row_tiles, rows = min(kRows, p.per * p.window - rt * kRows);
  const float2* ml = reinterpret_cast<const float2*>(p.part + 2 * static_cast<int64_t>(p.ctas) * kRows * DIM);
  auto slot = [&](int i) { return 2 * static_cast<int64_t>(c0 + i) + (i == 0 ? 1 : 0); };
  const int group = threadIdx.x / kLanes, col = threadIdx.x % kLanes;
  const auto finish = [&](int r) {
    const int row = rt * kRows + r, t = row / p.per;
    return static_cast<IT*>(p.out) + ((static_cast<int64_t>(b) * p.window + t) * p.H + g * p.per + row - t * p.per) * p.dim;
  };
  if (pieces <= 32) {
    constexpr int kWarps = kAttnJoinThreads / 32, kCols = DIM / 32;
    for (int r = part * kWarps + warp; r < rows; r += parts * kWarps) {
      const float2 own = lane < pieces ? ml[slot(lane) * kRows + r] : make_float2(kAttnLowest, 0.0f);
      constexpr int kFirst = 4;  // pieces that are on their way before their weights are known
      float first_v[kFirst][kCols];
#pragma unroll
      for (int i = 0; i < kFirst; ++i)
#pragma unroll
        for (int k = 0; k < kCols; ++k) first_v[i][k] = i < pieces ? p.part[(slot(i) * kRows + r) * DIM + lane + 32 * k] : 0.0f;
      float top = own.x;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const float f = exp2_fast(own.x - top);
      float sum = own.y * f, y[kCols];
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
#pragma unroll
      for (int k = 0; k < kCols; ++k) y[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < kFirst; ++i) {
        const float w = i < pieces ? __shfl_sync(0xFFFFFFFFu, f, i) : 0.0f;
#pragma unroll
        for (int k = 0; k < kCols; ++k) y[k] = fmaf(first_v[i][k], w, y[k]);
      }
#pragma unroll 4
      for (int i = kFirst; i < pieces; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, i);
        const float* from = p.part + (slot(i) * kRows + r) * DIM + lane;
#pragma unroll
        for (int k = 0; k < kCols; ++k) y[k] = fmaf(from[32 * k], w, y[k]);
      }
#pragma unroll
      for (int k = 0; k < kCols; ++k)
        if (lane + 32 * k < p.dim) put(finish(r) + lane + 32 * k, sum == 0.0f ? 0.0f : y[k] / sum);
    }
    return;
  }
  auto all = [&](float v, auto op) {  // over the CTA
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    __syncthreads();
    if (lane == 0) red_s[warp] = v;
    __syncthreads();
    v = red_s[0];
#pragma unroll
    for (int w = 1; w < kAttnJoinThreads / 32; ++w) v = op(v, red_s[w]);
    return v;
  };
  for (int r = part; r < rows; r += parts) {
    // a thread two pieces at most (p.ctas <= 2 kAttnJoinThreads)
    float2 s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = threadIdx.x + k * kAttnJoinThreads;
      s[k] = i < pieces ? ml[slot(i) * kRows + r] : make_float2(kAttnLowest, 0.0f);
    }
    const float top = all(fmaxf(s[0].x, s[1].x), [](float x, float y) { return fmaxf(x, y); });
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = threadIdx.x + k * kAttnJoinThreads;
      const float f = exp2_fast(s[k].x - top);
      if (i < pieces) weight_s[i] = f;
      sum = fmaf(s[k].y, f, sum);
    }
    sum = all(sum, [](float x, float y) { return x + y; });
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = group; i < pieces; i += kGroups * kU) {
      float4 v[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k)
        if (i + k * kGroups < pieces) v[k] = reinterpret_cast<const float4*>(p.part + (slot(i + k * kGroups) * kRows + r) * DIM)[col];
#pragma unroll
      for (int k = 0; k < kU; ++k)
        if (i + k * kGroups < pieces) {
          const float f = weight_s[i + k * kGroups];
          y.x = fmaf(v[k].x, f, y.x), y.y = fmaf(v[k].y, f, y.y), y.z = fmaf(v[k].z, f, y.z), y.w = fmaf(v[k].w, f, y.w);
        }
    }
    acc_s[group][col] = y;
    __syncthreads();
    IT* const out = finish(r);
    for (int c = threadIdx.x; c < p.dim; c += kAttnJoinThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kGroups; ++w) v += reinterpret_cast<const float*>(acc_s[w])[c];
      put(out + c, sum == 0.0f ? 0.0f : v / sum);
    }
    __syncthreads();
  }
}

}  // namespace hybrid
