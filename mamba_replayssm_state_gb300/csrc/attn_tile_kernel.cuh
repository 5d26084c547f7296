// attn_tile_kernel.cuh -- attention of new tokens over pages, on the tensor cores.
//
// For a key head the queries of its `per` heads and of all new tokens are the rows
// of one matrix Q: S = Q K^T, P = 2^(scale S - m), O = P V, with a running maximum m
// and sum l a row, so the cache is gone through once.
//
// Memory bounds it: 8 rows of 128 columns make 8 multiplications of a byte of keys and
// values.  So the cache is what is organised.  A CTA has four warps, and
// each streams 16 tokens at a time through shared memory of its own, S stages ahead
// (boxes of 16 rows by TMA where pages are whole groups of 16 tokens, else cp.async):
// no barrier of the CTA holds a load back, and warps are joined only at the end of
// a request's part.  The running maximum is one only to within 2^8: it is taken, and sums and
// outputs scaled anew, where a score passes it by more, which takes a few steps of a
// request instead of all.
//
// The products are m16n8k16 (bf16) and m16n8k8 (tf32) instructions on registers: with a
// few rows a 128-row tcgen05 tile would be mostly empty.  bf16 takes the products the other
// way round, S^T = K Q^T and O^T = V^T P^T, so that rows come in eights, and turns P^T
// between them with movmatrix.
//
// The work of a call is its (request, key head, group of rows) units' tiles of 64 tokens,
// one after the other, and with each unit kAttnUnit tiles more for what its end takes; every CTA
// takes the same number of them, wherever they begin and end, so that lengths (which only
// the device knows) may differ as they like.  A unit that a CTA has to itself is finished
// by it; pieces of others go to the workspace, two a CTA at most, and attn_join_kernel puts
// them together.
#pragma once
#include <type_traits>

#include "attn_plain_kernel.cuh"
#include "rsm_ptx.cuh"

namespace hybrid {

__device__ __forceinline__ int tiles_of(int64_t len) { return static_cast<int>((len + kAttnTile - 1) / kAttnTile); }

// What a unit of that many tiles counts.
__device__ __forceinline__ int64_t counts(int tiles) { return tiles == 0 ? 0 : tiles + kAttnUnit; }

// How a call's tiles are dealt out: the same in both kernels.
struct AttnDeal {
  int64_t total;  // tiles, the units' ends among them
  int64_t ctas;   // that have any
  __device__ __forceinline__ int64_t begin(int64_t c) const { return c * total / ctas; }
  __device__ __forceinline__ int64_t owner(int64_t tile) const { return ((tile + 1) * ctas - 1) / total; }
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
    return counts(tiles_of(request_tokens(p.pages, b, p.window, p.status, report))) * (p.G * p.row_tiles);
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

// The box of 16 tokens and 128 bytes at (column, head, row, page).
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, int column, int head, int row, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(column), "r"(head), "r"(row), "r"(page), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Lane 4 i + j's values (i, 2 j) and (i, 2 j + 1) of an 8 x 8 matrix become (2 j, i) and (2 j + 1, i).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t to_tf32(float v) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
  return r;
}
// v = hi + lo to 22 bits
__device__ __forceinline__ void split_tf32(float v, uint32_t& hi, uint32_t& lo) {
  hi = to_tf32(v);
  lo = to_tf32(v - __uint_as_float(hi));
}
// The same for keys and values, which may be infinite: then lo is 0, and so is `other`, elsewhere hi,
// which is what the other operand's lo is multiplied with (its sign would make the sum NaN).
__device__ __forceinline__ void split_tf32(float v, uint32_t& hi, uint32_t& lo, uint32_t& other) {
  split_tf32(v, hi, lo);
  const bool finite = (hi & 0x7F800000u) != 0x7F800000u;
  lo = finite ? lo : 0u;
  other = finite ? hi : 0u;
}
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Where a 16-byte chunk of a token's row lies: boxes of 16 rows of 128 bytes, the chunks
// of a row in an order of its own (the boxes' 128-byte swizzle; keys of fp32 another), so
// that what the lanes of an instruction read lies in different banks.
template <typename IT>
__device__ __forceinline__ int key_chunk(int token, int chunk) {
  const int order = sizeof(IT) == 2 ? token & 7 : (token & 1) << 2 | (token >> 1 & 3);
  return (chunk >> 3) * (kAttnStep * 128) + token * 128 + ((chunk & 7) ^ order) * 16;
}
__device__ __forceinline__ int value_chunk(int token, int chunk) {
  return (chunk >> 3) * (kAttnStep * 128) + token * 128 + ((chunk & 7) ^ (token & 7)) * 16;
}

constexpr float kAttnSlack = 8.0f;
constexpr float kAttnLowest = -3.402823466e38f;  // a maximum of nothing: no difference with it is NaN
constexpr uint64_t kAttnTimeoutNs = 2000000000ull;  // of a wait that takes microseconds

template <typename IT, int DIM>
struct AttnShape {
  static constexpr int kChunks = DIM * static_cast<int>(sizeof(IT)) / 16;  // of a row
  static constexpr int kHalf = kAttnStep * DIM * static_cast<int>(sizeof(IT));  // a warp's keys of a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = attn_stages(sizeof(IT), DIM);
  static constexpr int kQuery = sizeof(IT) == 4 ? 2 * 16 * DIM * 4 : 0;    // fp32: Q's parts as the products take them
};

// A place among the tiles, as one walks along them: request, key head, rows, tile.
struct AttnCursor {
  int b, g, rt, tile, tiles, len;
  __device__ __forceinline__ void at_request(const AttnParams& p) {
    len = static_cast<int>(request_tokens(p.pages, b, p.window, nullptr, false));
    tiles = tiles_of(len);
  }
  __device__ __forceinline__ void next_unit(const AttnParams& p) {
    tile = 0;
    if (++rt < p.row_tiles) return;
    rt = 0;
    if (++g < p.G) return;
    g = 0;
    do {
      if (++b >= p.pages.requests) return;
      at_request(p);
    } while (len == 0);
  }
  __device__ __forceinline__ void next(const AttnParams& p) {
    if (++tile == tiles) next_unit(p);
  }
  // Row r of the unit: its queries (null: there is none) and the last token that it sees.
  template <typename IT, int DIM>
  __device__ __forceinline__ const IT* query(const AttnParams& p, int rows, int row, int& last) const {
    const int r = rt * rows + row, t = r / p.per;
    last = len - p.window + t;
    if (r >= p.per * p.window) return nullptr;
    return static_cast<const IT*>(p.q) + b * p.q_bs + t * p.q_ts + static_cast<int64_t>(g * p.per + r - t * p.per) * DIM;
  }
};

// What a warp has seen of a step: 16 tokens at token0, those of the bits `seen`.
struct AttnStep {
  uint32_t keys, values;  // shared memory
  char* held;             // the values, to change them
  uint32_t seen;
  int token0;
  bool differ;            // rows differ in what they see
  int first_new;          // of the 16, the first that is not seen by all rows
};

// New tokens' values that are not finite go to the rows that see them, by add(token), and not
// into the product, where a weight of zero would not keep them from the others.
template <typename IT, int DIM, typename F>
__device__ __forceinline__ void odd_values(const AttnStep& a, int lane, F add) {
  constexpr int kChunks = AttnShape<IT, DIM>::kChunks;
  bool odd = false;
  for (int c = lane; c < kAttnStep * kChunks; c += 32) {
    if ((c >> 3) % kAttnStep < a.first_new) continue;
    const uint4 v = rsm::lds128(a.values + c * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      odd |= (w[k] & 0x7F800000u) == 0x7F800000u;
      if (sizeof(IT) == 2) odd |= (w[k] & 0x7F80u) == 0x7F80u;
    }
  }
  if (!__any_sync(0xFFFFFFFFu, odd)) return;
  for (int j = a.first_new; j < kAttnStep; ++j)
    if (a.seen >> j & 1u) add(j);
  __syncwarp();
  for (int c = lane; c < kAttnStep * kChunks; c += 32) {
    if ((c >> 3) % kAttnStep < a.first_new) continue;
    IT* v = reinterpret_cast<IT*>(a.held + c * 16);
#pragma unroll
    for (int k = 0; k < 16 / static_cast<int>(sizeof(IT)); ++k)
      if (!isfinite(get(v + k))) v[k] = IT(0);
  }
  rsm::fence_proxy_async_smem();
  __syncwarp();
}

template <typename IT>
__device__ __forceinline__ float held_value(const AttnStep& a, int token, int column) {
  const int c = column * static_cast<int>(sizeof(IT));
  return get(reinterpret_cast<const IT*>(a.held + value_chunk(token, c / 16) + c % 16));
}

// A warp's part of a unit, bf16: 8 N rows.  Lane (quad, four) holds of S^T tokens quad and quad
// + 8, rows 8 n + 2 four + {0, 1}; of O^T columns 16 i + quad and + 8, the same rows.
template <int DIM, int N>
struct AttnBf16 {
  using IT = uint16_t;
  static constexpr int kRows = 8 * N, kSteps = DIM / 16;
  static constexpr int kChains = N == 1 ? 4 : N == 2 ? 2 : 1;  // sums that do not wait for one another
  uint32_t q[N][kSteps][2];
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
  __device__ __forceinline__ void queries(const AttnParams& p, const AttnCursor& at, int lane, char*) {
    const int quad = lane >> 2, four = lane & 3;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      int last;
#pragma unroll
      for (int e = 0; e < 2; ++e) (void)at.query<IT, DIM>(p, kRows, 8 * n + 2 * four + e, limit[n][e]);
      const IT* from = at.query<IT, DIM>(p, kRows, 8 * n + quad, last);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t v = 0;
          if (from != nullptr) {
            const IT* s = from + 16 * ks + 8 * e + 2 * four;
            v = p.q_pairs ? *reinterpret_cast<const uint32_t*>(s) : static_cast<uint32_t>(s[0]) | static_cast<uint32_t>(s[1]) << 16;
          }
          q[n][ks][e] = v;
        }
    }
  }
  __device__ __forceinline__ void step(const AttnParams& p, const AttnStep& a, int lane, const char*) {
    const int quad = lane >> 2, four = lane & 3;
    float part[kChains][N][4], s[N][4];
#pragma unroll
    for (int c = 0; c < kChains; ++c)
#pragma unroll
      for (int n = 0; n < N; ++n) part[c][n][0] = part[c][n][1] = part[c][n][2] = part[c][n][3] = 0.0f;
    {
      const int token = lane & 15, odd = lane >> 4;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        uint32_t ka[4];
        ldmatrix4(ka, a.keys + key_chunk<IT>(token, 2 * ks + odd));
#pragma unroll
        for (int n = 0; n < N; ++n) mma_bf16(part[ks % kChains][n], ka, q[n][ks][0], q[n][ks][1]);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = part[0][n][e];
#pragma unroll
        for (int c = 1; c < kChains; ++c) s[n][e] += part[c][n][e];
      }
    if (a.differ || a.seen != (1u << kAttnStep) - 1u) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = quad + 8 * (e >> 1);
          if (!(a.seen >> j & 1u) || a.token0 + j > limit[n][e & 1]) s[n][e] = p.hidden;
        }
    }
    bool above = false;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) above |= fmaf(s[n][e], p.scale_log2, -m[n][e & 1]) > kAttnSlack;
    if (__any_sync(0xFFFFFFFFu, above)) {  // some row's maximum moves
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(s[n][e] * p.scale_log2, s[n][e + 2] * p.scale_log2);
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
          const float next = fmaxf(m[n][e], top), keep = exp2_fast(m[n][e] - next);
          m[n][e] = next;
          l[n][e] *= keep;
#pragma unroll
          for (int i = 0; i < kSteps; ++i) o[i][n][e] *= keep, o[i][n][e + 2] *= keep;
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = exp2_fast(fmaf(s[n][e], p.scale_log2, -m[n][e & 1]));
        l[n][e & 1] += s[n][e];
      }
    if (a.differ && p.window > 1)
      odd_values<IT, DIM>(a, lane, [&](int j) {
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
                const float v = held_value<IT>(a, j, 16 * i + 8 * h + quad);
                if (!isfinite(v)) o[i][n][2 * h + e] += w * v;
              }
          }
      });
    uint32_t pb[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) pb[n][h] = transpose8(rsm::pack_bf16x2(s[n][2 * h], s[n][2 * h + 1]));
    const int token = (lane >> 4) * 8 + (lane & 7), odd = lane >> 3 & 1;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      uint32_t va[4];
      ldmatrix4_trans(va, a.values + value_chunk(token, 2 * i + odd));
#pragma unroll
      for (int n = 0; n < N; ++n) mma_bf16(o[i][n], va, pb[n][0], pb[n][1]);
    }
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

// The same for fp32, 16 rows: each product is three of tf32 (hi hi, hi lo, lo hi).  Lane
// (quad, four) holds of S rows quad and quad + 8, tokens 8 n + 2 four + {0, 1}; of O the same rows.
template <int DIM>
struct AttnF32 {
  using IT = float;
  static constexpr int kRows = 16, kN = DIM / 8;
  int limit[2];
  float o[kN][4], m[2], l[2];

  // The column of o[n][e], e = 0 or 1: values are taken four columns at a time.
  __device__ __forceinline__ static int column(int four, int n, int e) { return 32 * (n / 4) + 4 * (2 * four + e) + (n & 3); }

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < kN; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    m[0] = m[1] = kAttnLowest;
    l[0] = l[1] = 0.0f;
  }
  // Q to shared memory: for each 8 columns the four registers of the left operand of every lane,
  // hi and then lo; columns 16 kk + 4 f + {0, 1} and {2, 3} are those of four = f in two products.
  __device__ __forceinline__ void queries(const AttnParams& p, const AttnCursor& at, int lane, char* smem) {
#pragma unroll
    for (int h = 0; h < 2; ++h) (void)at.query<IT, DIM>(p, kRows, 8 * h + (lane >> 2), limit[h]);
    __syncthreads();  // the last unit's are read
    for (int i = threadIdx.x; i < 32 * (DIM / 8); i += kAttnThreads) {
      const int ks = i / 32, ln = i & 31, qd = ln >> 2, fr = ln & 3;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int last;
        const IT* q = at.query<IT, DIM>(p, kRows, 8 * h + qd, last);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          split_tf32(q == nullptr ? 0.0f : q[16 * (ks / 2) + 4 * fr + 2 * (ks & 1) + e], hi[2 * e + h], lo[2 * e + h]);
      }
      uint4* to = reinterpret_cast<uint4*>(smem) + 2 * 32 * ks + ln;
      to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      to[32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    __syncthreads();
  }
  __device__ __forceinline__ void step(const AttnParams& p, const AttnStep& a, int lane, const char* smem) {
    const int quad = lane >> 2, four = lane & 3;
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
    const uint32_t qs = rsm::smem_addr(smem) + lane * 16;
#pragma unroll 4
    for (int kk = 0; kk < DIM / 16; ++kk) {
      uint32_t hi[2][4], lo[2][4], fin[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint4 v = rsm::lds128(a.keys + key_chunk<IT>(8 * n + quad, 4 * kk + four));
        split_tf32(__uint_as_float(v.x), hi[n][0], lo[n][0], fin[n][0]);
        split_tf32(__uint_as_float(v.y), hi[n][1], lo[n][1], fin[n][1]);
        split_tf32(__uint_as_float(v.z), hi[n][2], lo[n][2], fin[n][2]);
        split_tf32(__uint_as_float(v.w), hi[n][3], lo[n][3], fin[n][3]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 h4 = rsm::lds128(qs + (2 * kk + e) * 1024), l4 = rsm::lds128(qs + (2 * kk + e) * 1024 + 512);
        const uint32_t ah[4] = {h4.x, h4.y, h4.z, h4.w}, al[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          mma_tf32(s[n], al, fin[n][2 * e], fin[n][2 * e + 1]);
          mma_tf32(s[n], ah, lo[n][2 * e], lo[n][2 * e + 1]);
          mma_tf32(s[n], ah, hi[n][2 * e], hi[n][2 * e + 1]);
        }
      }
    }
    if (a.differ || a.seen != (1u << kAttnStep) - 1u) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * n + 2 * four + (e & 1);
          if (!(a.seen >> j & 1u) || a.token0 + j > limit[e >> 1]) s[n][e] = p.hidden;
        }
    }
    bool above = false;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) above |= fmaf(s[n][e], p.scale_log2, -m[e >> 1]) > kAttnSlack;
    if (__any_sync(0xFFFFFFFFu, above)) {  // some row's maximum moves
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = fmaxf(fmaxf(s[0][2 * h] * p.scale_log2, s[0][2 * h + 1] * p.scale_log2),
                          fmaxf(s[1][2 * h] * p.scale_log2, s[1][2 * h + 1] * p.scale_log2));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const float next = fmaxf(m[h], top), keep = exp2_fast(m[h] - next);
        m[h] = next;
        l[h] *= keep;
#pragma unroll
        for (int n = 0; n < kN; ++n) o[n][2 * h] *= keep, o[n][2 * h + 1] *= keep;
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = exp2_fast(fmaf(s[n][e], p.scale_log2, -m[e >> 1]));
        l[e >> 1] += s[n][e];
      }
    if (a.differ && p.window > 1)
      odd_values<IT, DIM>(a, lane, [&](int j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float even = j & 8 ? s[1][2 * h] : s[0][2 * h], other = j & 8 ? s[1][2 * h + 1] : s[0][2 * h + 1];
          const float w = __shfl_sync(0xFFFFFFFFu, j & 1 ? other : even, (lane & ~3) + (j & 7) / 2);
          if (a.token0 + j > limit[h]) continue;
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float v = held_value<IT>(a, j, column(four, n, e));
              if (!isfinite(v)) o[n][2 * h + e] += w * v;
            }
        }
      });
    // tokens 2 f and 2 f + 1 of eight are those of four = f, as S's columns are
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      uint32_t ph[4], pl[4];
      split_tf32(s[kt][0], ph[0], pl[0]);
      split_tf32(s[kt][2], ph[1], pl[1]);
      split_tf32(s[kt][1], ph[2], pl[2]);
      split_tf32(s[kt][3], ph[3], pl[3]);
      const int t0 = 8 * kt + 2 * four, t1 = t0 + 1;
#pragma unroll
      for (int n = 0; n < kN; n += 4) {
        const uint4 x = rsm::lds128(a.values + value_chunk(t0, 2 * n + quad)), y = rsm::lds128(a.values + value_chunk(t1, 2 * n + quad));
        const uint32_t va[4] = {x.x, x.y, x.z, x.w}, vb[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t h0, l0, f0, h1, l1, f1;
          split_tf32(__uint_as_float(va[k]), h0, l0, f0);
          split_tf32(__uint_as_float(vb[k]), h1, l1, f1);
          mma_tf32(o[n + k], pl, f0, f1);
          mma_tf32(o[n + k], ph, l0, l1);
          mma_tf32(o[n + k], ph, h0, h1);
        }
      }
    }
  }
  __device__ __forceinline__ void stats(float* ms, float* ls, int lane) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = l[h];
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      if ((lane & 3) == 0) ms[8 * h + (lane >> 2)] = m[h], ls[8 * h + (lane >> 2)] = sum;
    }
  }
  __device__ __forceinline__ static int place(int row, int column) { return row * DIM + (column ^ (row & 3) << 3); }
  template <int PASS>
  __device__ __forceinline__ void outputs(float* own, int lane) const {
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) own[place(8 * (e >> 1) + (lane >> 2), column(lane & 3, n, e & 1))] = o[n][e];
  }
};

// BOXES: loads by TMA; the pages are whole groups of 16 tokens.
template <typename Math, int DIM, bool BOXES>
__global__ void __launch_bounds__(kAttnThreads, attn_ctas_per_sm(sizeof(typename Math::IT), DIM))
    attn_tile_kernel(const __grid_constant__ AttnTileParams tp) {
  using IT = typename Math::IT;
  using Shape = AttnShape<IT, DIM>;
  constexpr int kWarps = kAttnThreads / 32, kRows = Math::kRows, S = Shape::kStages, kChunks = Shape::kChunks;
  constexpr uint32_t kAll = (1u << kAttnStep) - 1u;
  extern __shared__ __align__(1024) char smem[];
  __shared__ float m_s[kWarps][kRows], l_s[kWarps][kRows];
  __shared__ uint32_t seen_s[kWarps][S];
  __shared__ __align__(8) uint64_t full_s[kWarps][S];  // BOXES: a stage's loads
  const AttnParams& p = tp.p;
  const rsm_pages& pg = p.pages;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (BOXES) {
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
        const int64_t n = static_cast<int64_t>(p.window) * p.H * DIM;
        IT* out = static_cast<IT*>(p.out) + b * n;
        for (int64_t i = threadIdx.x; i < n; i += kAttnThreads) out[i] = IT(0);
      }
  };
  const Deal<kAttnThreads> requests(p, blockIdx.x == 0);
  const AttnDeal deal{requests.total, min(static_cast<int64_t>(gridDim.x), requests.total)};
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
    const int unit = static_cast<int>(into / counts(at.tiles)), tile = static_cast<int>(into - unit * counts(at.tiles));
    at.g = unit / p.row_tiles;
    at.rt = unit - at.g * p.row_tiles;
    at.tile = tile;
    if (tile >= at.tiles) {  // the share begins in what a unit's end counts
      room -= counts(at.tiles) - tile;
      if (room <= 0) return skipped();
      at.next_unit(p);
    }
  }
  AttnCursor ask = at;
  int64_t ask_room = room;

  // ---- loads: a warp's 16 tokens of a tile ----
  const uint32_t ring = rsm::smem_addr(smem) + Shape::kQuery + warp * (S * Shape::kStage);
  const uint32_t full = rsm::smem_addr(&full_s[warp][0]);
  const bool one_page = BOXES || pg.page_size % kAttnStep == 0;  // the 16 tokens lie in one page
  auto page_at = [&](int64_t token) {
    if (token >= ask.len) return -1;  // no token
    const int i = p.page_shift >= 0 ? static_cast<int>(token) >> p.page_shift : static_cast<int>(token) / pg.page_size;
    return __ldg(pg.page_table + ask.b * pg.table_stride + i);
  };
  // One page a step: a lane looks up that of the tile lane of each 32, all at once; else a lane a token, a step ahead.
  int looked = -1, pages = -1;
  auto look_up = [&](bool request) {
    if (one_page) {
      const int group = ask.tile >> 5;
      if (!request && group == looked) return;
      looked = group;
      pages = page_at((static_cast<int64_t>(group) * 32 + lane) * kAttnTile + warp * kAttnStep);
    } else {
      pages = page_at(static_cast<int64_t>(ask.tile) * kAttnTile + warp * kAttnStep + lane % kAttnStep);
    }
  };
  look_up(true);
  auto load = [&](int stage) {
    if (ask_room <= 0) {
      if constexpr (!BOXES) cp_async_commit();
      return;
    }
    const int g = ask.g, token0 = ask.tile * kAttnTile + warp * kAttnStep;
    const int page = one_page ? __shfl_sync(0xFFFFFFFFu, pages, ask.tile & 31) : pages;
    const bool good = page >= 0 && page < pg.num_pages;
    if (!good && token0 + (one_page ? 0 : lane % kAttnStep) < ask.len) flag(p.status, RSM_STATUS_BAD_PAGE);
    const uint32_t base = ring + stage * Shape::kStage;
    uint32_t seen;
    if constexpr (BOXES) {
      seen = good ? (1u << min(kAttnStep, ask.len - token0)) - 1u : 0u;
      if (lane == 0) {
        const uint32_t bar = full + stage * 8;
        if (good) {
          const int row = p.page_shift >= 0 ? token0 & (pg.page_size - 1) : token0 % pg.page_size;
          rsm::mbar_arrive_expect_tx(bar, Shape::kStage);
#pragma unroll
          for (int c = 0; c < DIM / 64; ++c) {
            box_load(base + c * (kAttnStep * 128), &tp.k_map, 64 * c, g, row, page, bar);
            box_load(base + Shape::kHalf + c * (kAttnStep * 128), &tp.v_map, 64 * c, g, row, page, bar);
          }
        } else {
          rsm::mbar_arrive(bar);
        }
      }
    } else {
      constexpr int kAt = 32 / kChunks;  // rows at a time
      const int row0 = lane / kChunks, chunk = lane % kChunks;
      const int token = token0 + (one_page ? 0 : lane % kAttnStep);
      const int row = p.page_shift >= 0 ? token & (pg.page_size - 1) : token % pg.page_size;
      seen = one_page ? (good ? (1u << min(kAttnStep, ask.len - token0)) - 1u : 0u) : __ballot_sync(0xFFFFFFFFu, good) & kAll;
#pragma unroll 4
      for (int i = 0; i < kAttnStep / kAt; ++i) {
        const int r = i * kAt + row0;
        int pr = page, rr = row + r;
        if (!one_page) pr = __shfl_sync(0xFFFFFFFFu, page, r), rr = __shfl_sync(0xFFFFFFFFu, row, r);
        const bool yes = seen >> r & 1u;
        const IT* kr = static_cast<const IT*>(pg.k) + (yes ? pr * pg.k_page_stride + rr * pg.k_row_stride + g * pg.k_head_stride : 0);
        const IT* vr = static_cast<const IT*>(pg.v) + (yes ? pr * pg.v_page_stride + rr * pg.v_row_stride + g * pg.v_head_stride : 0);
        cp_async_16_or_zero(base + key_chunk<IT>(r, chunk), reinterpret_cast<const char*>(kr) + chunk * 16, yes);
        cp_async_16_or_zero(base + Shape::kHalf + value_chunk(r, chunk), reinterpret_cast<const char*>(vr) + chunk * 16, yes);
      }
      cp_async_commit();
    }
    if (lane == 0) seen_s[warp][stage] = seen;
    ask_room -= ask.tile + 1 == ask.tiles ? 1 + kAttnUnit : 1;
    if (ask_room > 0) {
      const int b = ask.b;
      ask.next(p);
      look_up(ask.b != b);
    }
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) load(s);

  Math math;
  math.queries(p, at, lane, smem);
  math.reset();
  skipped();
  int from = at.tile;  // the piece's first tile
  uint32_t phase = 0;
  for (int stage = 0;;) {
    if constexpr (BOXES) {
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
      a.token0 = at.tile * kAttnTile + warp * kAttnStep;
      a.differ = a.token0 + kAttnStep - 1 > at.len - p.window;
      a.first_new = max(at.len - p.window + 1 - a.token0, 0);
      if constexpr (BOXES) {  // rows behind the last token came with the box
        if (a.seen != kAll) {
          for (int c = lane; c < kAttnStep * kChunks; c += 32)
            if (!(a.seen >> ((c >> 3) % kAttnStep) & 1u)) *reinterpret_cast<uint4*>(a.held + c * 16) = make_uint4(0, 0, 0, 0);
          rsm::fence_proxy_async_smem();
          __syncwarp();
        }
      }
      math.step(p, a, lane, smem);
    }

    // ---- the end of a unit, or of this CTA's part of it ----
    const bool last_tile = at.tile + 1 == at.tiles;
    room -= last_tile ? 1 + kAttnUnit : 1;
    const bool over = room <= 0;
    if (last_tile || over) {
      const AttnCursor was = at;
      const bool whole = from == 0 && last_tile;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (from == 0 ? 1 : 0);
      math.stats(m_s[warp], l_s[warp], lane);
      // the next unit's queries are on their way meanwhile (fp32: see below)
      if (!over) {
        at.next(p);
        if constexpr (Shape::kQuery == 0) math.queries(p, at, lane, smem);
      }
      // the warps' outputs pass through the stages just read, 16 rows at a time
      char* const pass_at = smem + Shape::kQuery + stage * Shape::kStage;
      auto pass = [&](auto index) {
        constexpr int kPass = decltype(index)::value, kHere = kRows - 16 * kPass < 16 ? kRows - 16 * kPass : 16;
        math.template outputs<kPass>(reinterpret_cast<float*>(pass_at + warp * (S * Shape::kStage)), lane);
        __syncthreads();
        for (int c = threadIdx.x; c < kHere * DIM / 4; c += kAttnThreads) {
          const int row = c / (DIM / 4), col = (c - row * (DIM / 4)) * 4, r = 16 * kPass + row, all = was.rt * kRows + r;
          if (all >= p.per * p.window) continue;
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
            IT* out = static_cast<IT*>(p.out) + ((static_cast<int64_t>(was.b) * p.window + t) * p.H + was.g * p.per + all - t * p.per) * DIM + col;
            if constexpr (sizeof(IT) == 4)
              *reinterpret_cast<float4*>(out) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
            else
              *reinterpret_cast<uint2*>(out) = make_uint2(rsm::pack_bf16x2(y.x * f, y.y * f), rsm::pack_bf16x2(y.z * f, y.w * f));
          } else {
            *reinterpret_cast<float4*>(p.part + (slot * kRows + r) * DIM + col) = y;
            if (col == 0)
              *reinterpret_cast<float2*>(p.part + 2 * static_cast<int64_t>(p.ctas) * kRows * DIM + (slot * kRows + r) * 2) = make_float2(top, sum);
          }
        }
        if constexpr (BOXES) rsm::fence_proxy_async_smem();  // the boxes to come write here too
        __syncthreads();
      };
      pass(std::integral_constant<int, 0>{});
      if constexpr (kRows > 16) pass(std::integral_constant<int, 1>{});
      if (over) break;
      if constexpr (Shape::kQuery != 0) math.queries(p, at, lane, smem);
      math.reset();
      from = 0;
    } else {
      ++at.tile;
    }
    if (++stage == S) stage = 0, phase ^= 1u;
  }
  if constexpr (!BOXES) cp_async_wait<0>();
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
  const AttnDeal deal{d.total, min(static_cast<int64_t>(p.ctas), d.total)};
  int64_t first = 0;
  int b = 0, u = 0, tiles = 0;
  if (by_unit) {
    b = index / units;
    u = index - b * units;
    tiles = tiles_of(request_tokens(p.pages, b, p.window, nullptr, false));
    first = d.before(p, b) + u * counts(tiles);
  } else if (index < deal.ctas) {
    const Place place = d.find(p, deal.begin(index + 1) - 1);
    b = place.b;
    tiles = tiles_of(request_tokens(p.pages, b, p.window, nullptr, false));
    u = static_cast<int>((deal.begin(index + 1) - 1 - place.first) / counts(tiles));
    first = place.first + u * counts(tiles);
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
    return static_cast<IT*>(p.out) + ((static_cast<int64_t>(b) * p.window + t) * p.H + g * p.per + row - t * p.per) * DIM;
  };
  if (pieces <= 32) {
    constexpr int kWarps = kAttnJoinThreads / 32, kCols = DIM / 32;
    for (int r = part * kWarps + warp; r < rows; r += parts * kWarps) {
      const float2 own = lane < pieces ? ml[slot(lane) * kRows + r] : make_float2(kAttnLowest, 0.0f);
      float top = own.x;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const float f = exp2_fast(own.x - top);
      float sum = own.y * f, y[kCols];
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
#pragma unroll
      for (int k = 0; k < kCols; ++k) y[k] = 0.0f;
#pragma unroll 4
      for (int i = 0; i < pieces; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, i);
        const float* from = p.part + (slot(i) * kRows + r) * DIM + lane;
#pragma unroll
        for (int k = 0; k < kCols; ++k) y[k] = fmaf(from[32 * k], w, y[k]);
      }
#pragma unroll
      for (int k = 0; k < kCols; ++k) put(finish(r) + lane + 32 * k, sum == 0.0f ? 0.0f : y[k] / sum);
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
    for (int c = threadIdx.x; c < DIM; c += kAttnJoinThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kGroups; ++w) v += reinterpret_cast<const float*>(acc_s[w])[c];
      put(out + c, sum == 0.0f ? 0.0f : v / sum);
    }
    __syncthreads();
  }
}

}  // namespace hybrid
