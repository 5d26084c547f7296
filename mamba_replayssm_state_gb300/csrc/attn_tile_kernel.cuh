// attn_tile_kernel.cuh -- attention of new tokens over pages, on the tensor cores.
//
// For a key head the queries of its `per` heads and of all new tokens are the rows
// of one matrix Q: S = Q K^T, P = 2^(scale S - m), O = P V, with a running maximum m
// and sum l a row, so the cache is gone through once.
//
// Memory bounds it: 16 rows of 128 columns make 16 multiplications of a byte of keys and
// values.  So the cache is what is organised.  A CTA has four warps, and
// each streams 16 tokens at a time through shared memory of its own (cp.async, S
// stages ahead): no barrier holds a load back, and warps are joined only at the end of
// a request's part.  The products are m16n8k16 (bf16) or m16n8k8 (tf32) instructions on
// registers: with 16 or 32 rows a 128-row tcgen05 tile would be mostly empty.
//
// The work of a call is its (request, key head, 16 or 32 rows) units' tiles of 64 tokens,
// one after the other; every CTA takes the same number of them, wherever they begin and
// end, so that lengths (which only the device knows) may differ as they like.  A unit that
// a CTA has to itself is finished by it; pieces of others go to the workspace, two a CTA at
// most, and attn_join_kernel puts them together.
#pragma once
#include "attn_plain_kernel.cuh"
#include "rsm_ptx.cuh"

namespace hybrid {

// How the calls' tiles are dealt out: the same in both kernels.
struct AttnDeal {
  int64_t total;  // tiles
  int64_t ctas;   // that have any
  __device__ __forceinline__ int64_t begin(int64_t c) const { return c * total / ctas; }
  __device__ __forceinline__ int64_t owner(int64_t tile) const { return ((tile + 1) * ctas - 1) / total; }
};

__device__ __forceinline__ int tiles_of(int64_t len) { return static_cast<int>((len + kAttnTile - 1) / kAttnTile); }

// All tiles of the call; by the whole CTA.
template <int THREADS>
__device__ __forceinline__ int64_t deal_total(const AttnParams& p, bool report) {
  __shared__ int64_t sums[THREADS / 32];
  int64_t n = 0;
  for (int b = threadIdx.x; b < p.pages.requests; b += THREADS) n += tiles_of(request_tokens(p.pages, b, p.window, p.status, report));
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) n += sums[i];
  return n * (p.G * p.row_tiles);
}

struct Place {
  int b;          // request
  int64_t first;  // its first tile
};

// The request that has tile number `tile`; by the whole CTA.
template <int THREADS>
__device__ __forceinline__ Place deal_find(const AttnParams& p, int64_t tile) {
  __shared__ int64_t sums[THREADS / 32];
  __shared__ Place place;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t before = 0;
  for (int base = 0;; base += THREADS) {
    const int b = base + static_cast<int>(threadIdx.x);
    const int64_t own = b < p.pages.requests
                            ? static_cast<int64_t>(tiles_of(request_tokens(p.pages, b, p.window, nullptr, false))) * (p.G * p.row_tiles)
                            : 0;
    int64_t upto = own;
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
    if (tile < upto && tile >= upto - own) place = Place{b, upto - own};
    __syncthreads();
    if (tile < all || base + THREADS >= p.pages.requests) return place;
    before = all;
  }
}

__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool yes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(yes ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// A row's 16-byte chunks are stored in an order of its own, so that what the lanes of
// an instruction read lies in different banks.
template <typename IT>
__device__ __forceinline__ int key_order(int token) {
  return sizeof(IT) == 2 ? token & 7 : (token & 1) << 2 | (token >> 1 & 3);
}
__device__ __forceinline__ int value_order(int token) { return token & 7; }

template <typename IT, int DIM>
struct AttnShape {
  static constexpr int kChunks = DIM * static_cast<int>(sizeof(IT)) / 16;  // of a row
  static constexpr int kRow = DIM * static_cast<int>(sizeof(IT));
  static constexpr int kHalf = kAttnStep * kRow;                           // a warp's keys of a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = attn_stages(sizeof(IT), DIM);
  static constexpr int kQuery = sizeof(IT) == 4 ? 2 * 16 * DIM * 4 : 0;    // fp32: Q's parts as the products take them
};

// Where a unit's tiles are, as one walks along them.
struct AttnCursor {
  int b, u, tile, tiles, len;
  __device__ __forceinline__ void at_request(const AttnParams& p) {
    len = static_cast<int>(request_tokens(p.pages, b, p.window, nullptr, false));
    tiles = tiles_of(len);
  }
  __device__ __forceinline__ void next(const AttnParams& p, int units) {
    if (++tile < tiles) return;
    tile = 0;
    if (++u < units) return;
    u = 0;
    do {
      if (++b >= p.pages.requests) return;
      at_request(p);
    } while (len == 0);
  }
};

template <typename IT, int DIM, int M>
__global__ void __launch_bounds__(kAttnThreads, attn_ctas_per_sm(sizeof(IT), DIM)) attn_tile_kernel(const __grid_constant__ AttnParams p) {
  using Shape = AttnShape<IT, DIM>;
  constexpr bool kF32 = sizeof(IT) == 4;
  constexpr int kWarps = kAttnThreads / 32, kRows = 16 * M, kN = DIM / 8;  // kN: n-tiles of 8 columns
  constexpr int S = Shape::kStages, kChunks = Shape::kChunks;
  static_assert(!kF32 || M == 1);
  extern __shared__ __align__(128) char smem[];
  __shared__ float m_s[kWarps][kRows], l_s[kWarps][kRows];
  __shared__ uint32_t seen_s[kWarps][S];
  const rsm_pages& pg = p.pages;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane >> 2, four = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  for (int b = blockIdx.x; b < pg.requests; b += gridDim.x)  // rows of skipped requests
    if (request_tokens(pg, b, p.window, nullptr, false) == 0) {
      IT* out = static_cast<IT*>(p.out) + static_cast<int64_t>(b) * p.window * p.H * DIM;
      const int64_t n = static_cast<int64_t>(p.window) * p.H * DIM;
      for (int64_t i = threadIdx.x; i < n; i += kAttnThreads) out[i] = IT(0);
    }
  AttnDeal deal;
  deal.total = deal_total<kAttnThreads>(p, blockIdx.x == 0);
  deal.ctas = min(static_cast<int64_t>(gridDim.x), deal.total);
  if (blockIdx.x >= deal.ctas) return;
  const int64_t begin = deal.begin(blockIdx.x);
  const int count = static_cast<int>(deal.begin(blockIdx.x + 1) - begin);
  const Place place = deal_find<kAttnThreads>(p, begin);
  const int units = p.G * p.row_tiles;
  AttnCursor at;
  at.b = place.b;
  at.at_request(p);
  at.u = static_cast<int>((begin - place.first) / at.tiles);
  at.tile = static_cast<int>(begin - place.first - static_cast<int64_t>(at.u) * at.tiles);
  AttnCursor ask = at;

  // ---- loads: a warp's 16 tokens of a tile.  The page is looked up a step ahead. ----
  const uint32_t ring = rsm::smem_addr(smem) + Shape::kQuery + warp * (S * Shape::kStage);
  const bool one_page = pg.page_size % kAttnStep == 0;  // the 16 tokens lie in one page
  auto page_of = [&](const AttnCursor& c) {
    const int token = c.tile * kAttnTile + warp * kAttnStep + (one_page ? 0 : lane % kAttnStep);
    if (token >= c.len) return -1;  // no token
    const int i = p.page_shift >= 0 ? token >> p.page_shift : token / pg.page_size;
    return __ldg(pg.page_table + c.b * pg.table_stride + i);
  };
  int page = page_of(ask), left = count;
  auto load = [&](int stage) {
    if (left <= 0) {
      cp_async_commit();
      return;
    }
    const int g = ask.u / p.row_tiles, token0 = ask.tile * kAttnTile + warp * kAttnStep;
    const bool good = page >= 0 && page < pg.num_pages;
    if (!good && token0 + (one_page ? 0 : lane % kAttnStep) < ask.len) flag(p.status, RSM_STATUS_BAD_PAGE);
    const uint32_t base = ring + stage * Shape::kStage;
    constexpr int kPer = kChunks > 32 ? kChunks / 32 : 1;  // chunks of a row a lane
    constexpr int kAt = kChunks > 32 ? 1 : 32 / kChunks;   // rows at a time
    const int row0 = kChunks > 32 ? 0 : lane / kChunks, chunk0 = lane % kChunks;
    uint32_t seen;
    if (one_page) {
      const int row = p.page_shift >= 0 ? token0 & (pg.page_size - 1) : token0 % pg.page_size;
      const int64_t ko = good ? page * pg.k_page_stride + row * pg.k_row_stride + g * pg.k_head_stride : 0;
      const int64_t vo = good ? page * pg.v_page_stride + row * pg.v_row_stride + g * pg.v_head_stride : 0;
      const int n = good ? min(kAttnStep, ask.len - token0) : 0;
      seen = (1u << n) - 1u;
      const char* k = reinterpret_cast<const char*>(static_cast<const IT*>(pg.k) + ko);
      const char* v = reinterpret_cast<const char*>(static_cast<const IT*>(pg.v) + vo);
      const int64_t ks = pg.k_row_stride * static_cast<int64_t>(sizeof(IT)), vs = pg.v_row_stride * static_cast<int64_t>(sizeof(IT));
#pragma unroll
      for (int i = 0; i < kAttnStep / kAt; ++i) {
        const int r = i * kAt + row0;
        const bool yes = r < n;
        const char* kr = yes ? k + r * ks : static_cast<const char*>(pg.k);
        const char* vr = yes ? v + r * vs : static_cast<const char*>(pg.v);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int chunk = chunk0 + 32 * j;
          cp_async_16_or_zero(base + r * Shape::kRow + (chunk ^ key_order<IT>(r)) * 16, kr + chunk * 16, yes);
          cp_async_16_or_zero(base + Shape::kHalf + r * Shape::kRow + (chunk ^ value_order(r)) * 16, vr + chunk * 16, yes);
        }
      }
    } else {
      seen = __ballot_sync(0xFFFFFFFFu, good) & ((1u << kAttnStep) - 1u);
      const int token = token0 + lane % kAttnStep;
      const int row = p.page_shift >= 0 ? token & (pg.page_size - 1) : token % pg.page_size;
#pragma unroll 1
      for (int i = 0; i < kAttnStep / kAt; ++i) {
        const int r = i * kAt + row0;
        const int pr = __shfl_sync(0xFFFFFFFFu, page, r), rr = __shfl_sync(0xFFFFFFFFu, row, r);
        const bool yes = seen >> r & 1u;
        const char* kr = reinterpret_cast<const char*>(static_cast<const IT*>(pg.k) +
                                                       (yes ? pr * pg.k_page_stride + rr * pg.k_row_stride + g * pg.k_head_stride : 0));
        const char* vr = reinterpret_cast<const char*>(static_cast<const IT*>(pg.v) +
                                                       (yes ? pr * pg.v_page_stride + rr * pg.v_row_stride + g * pg.v_head_stride : 0));
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int chunk = chunk0 + 32 * j;
          cp_async_16_or_zero(base + r * Shape::kRow + (chunk ^ key_order<IT>(r)) * 16, kr + chunk * 16, yes);
          cp_async_16_or_zero(base + Shape::kHalf + r * Shape::kRow + (chunk ^ value_order(r)) * 16, vr + chunk * 16, yes);
        }
      }
    }
    if (lane == 0) seen_s[warp][stage] = seen;
    cp_async_commit();
    if (--left > 0) {
      ask.next(p, units);
      page = page_of(ask);
    }
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) load(s);

  // ---- a unit's queries ----
  const int rows_all = p.per * p.window;
  uint32_t qa[kF32 ? 1 : M][kF32 ? 1 : DIM / 16][4];
  int limit[M][2];  // the last token that a row sees
  auto query = [&](int row, int rt, int g, int& last) -> const IT* {
    const int r = rt * kRows + row;
    const int t = r / p.per;
    last = at.len - p.window + t;
    if (r >= rows_all) return nullptr;
    return static_cast<const IT*>(p.q) + at.b * p.q_bs + t * p.q_ts + static_cast<int64_t>(g * p.per + r - t * p.per) * DIM;
  };
  auto load_queries = [&]() {
    const int g = at.u / p.row_tiles, rt = at.u - g * p.row_tiles;
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const IT* q = query(16 * i + 8 * h + quad, rt, g, limit[i][h]);
        if constexpr (!kF32) {
#pragma unroll
          for (int ks = 0; ks < DIM / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t v = 0;
              if (q != nullptr) {
                const IT* s = q + 16 * ks + 8 * e + 2 * four;
                v = p.q_pairs ? *reinterpret_cast<const uint32_t*>(s) : static_cast<uint32_t>(s[0]) | static_cast<uint32_t>(s[1]) << 16;
              }
              qa[i][ks][2 * e + h] = v;
            }
        }
      }
    if constexpr (kF32) {
      // for each 8 columns the four registers of the left operand of every lane, hi and
      // then lo; column 16 kk + 4 f + {0, 1} and {2, 3} are those of four = f in two products
      __syncthreads();  // the last unit's are read
      for (int i = threadIdx.x; i < 32 * (DIM / 8); i += kAttnThreads) {
        const int ks = i / 32, ln = i & 31, qd = ln >> 2, fr = ln & 3;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int last;
          const IT* q = query(8 * h + qd, rt, g, last);
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
  };

  float o[M][kN][4], m[M][2], l[M][2];
  auto reset = [&]() {
#pragma unroll
    for (int i = 0; i < M; ++i) {
#pragma unroll
      for (int n = 0; n < kN; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.0f;
    }
  };
  // The column of o[.][n][e], e = 0 or 1: products of fp32 take values four columns at a time.
  auto column = [&](int n, int e) { return kF32 ? 32 * (n / 4) + 4 * (2 * four + e) + (n & 3) : 8 * n + 2 * four + e; };

  load_queries();
  reset();
  int from = at.tile;  // the piece's first tile
  for (int i = 0, stage = 0; i < count; ++i, stage = stage + 1 == S ? 0 : stage + 1) {
    cp_async_wait<S - 2>();
    __syncwarp();
    load(stage == 0 ? S - 1 : stage - 1);
    const uint32_t keys = ring + stage * Shape::kStage, values = keys + Shape::kHalf;
    const uint32_t seen = seen_s[warp][stage];
    const int token0 = at.tile * kAttnTile + warp * kAttnStep;
    const bool diagonal = token0 + kAttnStep - 1 > at.len - p.window;  // rows differ in what they see

    if (seen != 0) {
      float s[M][2][4];
#pragma unroll
      for (int i2 = 0; i2 < M; ++i2)
#pragma unroll
        for (int n = 0; n < 2; ++n) s[i2][n][0] = s[i2][n][1] = s[i2][n][2] = s[i2][n][3] = 0.0f;
      if constexpr (!kF32) {
        const int token = (lane >> 4) * 8 + (lane & 7), odd = lane >> 3 & 1;
#pragma unroll
        for (int ks = 0; ks < DIM / 16; ++ks) {
          uint32_t kb[4];
          ldmatrix4(kb, keys + token * Shape::kRow + ((2 * ks + odd) ^ key_order<IT>(token)) * 16);
#pragma unroll
          for (int i2 = 0; i2 < M; ++i2) {
            mma_bf16(s[i2][0], qa[i2][ks], kb[0], kb[1]);
            mma_bf16(s[i2][1], qa[i2][ks], kb[2], kb[3]);
          }
        }
      } else {
        const uint32_t qs = rsm::smem_addr(smem) + lane * 16;
#pragma unroll 4
        for (int kk = 0; kk < DIM / 16; ++kk) {
          uint32_t hi[2][4], lo[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int token = 8 * n + quad;
            const uint4 v = rsm::lds128(keys + token * Shape::kRow + ((4 * kk + four) ^ key_order<IT>(token)) * 16);
            split_tf32(__uint_as_float(v.x), hi[n][0], lo[n][0]);
            split_tf32(__uint_as_float(v.y), hi[n][1], lo[n][1]);
            split_tf32(__uint_as_float(v.z), hi[n][2], lo[n][2]);
            split_tf32(__uint_as_float(v.w), hi[n][3], lo[n][3]);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 h4 = rsm::lds128(qs + (2 * kk + e) * 1024), l4 = rsm::lds128(qs + (2 * kk + e) * 1024 + 512);
            const uint32_t ah[4] = {h4.x, h4.y, h4.z, h4.w}, al[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              mma_tf32(s[0][n], al, hi[n][2 * e], hi[n][2 * e + 1]);
              mma_tf32(s[0][n], ah, lo[n][2 * e], lo[n][2 * e + 1]);
              mma_tf32(s[0][n], ah, hi[n][2 * e], hi[n][2 * e + 1]);
            }
          }
        }
      }
      // ---- what is not seen, the running maximum, the weights ----
#pragma unroll
      for (int i2 = 0; i2 < M; ++i2)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i2][n][e] *= p.scale_log2;
      if (diagonal || seen != (1u << kAttnStep) - 1u) {
#pragma unroll
        for (int i2 = 0; i2 < M; ++i2)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = 8 * n + 2 * four + (e & 1);
              if (!(seen >> j & 1u) || token0 + j > limit[i2][e >> 1]) s[i2][n][e] = -INFINITY;
            }
      }
      bool moved = false;
      float keep[M][2];
#pragma unroll
      for (int i2 = 0; i2 < M; ++i2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float top = fmaxf(fmaxf(s[i2][0][2 * h], s[i2][0][2 * h + 1]), fmaxf(s[i2][1][2 * h], s[i2][1][2 * h + 1]));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const float next = fmaxf(m[i2][h], top), base = next == -INFINITY ? 0.0f : next;
          keep[i2][h] = exp2_fast(m[i2][h] - base);
          moved |= next != m[i2][h];
          m[i2][h] = next;
          float sum = 0.0f;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float w = exp2_fast(s[i2][n][2 * h + e] - base);
              s[i2][n][2 * h + e] = w;
              sum += w;
            }
          l[i2][h] = fmaf(l[i2][h], keep[i2][h], sum);
        }
      if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
        for (int i2 = 0; i2 < M; ++i2)
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i2][n][e] *= keep[i2][e >> 1];
      }
      // ---- a new token's values that are not finite go to the rows that see it, and not
      // into the product, where a weight of zero would not keep them from the others ----
      if (diagonal && p.window > 1) {
        const int first_new = max(at.len - p.window - token0, 0);
        bool odd = false;
        for (int c = lane; c < kAttnStep * kChunks; c += 32) {
          const int j = c / kChunks;
          if (j < first_new) continue;
          const uint4 v = rsm::lds128(values + c * 16);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            odd |= (w[k] & 0x7F800000u) == 0x7F800000u;
            if (!kF32) odd |= (w[k] & 0x7F80u) == 0x7F80u;
          }
        }
        if (__any_sync(0xFFFFFFFFu, odd)) {
          for (int j = first_new; j < kAttnStep; ++j) {
            if (!(seen >> j & 1u)) continue;
            const char* row = smem + (values - rsm::smem_addr(smem)) + j * Shape::kRow;
#pragma unroll
            for (int i2 = 0; i2 < M; ++i2)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float even = j & 8 ? s[i2][1][2 * h] : s[i2][0][2 * h], other = j & 8 ? s[i2][1][2 * h + 1] : s[i2][0][2 * h + 1];
                const float w = __shfl_sync(0xFFFFFFFFu, j & 1 ? other : even, (lane & ~3) + (j & 7) / 2);
                if (token0 + j <= limit[i2][h]) {
#pragma unroll
                  for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                      const int c = column(n, e) * static_cast<int>(sizeof(IT));
                      const float v = get(reinterpret_cast<const IT*>(row + ((c / 16) ^ value_order(j)) * 16 + c % 16));
                      if (!isfinite(v)) o[i2][n][2 * h + e] += w * v;
                    }
                }
              }
          }
          __syncwarp();
          for (int c = lane; c < kAttnStep * kChunks; c += 32) {
            if (c / kChunks < first_new) continue;
            IT* v = reinterpret_cast<IT*>(smem + (values - rsm::smem_addr(smem)) + c * 16);
#pragma unroll
            for (int k = 0; k < 16 / static_cast<int>(sizeof(IT)); ++k)
              if (!isfinite(get(v + k))) v[k] = IT(0);
          }
          __syncwarp();
        }
      }
      if constexpr (!kF32) {
        uint32_t pa[M][4];
#pragma unroll
        for (int i2 = 0; i2 < M; ++i2)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            pa[i2][2 * n] = rsm::pack_bf16x2(s[i2][n][0], s[i2][n][1]);
            pa[i2][2 * n + 1] = rsm::pack_bf16x2(s[i2][n][2], s[i2][n][3]);
          }
        const int token = (lane >> 3 & 1) * 8 + (lane & 7);
#pragma unroll
        for (int n = 0; n < kN; n += 2) {
          uint32_t vb[4];
          ldmatrix4_trans(vb, values + token * Shape::kRow + ((n + (lane >> 4)) ^ value_order(token)) * 16);
#pragma unroll
          for (int i2 = 0; i2 < M; ++i2) {
            mma_bf16(o[i2][n], pa[i2], vb[0], vb[1]);
            mma_bf16(o[i2][n + 1], pa[i2], vb[2], vb[3]);
          }
        }
      } else {
        // tokens 2 f and 2 f + 1 of eight are those of four = f, as S's columns are
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          uint32_t ph[4], pl[4];
          split_tf32(s[0][kt][0], ph[0], pl[0]);
          split_tf32(s[0][kt][2], ph[1], pl[1]);
          split_tf32(s[0][kt][1], ph[2], pl[2]);
          split_tf32(s[0][kt][3], ph[3], pl[3]);
          const int t0 = 8 * kt + 2 * four, t1 = t0 + 1;
#pragma unroll
          for (int n = 0; n < kN; n += 4) {
            const uint4 a = rsm::lds128(values + t0 * Shape::kRow + ((2 * n + quad) ^ value_order(t0)) * 16);
            const uint4 b = rsm::lds128(values + t1 * Shape::kRow + ((2 * n + quad) ^ value_order(t1)) * 16);
            const uint32_t va[4] = {a.x, a.y, a.z, a.w}, vb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h0, l0, h1, l1;
              split_tf32(__uint_as_float(va[k]), h0, l0);
              split_tf32(__uint_as_float(vb[k]), h1, l1);
              mma_tf32(o[0][n + k], pl, h0, h1);
              mma_tf32(o[0][n + k], ph, l0, l1);
              mma_tf32(o[0][n + k], ph, h0, h1);
            }
          }
        }
      }
    }

    // ---- the end of a unit, or of this CTA's part of it ----
    const bool last_tile = at.tile + 1 == at.tiles;
    if (last_tile || i + 1 == count) {
      const int g = at.u / p.row_tiles, rt = at.u - g * p.row_tiles;
      const bool whole = from == 0 && last_tile;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (from == 0 ? 1 : 0);
#pragma unroll
      for (int i2 = 0; i2 < M; ++i2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sum = l[i2][h];
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
          if (four == 0) m_s[warp][16 * i2 + 8 * h + quad] = m[i2][h], l_s[warp][16 * i2 + 8 * h + quad] = sum;
        }
      // the warps' outputs pass through the stages just read, 16 rows at a time
      const uint32_t pass = Shape::kQuery + stage * Shape::kStage;
#pragma unroll
      for (int i2 = 0; i2 < M; ++i2) {
        float* own = reinterpret_cast<float*>(smem + pass + warp * (S * Shape::kStage));
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = 8 * h + quad;
            if constexpr (kF32) {
#pragma unroll
              for (int e = 0; e < 2; ++e) own[row * DIM + (column(n, e) ^ (row & 3) << 3)] = o[i2][n][2 * h + e];
            } else {
              *reinterpret_cast<float2*>(own + row * DIM + (column(n, 0) ^ (row & 3) << 3)) = make_float2(o[i2][n][2 * h], o[i2][n][2 * h + 1]);
            }
          }
        __syncthreads();
        for (int c = threadIdx.x; c < 16 * DIM / 4; c += kAttnThreads) {
          const int row = c / (DIM / 4), col = (c - row * (DIM / 4)) * 4, r = 16 * i2 + row, all = rt * kRows + r;
          if (all >= rows_all) continue;
          float top = -INFINITY, sum = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w][r]);
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float f = top == -INFINITY ? 0.0f : exp2_fast(m_s[w][r] - top);
            const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + pass + w * (S * Shape::kStage)) +
                                                              row * DIM + (col ^ (row & 3) << 3));
            y.x = fmaf(v.x, f, y.x), y.y = fmaf(v.y, f, y.y), y.z = fmaf(v.z, f, y.z), y.w = fmaf(v.w, f, y.w);
            sum = fmaf(l_s[w][r], f, sum);
          }
          if (whole) {
            const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
            const int t = all / p.per;
            IT* out = static_cast<IT*>(p.out) + ((static_cast<int64_t>(at.b) * p.window + t) * p.H + g * p.per + all - t * p.per) * DIM + col;
            if constexpr (kF32)
              *reinterpret_cast<float4*>(out) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
            else
              *reinterpret_cast<uint2*>(out) = make_uint2(rsm::pack_bf16x2(y.x * f, y.y * f), rsm::pack_bf16x2(y.z * f, y.w * f));
          } else {
            *reinterpret_cast<float4*>(p.part + (slot * kRows + r) * DIM + col) = y;
            if (col == 0) {
              float* ml = p.part + 2 * static_cast<int64_t>(p.ctas) * kRows * DIM + (slot * kRows + r) * 2;
              ml[0] = top;
              ml[1] = sum;
            }
          }
        }
        __syncthreads();
      }
    }
    if (i + 1 == count) break;
    at.next(p, units);
    if (last_tile) {
      from = 0;
      load_queries();
      reset();
    }
  }
  cp_async_wait<0>();
}

// Units in pieces, each by the CTAs of the one that has its first piece: `parts` of
// them, which share its rows out.
template <typename IT, int DIM, int M>
__global__ void __launch_bounds__(kAttnJoinThreads) attn_join_kernel(const __grid_constant__ AttnParams p, int parts) {
  constexpr int kRows = 16 * M, kWarps = kAttnJoinThreads / 32, kPer = DIM / 32;
  __shared__ float acc_s[kWarps][DIM], l_s[kWarps];
  const int c0 = blockIdx.x / parts, part = blockIdx.x - c0 * parts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  AttnDeal deal;
  deal.total = deal_total<kAttnJoinThreads>(p, false);
  deal.ctas = min(static_cast<int64_t>(p.ctas), deal.total);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // by every CTA: the call is over when this kernel is
  if (c0 >= deal.ctas) return;
  const int64_t begin = deal.begin(c0), end = deal.begin(c0 + 1);
  const Place place = deal_find<kAttnJoinThreads>(p, end - 1);
  const int tiles = tiles_of(request_tokens(p.pages, place.b, p.window, nullptr, false));
  const int u = static_cast<int>((end - 1 - place.first) / tiles);
  const int64_t first = place.first + static_cast<int64_t>(u) * tiles;
  if (first + tiles <= end || first < begin) return;  // it ends here, or began before
  const int pieces = static_cast<int>(deal.owner(first + tiles - 1)) - c0 + 1;
  const int g = u / p.row_tiles, rt = u - g * p.row_tiles, rows = min(kRows, p.per * p.window - rt * kRows);
  const float* ml = p.part + 2 * static_cast<int64_t>(p.ctas) * kRows * DIM;
  auto slot = [&](int i) { return 2 * static_cast<int64_t>(c0 + i) + (i == 0 ? 1 : 0); };
  for (int r = part; r < rows; r += parts) {
    float top = -INFINITY;
    for (int i = lane; i < pieces; i += 32) top = fmaxf(top, ml[(slot(i) * kRows + r) * 2]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float acc[kPer], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
#pragma unroll 4
    for (int i = warp; i < pieces; i += kWarps) {
      const int64_t at = slot(i) * kRows + r;
      const float f = top == -INFINITY ? 0.0f : exp2_fast(ml[at * 2] - top);
      sum = fmaf(ml[at * 2 + 1], f, sum);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(p.part[at * DIM + lane + 32 * k], f, acc[k]);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc_s[warp][lane + 32 * k] = acc[k];
    if (lane == 0) l_s[warp] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += l_s[w];
    const int all = rt * kRows + r, t = all / p.per;
    IT* out = static_cast<IT*>(p.out) + ((static_cast<int64_t>(place.b) * p.window + t) * p.H + g * p.per + all - t * p.per) * DIM;
    for (int c = threadIdx.x; c < DIM; c += kAttnJoinThreads) {
      float y = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) y += acc_s[w][c];
      put(out + c, sum == 0.0f ? 0.0f : y / sum);
    }
    __syncthreads();
  }
}

}  // namespace hybrid
