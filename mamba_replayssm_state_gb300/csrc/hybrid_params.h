// hybrid_params.h -- what the convolution, rotary, attention and page kernels are given.
#pragma once
#include <cuda.h>

#include <cstdint>

#include "../../include/replayssm_hybrid.h"

namespace hybrid {

struct ConvParams {
  const void* x;
  const float *weight, *bias;
  const int32_t* cu;  // packed prompts
  void* cache;
  const int32_t *slots, *positions;
  void* out;
  uint32_t* status;
  int64_t tokens, x_bs, x_ts, out_ts, cache_ss;
  int32_t seqs, window, num_slots, C, R, silu, pad;
  int32_t cblocks;  // CTAs across the channels
  int32_t block;    // tokens, or requests, of a CTA
};

constexpr int kConvThreads = 128;
constexpr int kConvAhead = 16;         // tokens whose rows are on their way, prompts
constexpr int kConvStepRequests = 16;  // of a CTA at most

// vec: eight bf16 or four fp32 channels a thread, on 16 bytes; else one channel.
const void* conv_kernel(int input_dtype, int width, bool vec);
const void* conv_step_kernel_of(int input_dtype, int width, bool vec);
constexpr int conv_channels(int input_dtype, bool vec) { return !vec ? 1 : input_dtype == RSM_BF16 ? 8 : 4; }

struct RotaryParams {
  const void *q, *k, *v;
  const float* inv_freq;
  const int32_t* cu;
  void* q_out;
  uint32_t* status;
  rsm_pages pages;
  int64_t tokens, q_bs, q_ts, k_bs, k_ts, v_bs, v_ts, out_bs, out_ts;
  int32_t window, H, G, dim, half, interleaved;  // half: rotary_dim / 2
  float amplitude;
  int32_t stages;  // tokens that a ring holds
};

// A CTA's ring: up to kRotaryRing bytes where two CTAs share an SM, up to kRotaryRingAlone for long tokens.
constexpr int kRotaryThreads = 160, kRotaryMaxStages = 8, kRotaryMaxHalf = 128, kRotaryPlainThreads = 256;
constexpr int kRotaryRing = 104 * 1024, kRotaryRingAlone = 216 * 1024;
constexpr uint64_t kRotaryTimeoutNs = 2000000000ull;  // of a wait that takes microseconds
// at_once: values that a thread takes, 1 (the kernel of a CTA a token alone), 4 or (bf16) 8.
const void* rotary_kernel(int input_dtype, int at_once);
const void* rotary_token_kernel_of(int input_dtype, int at_once);

struct AttnParams {
  const void* q;
  void* out;
  uint32_t* status;
  rsm_pages pages;
  int64_t q_bs, q_ts;
  int32_t window, H, G, per, dim;  // per: heads of a key head
  float scale_log2;                // scale * log2(e)
  // the tiled kernel
  float* part;                     // partial outputs, then their maxima and sums
  int32_t row_tiles, ctas, page_shift, tile_shift;  // page_shift: log2(page_size), or -1; tile_shift: of a tile's tokens
  int32_t unit_end;                // tiles that the end of a unit counts
  int32_t q_pairs, q_wide;         // queries may be read two at a time, and 16 bytes
  int32_t out_wide;                // the outputs' rows start on 16 bytes
  int32_t page_rows, head_rows, head_columns;  // loads of rows from anywhere: a page's and a head's distance in the maps' rows and columns
  float hidden;                    // a score that times scale_log2 is -infinity
};

// The tiled kernel, for heads of up to 64, 128 and 256 columns (`dim`, here, is the one of these that holds
// a head): a warp takes attn_step() tokens at a time, a CTA's four warps a tile of four times as
// many; attn_stages() of them are on the way at once, 96 KB a CTA where two of them share an SM, 48 or 64 where three do.
constexpr int kAttnThreads = 128, kAttnJoinThreads = 256;
// Tiles that the end of a unit counts: the more, the more values its warps have to put together (100000 tokens of 8 key
// heads of 128: 32 rows in 32 requests 85 us with four tiles, 99 with two; 24 rows in 128 83 and 99; 16 in 128 78 with
// three, 87 with two; heads of 256, 50000 tokens: 8 rows 74 with three, 79 with two, 16 rows 81 with four, 84 with three.
// One tile: 20 rows 77 us, 67 with more; six or eight: 24 rows in 128 requests 87 and 94.  fp32, 1, 2 and 3 tiles: heads of 128, 50000
// tokens, 8 rows in 32 requests 99, 95 and 94, in 128 123, 118 and 119, 1 row in 32 67.6, 67.9 and 69.0, in 128 70, 71 and 73; heads of
// 64, 100000 tokens, 8 rows in 128 93, 84 and 86; heads of 256, 25000 tokens, 1 row in 128 75, 78 and 81, 4 rows 96, 94 and 99).
constexpr int attn_unit_end(int esize, int dim, int rows) {
  const int values = dim * rows;  // of an output
  return esize == 4 ? 2 : rows > 16 || values > 2048 ? 4 : rows > 8 || values > 1024 ? 3 : 2;
}
constexpr int attn_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
// Up to 16 rows of bf16 heads of 64 and eight of 128 leave registers for a third CTA an SM (`three`).  Heads of 64 take
// it, with shorter steps (8 key heads: 100000 tokens in 256 requests 41 us, 47 by steps of 32 of two CTAs; one request of
// 16000, which more CTAs share, 12.6 and 17.2; 16 rows, 400000 tokens, 145 and 152, but 4 requests of 1000 12.7 and 11.3).
// Heads of 128, with two stages, where there are two units an SM or more (64 requests, 200000
// tokens, 8 key heads: 125.5 us, 130.5 of two CTAs; 256 of 78 tokens each 27.7 and 31.1, of 390 73.6 and 72.8); with fewer
// units there are more pieces to join (8 requests of 1000 tokens 13.6 us, 14.9 of three; one of 131072 29.7 and 30.6).
constexpr bool attn_three(int esize, int dim, int rows, bool many) { return esize == 2 && (dim == 64 ? rows <= 16 : rows == 8 && dim == 128 && many); }
// Whether bf16 weights meet the values with 16 bits (`low`; rows: all of a key head), as sums of two bf16 values: outputs are
// then as near to 64 bits as with fp32 weights (64 ragged requests: 0.00165 of the norm, their own rounding; 0.0020 with
// weights rounded to 8 bits).  us with one product and with two, 8 key heads of 128, 100000 tokens in 32 requests:
//   8 rows 70.9 and 71.2, 16 rows 75.3 and 76.1, 24 rows 80.1 and 80.3: memory hides the second
//   24 rows in 128 requests 84 and 91.5; 32 rows 86 and 90; windows of 64 and 128 rows 137 and 157, 262 and 297; 40 rows, two
//   units of 24, 117 and 133: the products bind
// Heads of 64, 200000 tokens: 16 rows 79.3 and 80.3, 24 rows 85.2 and 85.0, 32 rows 86.5 and 99.7; of 256, 50000 tokens: 8 rows 74.7
// and 75.3, 16 rows 81 and 86.
constexpr bool attn_low(int dim, int64_t rows) { return rows <= (dim == 256 ? 8 : 24); }
constexpr int attn_step(int esize, int dim, bool three) { return esize * dim > 512 ? 8 : esize * dim > 128 || three ? 16 : 32; }
constexpr int attn_stages(int esize, int dim, bool three) { return three && esize * dim > 128 ? 2 : 3; }
constexpr int attn_box(int esize, int dim) { return esize * dim > 512 ? 8 : 16; }  // tokens of a TMA box
// The rows of a unit at most, for the one type and the other.
constexpr int attn_rows(int esize, int dim) { return esize == 4 ? (dim == 256 ? 4 : 8) : dim == 256 ? 16 : 32; }
// bf16 queries that lie in shared memory
constexpr bool attn_shared_queries(int dim, int rows) { return dim * rows > 2048; }
// What lies before the stages: those queries, or fp32's weights (each twice).
constexpr int attn_query(int esize, int dim, int rows) {
  return esize == 4 ? (4 * attn_step(4, dim, false) * rows * 8 + 1023) / 1024 * 1024 : attn_shared_queries(dim, rows) ? 2 * dim * rows : 0;
}
constexpr int attn_smem(int esize, int dim, int rows, bool three) {
  return attn_stages(esize, dim, three) * 4 * attn_step(esize, dim, three) * 2 * dim * esize + attn_query(esize, dim, rows);
}
constexpr int attn_ctas_per_sm(int esize, int dim, bool three) {
  return three ? 3 : attn_smem(esize, dim, attn_rows(esize, dim), false) > 110 * 1024 ? 1 : 2;
}
struct AttnTileParams {
  AttnParams p;
  // boxes: [pages, page_size, kv heads, dim], of attn_box() rows of a head, 128 bytes of columns; gathers: [rows, columns]
  CUtensorMap k_map, v_map;
};
enum class AttnLoads { kRows, kBoxes, kGather };
// rows: of a unit, 1, 2, 4 or 8 for fp32 and a multiple of 8 for bf16.  tiles: by AttnLoads.
struct AttnKernels {
  const void *tiles[3], *join;
};
AttnKernels attn_bf16_64(int rows, bool low);
AttnKernels attn_bf16_128(int rows, bool three, bool low);
AttnKernels attn_bf16_256(int rows);
AttnKernels attn_f32_64(int rows);
AttnKernels attn_f32_128(int rows);
AttnKernels attn_f32_256(int rows);

constexpr int kAttnPlainThreads = 128;
const void* attn_plain_kernel(int input_dtype);

struct CopyParams {
  const int64_t *ptrs, *strides;
  const int32_t *src, *dst;
  uint32_t* status;
  int64_t page_bytes;
  int32_t pools, pairs, pages, esize;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = 16384;  // of a CTA
const void* copy_kernel();

}  // namespace hybrid
