// ssm_tc_params.h -- the tensor-core prompt kernel: its parameters, shared
// memory and tensor memory plan.
#pragma once
#include <cuda.h>

#include "ssm_params.h"

namespace ssm {

constexpr int kChunk = 128;  // tokens of a chunk: the MMAs' M, and the K of two of them
constexpr int kDim = 64, kState = 128;
constexpr int kTile = kChunk * 128;  // bytes of a [128 rows x 64 bf16] tile, 128-byte swizzled

struct TcParams {
  CUtensorMap x_map, B_map, C_map;  // [tokens, H * 64], [tokens, G * 128] bf16, boxes of 128 rows x 64 columns
  Params p;
  uint32_t seg;        // tokens of a segment, a multiple of kChunk, below 2^31
  float* seg_state;    // [segments, H, 64, 128]: states between segments (NULL when nothing is split)
  float* seg_decay;    // [segments, H]
  int32_t pairs;       // head groups of a CTA in all: H / NH
  int32_t states_only; // the pass that makes the segments' own states
};

// Shared memory, bytes: two stages each of C, B and the heads' x (where w x or
// its hi part replaces x), and one more pair of tiles.  Those hold the bf16
// state, or, where the update has a lo part, that; the state then takes the x
// stage of the chunk that made it, which is free from that chunk's update until
// the next one's Y1 has read the state.  Then the small things.
constexpr uint32_t kOffC = 0;
constexpr uint32_t kOffB = kOffC + 4 * kTile;
constexpr uint32_t kOffX = kOffB + 4 * kTile;
constexpr uint32_t kOffMore = kOffX + 4 * kTile;
constexpr uint32_t kOffDt = kOffMore + 2 * kTile;       // [2 stages][2 heads][128] fp32
constexpr uint32_t kOffV = kOffDt + 2 * 2 * kChunk * 4; // [2 heads][96] fp32
constexpr uint32_t kOffBar = kOffV + 2 * 96 * 4;
enum Bar : uint32_t {
  kFullBC = 0, kEmptyBC = 2, kFullX = 4, kEmptyX = 6, kFullDt = 8, kEmptyDt = 10, kGFull = 12, kPFull = 13,
  kPxDone = 15, kY2Empty = 17, kSFull = 19, kY1Full = 20, kVRead = 21, kWFull = 22, kClean = 23, kUFull = 24,
  kVSync = 25, kExit = 27, kBars = 28
};
constexpr uint32_t kOffTmem = kOffBar + 8 * kBars;
constexpr uint32_t kOffAbort = kOffTmem + 4;
constexpr uint32_t kTcSmem = kOffAbort + 4;
static_assert(kTcSmem <= 232448, "shared memory of one CTA");

// tensor memory, columns: G = C B^T, the heads' P (bf16 pairs), P X, and one
// region that holds C S^T and then the state update
constexpr uint32_t kColG = 0, kColP = 128, kColY2 = 256, kColV = 384;

constexpr int kTcThreads = 768;  // one warpgroup for loader, MMA and dt, two for P, one for w X, two for y and S
constexpr uint64_t kTcTimeoutNs = 2000000000ull;

// heads: 1 or 2 a CTA; lo: the state update keeps 16 bits of w x
const void* tc_kernel(int heads, bool lo);

// Between the two passes of a split call: the state every segment starts from.
// Grid: (num_seqs * H), 256 threads.
const void* join_kernel();

}  // namespace ssm
