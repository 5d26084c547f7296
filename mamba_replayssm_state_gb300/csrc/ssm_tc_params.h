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
  CUtensorMap y_map;                // [tokens, H * 64], boxes of 32 rows x 32 columns
  Params p;
  uint32_t seg;        // tokens of a segment, a multiple of kChunk, below 2^31
  float* seg_state;    // [segments, H, 64, 128]: states between segments (NULL when nothing is split)
  float* seg_decay;    // [segments, H]
  int32_t pairs;       // head groups of a CTA in all: H / NH
  int32_t states_only; // the pass that makes the segments' own states
};

// Shared memory, bytes: two stages each of C, B and the heads' x (where w x or
// its hi part replaces x), the outputs on their way out, and the decay tables.
// Two things live in what others leave free: the lo part of w x in its chunk's C
// stage, from Y1, the last to read C, to the update; the bf16 state in the x stage
// of the chunk that made it, from that chunk's update to the next one's Y1.
constexpr uint32_t kOffC = 0;
constexpr uint32_t kOffB = kOffC + 4 * kTile;
constexpr uint32_t kOffX = kOffB + 4 * kTile;
constexpr uint32_t kOffY = kOffX + 4 * kTile;  // of a head's 32 rows: 32 columns, 64-byte swizzled
constexpr uint32_t kYBytes = 2 * 32 * 32;
// A table of [stage][head], made by a dt warp; fp32, 128 tokens where not said otherwise.
// p is the decay (log2) from the start of a token's half of the chunk up to and with it, mid
// half of the half's (a mild or a steep one: 0).
enum Table : uint32_t {
  kTabCol = 0,     // dt 2^(mid-p): what a column of P is scaled by in its own half (a steep half: p itself)
  kTabDt = 512,    // dt
  kTabV = 1024,    // [64] first half: dt 2^(decay after the token up to the half's end + the second's mid)
  kTabW = 1280,    // dt 2^(decay after the token up to the chunk's end)
  kTabM1 = 1792,   // y = m1 Y1 + m2 Y2: 2^(decay from the chunk's start)
  kTabM2 = 2304,   //                    2^(p-mid) (a steep half: 1)
  kTabSkip = 2816, // D 2^(mid-p) (a steep half: D)
  kTabMisc = 3328, // 2^(decay of the chunk); its log2; whether each half is steep
  kTabBytes = 3344
};
constexpr uint32_t kOffTab = kOffY + 8 * kYBytes;
constexpr uint32_t kOffBar = kOffTab + 4 * kTabBytes;
enum Bar : uint32_t {
  kFullBC = 0, kEmptyB = 2, kEmptyC = 4, kFullX = 6, kEmptyX = 8, kFullTab = 10, kEmptyTab = 12, kGFull = 14, kPFull = 16,
  kWFull = 18, kLoFull = 20, kUFull = 22, kURead = 24, kPxDone = 26, kSFull = 27, kY1Full = 28, kYRead = 29, kClean = 30,
  kExit = 31, kBars = 33
};
constexpr uint32_t kOffTmem = kOffBar + 8 * kBars;
constexpr uint32_t kOffOrder = kOffTmem + 8;  // the sequences, longest first, if they are few
constexpr int kSorted = 32;
constexpr uint32_t kTcSmem = kOffOrder + 4 * kSorted;
static_assert(kTcSmem <= 232448, "shared memory of one CTA");

// tensor memory, columns: of every other chunk G = C B^T, P in its place (a block
// of 32 columns becomes the two heads' 16 of bf16 pairs) and then the state update
// in P's; P X; C S^T
constexpr uint32_t kColG = 0, kColY2 = 256, kColY1 = 384;

constexpr int kTcThreads = 896;  // a warpgroup for loader, MMA and tables, two each for P, for w X, for the states and y
// A wait gives up after this many tries, each of which rests for up to 2700 cycles
// (measured): after a second and a half at most.
constexpr uint32_t kTcTries = 1u << 20;

// heads: 1 or 2 a CTA; lo: the state update keeps 16 bits of w x
const void* tc_kernel(int heads, bool lo);

// Between the two passes of a split call: the state every segment starts from.
// Grid: num_seqs * H * the state's elements / (4 kJoinThreads).
constexpr int kJoinThreads = 128;
const void* join_kernel();

}  // namespace ssm
