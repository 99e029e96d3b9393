// Work lists of attention with modified scores.
//
// The P simulated ranks are partitions of one memory and a query row sees the
// same keys whichever rank owns them, so these lists walk every sample's rows in
// natural order: no gather, one key run per query tile, one query run per key
// tile, and distances are differences of positions.  Where few tiles would leave
// SMs idle behind the longest of them, long runs are cut into parts (part_limit):
// the forward's parts leave fp32 results that a last kernel joins, the backward's
// add their dK and dV.  A plan is one flat block,
// built on the host, that the caller copies to the device once and keeps for
// every call with the same packing.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <string>

#include "plan.h"

namespace cpattn {

constexpr int kTile32 = 64;   // rows of one tile of the fp32 kernels

// One 64-row tile of a sample (fp32 kernels, queries and keys alike, and the passes
// over the rows of short samples).
struct Tile32 {
  int32_t row0, len;     // natural rows [row0, row0 + len)
  int32_t seq0, seq_len; // the sample's rows
  int32_t prefix;        // rows that see one another in both directions (0: causal)
  int32_t sample;
  int32_t pad[2];
};
static_assert(sizeof(Tile32) == 32, "Tile32 layout");

// A forward tile whose keys were cut: its rows, and the first row of its `parts`
// partial results, each `len` rows long.
struct Join {
  int32_t out_row0, len, run_row0, parts;
};
static_assert(sizeof(Join) == 16, "Join layout");

constexpr uint32_t kScorePlanMagic = 0x43505350u;
constexpr int kMaxDist = 1 << 16;
// Longest sample whose backward may take f16 operands (operand_range.cuh).
constexpr int kF16Tokens = 1024;

// At the start of the block; offsets are bytes from there.
struct ScorePlanHeader {
  uint32_t magic;
  int32_t T, H, n_seqs, bidirectional;
  int32_t n_dist, n_buckets;       // 0: no table
  int32_t n_fwd, n_bwd, n_tiles;
  int32_t fwd_part, bwd_part;      // tiles of the longest part of a cut run (0: none cut)
  int32_t n_joins, run_rows;       // forward: cut tiles and their partial rows per head
  int32_t bwd_cut;                 // nonzero: several backward items share a key tile
  int32_t max_walk;                // tiles of the longest sample (fp32 kernels)
  int32_t n_units, grid;           // forward: units and persistent CTAs
  int32_t item_major;              // the forward's unit order
  int32_t n_sms;
  int32_t n_short;                 // tiles of samples of up to kF16Tokens tokens
  uint64_t fwd, bwd, runs, units, buckets, tiles, joins, total;
};
static_assert(sizeof(ScorePlanHeader) <= 256, "plan header");

// Order of a launch's work units: item by item, heaviest first over all heads,
// below 16 units per SM, where a heavy unit that starts late costs most; head by
// head above, where K / V (or Q / dO) of one or two heads stay in L2.
inline bool item_major(int64_t units, int sms) { return units < 16LL * sms; }

// Checks the arguments ("" or a message) and fills `h` without building.
std::string score_plan_layout(const int32_t* cu, int n_seqs, const int32_t* prefix_lens,
                              bool bidirectional, int H, int sms, const int32_t* buckets,
                              int n_dist, ScorePlanHeader* h);
// Writes the block (h.total bytes).
void score_plan_build(const ScorePlanHeader& h, const int32_t* cu, const int32_t* prefix_lens,
                      const int32_t* buckets, void* block);

}  // namespace cpattn
