// The order in which a product's tiles are walked.
#pragma once
#include "ffn.h"

namespace cpattn {

namespace {

// m tiles whose n tiles are walked together: about square patches of tiles run at a
// time, which reads the least of A and B.
constexpr int kGroupM = 8;

struct TilePlace {
  int m, n;
};
__device__ __forceinline__ TilePlace tile_place(const GemmArgs& g, int tile) {
  const unsigned per_group = kGroupM * g.n_tiles;
  const unsigned group = (unsigned)tile / per_group, in = (unsigned)tile % per_group;
  const unsigned first = group * kGroupM;
  const unsigned rows = min(kGroupM, g.m_tiles - (int)first);
  return {(int)(first + in % rows), (int)(in / rows)};
}

}  // namespace

}  // namespace cpattn
