// Work split of the feed-forward products' persistent kernels: units of (product, tile,
// share of k), and the sums of shared tiles.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "check.cuh"
#include "ffn.h"
#include "ptx.cuh"

namespace cpattn {

// m tiles whose n tiles are walked together: about square patches of tiles run at a
// time, which reads the least of A and B.
constexpr int kGroupM = 8;

// Unit u: a tile of a problem, and which of its k tiles.  The issuing thread asks for
// no more: between two tiles the tensor core waits for it.
struct Work {
  int p, tile, k0, k1;
  int slot, share, ticket;   // of the partial sums, the slot -1 for a whole tile
};
template <class Args>
__device__ __forceinline__ Work work_at(const Args& g, int u) {
  Work w;
  w.p = 0;
  while (w.p + 1 < g.problems && u >= g.p[w.p + 1].first) ++w.p;
  const GemmTiles& p = g.p[w.p];
  w.tile = u - p.first;
  w.slot = -1;
  w.share = w.ticket = 0;
  unsigned shares = 1;
  if (w.tile >= p.whole) {
    const unsigned v = w.tile - p.whole;
    shares = p.shares;
    w.ticket = p.first_ticket + (int)(v / shares);
    w.share = (int)(v % shares);
    w.tile = p.whole + (int)(v / shares);
    w.slot = p.first_slot + (int)v;
  }
  const unsigned k_tiles = p.k_tiles;
  w.k0 = w.share == 0 ? 0 : (int)(k_tiles * w.share / shares);
  w.k1 = w.share + 1 == (int)shares ? (int)k_tiles : (int)(k_tiles * (w.share + 1) / shares);
  return w;
}
struct Unit : Work {
  int m, n;
};
template <class Args>
__device__ __forceinline__ Unit unit_at(const Args& g, int u) {
  Unit t;
  static_cast<Work&>(t) = work_at(g, u);
  const GemmTiles& p = g.p[t.p];
  const unsigned per_group = kGroupM * p.n_tiles;
  const unsigned group = t.tile / per_group, in = t.tile % per_group;
  const unsigned first = group * kGroupM;
  const unsigned rows = min(kGroupM, p.m_tiles - (int)first);
  t.m = (int)(first + in % rows);
  t.n = (int)(in / rows);
  return t;
}

// kCols columns from `col` on of tile row `row` into a shared tile's sums.
template <int kN, int kCols>
__device__ __forceinline__ void store_partial(float* partial, int slot, int col, int row,
                                              const float (&f)[kCols]) {
  float4* p = reinterpret_cast<float4*>(partial) +
              ((int64_t)slot * (kN / 4) + col / 4) * kGemmM + row;
#pragma unroll
  for (int i = 0; i < kCols / 4; ++i)
    p[i * kGemmM] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}

// The same columns of all shares of a tile, from slot `slot` on, added in order.
template <int kN, int kCols>
__device__ __forceinline__ void load_partials(const float* partial, int slot, int shares, int col,
                                              int row, float (&f)[kCols]) {
#pragma unroll
  for (int i = 0; i < kCols; ++i) f[i] = 0.f;
#pragma unroll 64 / kCols
  for (int s = 0; s < shares; ++s) {
    const float4* p = reinterpret_cast<const float4*>(partial) +
                      ((int64_t)(slot + s) * (kN / 4) + col / 4) * kGemmM + row;
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i) {
      const float4 v = __ldcg(p + i * kGemmM);   // written by other CTAs of this launch
      f[4 * i] += v.x;
      f[4 * i + 1] += v.y;
      f[4 * i + 2] += v.z;
      f[4 * i + 3] += v.w;
    }
  }
}

template <int kCols>
__device__ __forceinline__ void load_acc(uint32_t taddr, float (&f)[kCols]) {
  uint32_t r[kCols];
  if constexpr (kCols == 32) ptx::tmem_ld32(taddr, r);
  else ptx::tmem_ld16(taddr, r);
  ptx::tmem_ld_wait();
  ptx::reg_fence(r);
#pragma unroll
  for (int i = 0; i < kCols; ++i) f[i] = __uint_as_float(r[i]);
}

}  // namespace cpattn
