// Modified attention scores inside the tensor-core kernels, in log2 units:
//
//   y = cap2 tanh(a / cap2) + bias(distance),   a = s * scale * log2(e)
//
// with cap2 = softcap * log2(e) and bias 0, minus slope times |distance|, or an
// entry of a table by signed distance (the learned bias of every bucket, laid
// out by distance and scaled by log2(e) before the launch).
//
// tanh is wanted to about 1e-6: the scores feed an exponential, and lse is an
// fp32 result.  tanh.approx (2^-11) is too coarse.  Where a whole warp's scores
// stay within |a| <= 0.75 cap2, tanh(z) = z (1 + c1 z^2 + .. + c4 z^8) with
// minimax coefficients on |z| <= 0.75 (off by at most 6e-7 of the value): fused
// multiply-adds alone, two scores per instruction.  Otherwise 1 - 2 / (1 +
// e^(2z)), two more special-function instructions per score.
//
// A bias costs as little as the tile allows: beyond the table's last distance it
// is one number per row, which joins the softmax's own subtraction; slopes add one
// multiply-add per score (their row part joins the same subtraction); only tiles
// near the diagonal read the table (through L1, neighbouring lanes neighbouring
// entries), and only those inside a two-way prefix take |distance|.
#pragma once
#include <stdint.h>

#include "ptx.cuh"
#include "tc.h"

namespace cpattn {
namespace score {

using namespace ptx;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPolyRange = kCapPolyRange;
constexpr float kC1 = kCapPoly[0], kC2 = kCapPoly[1], kC3 = kCapPoly[2], kC4 = kCapPoly[3];

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The forward's cap: products s become scores s * factor(s), a polynomial in s^2
// with the scale and the cap in its coefficients (six fused operations a score
// with the softmax's own subtraction, where scaling, tanh and scaling back take
// eight: 18 688 tokens x 8 of 128 812 -> 780 us, with slopes 890 -> 815, with a
// table 863 -> 796), or any(s) * mul.
template <bool kCap>
struct FwdCap {
  float in = 0.f, mul = 0.f, reach = -1.f;
  uint64_t k[5] = {0, 0, 0, 0, 0};
  __device__ __forceinline__ FwdCap(const ScoreArgs& s, float scale_log2) {
    if constexpr (kCap) {
      mul = s.cap_log2;
      in = scale_log2 * s.inv_cap_log2;
      reach = s.cap_reach;
#pragma unroll
      for (int i = 0; i < 5; ++i) k[i] = pack2(s.cap_k[i], s.cap_k[i]);
    }
  }
  // the largest |s| of a warp lets the polynomial serve
  __device__ __forceinline__ bool in_range(float big) const {
    return __all_sync(0xffffffffu, big <= reach);
  }
  __device__ __forceinline__ uint64_t factor(uint64_t s) const {
    const uint64_t v = mul2(s, s);
    uint64_t p = fma2(k[4], v, k[3]);
    p = fma2(p, v, k[2]);
    p = fma2(p, v, k[1]);
    return fma2(p, v, k[0]);
  }
  // any s: tanh z = 1 - 2 / (1 + e^(2z)), e^(2z) = 2^(2 z log2 e)
  __device__ __forceinline__ float any(float s) const {
    return fmaf(-2.f, rcp_approx(1.f + ex2(s * in * (2.f * kLog2e))), 1.f);
  }
};

// The backward's cap: products s become t = -tanh(s * in), in = scale / softcap; the
// scores are t * mul, mul = -cap2.  (With the sign reversed one constant, -1, serves
// the polynomial and the slope.  The products are scaled before the polynomial, as
// tanh itself is wanted.)
template <bool kCap>
struct BwdCap {
  static constexpr float kUnit = -1.f;
  float in = 0.f, mul = 0.f;
  uint64_t in2 = 0, unit = 0, k[4] = {0, 0, 0, 0};
  __device__ __forceinline__ BwdCap(const ScoreArgs& s, float scale_log2) {
    if constexpr (kCap) {
      mul = kUnit * s.cap_log2;
      in = scale_log2 * s.inv_cap_log2;
      in2 = pack2(in, in);
      unit = pack2(kUnit, kUnit);
      k[0] = pack2(kUnit * kC1, kUnit * kC1);
      k[1] = pack2(kUnit * kC2, kUnit * kC2);
      k[2] = pack2(kUnit * kC3, kUnit * kC3);
      k[3] = pack2(kUnit * kC4, kUnit * kC4);
    }
  }
  // the largest |s| of a warp, times in, lets the polynomial serve
  __device__ __forceinline__ bool in_range(float big) const {
    return __all_sync(0xffffffffu, big * in <= kPolyRange);
  }
  __device__ __forceinline__ uint64_t poly(uint64_t s) const {
    const uint64_t z = mul2(s, in2), v = mul2(z, z);
    uint64_t p = fma2(k[3], v, k[2]);
    p = fma2(p, v, k[1]);
    p = fma2(p, v, k[0]);
    p = fma2(p, v, unit);
    return mul2(z, p);
  }
  __device__ __forceinline__ float any(float s) const {
    return fmaf(-2.f * kUnit, rcp_approx(1.f + ex2(s * in * (2.f * kLog2e))), kUnit);
  }
  // t^2 - 1
  __device__ __forceinline__ uint64_t minus_slope(uint64_t t) const {
    return fma2(t, t, unit);
  }
};

// The bias of one tile for one thread: columns run over keys (forward, the
// distance falls by one per column) or queries (backward, it rises).
struct TileBias {
  float base = 0.f;             // added to every column, log2 units
  float step = 0.f;             // slopes: change per column, log2 units
  const float* tab = nullptr;   // near tile of a table bias: entry of column 0
  bool both = false;            // slopes: distances of both signs are visible
  float slope = 0.f, dist0 = 0.f;
};

// kSign: distance of column c is dist0 + kSign * c.  [lo, hi]: the smallest and
// largest distance in the whole tile (the same for all its threads).
template <int kBias, int kSign>
__device__ __forceinline__ TileBias tile_bias(const ScoreArgs& s, int h, float slope2, int dist0,
                                              int lo, int hi, bool causal) {
  TileBias b;
  if constexpr (kBias == SCORE_SLOPES) {
    b.slope = slope2;
    b.dist0 = (float)dist0;
    b.both = !causal && lo < 0;
    if (!b.both) {
      b.base = -slope2 * (float)dist0;
      b.step = kSign > 0 ? -slope2 : slope2;
    }
  } else if constexpr (kBias == SCORE_TABLE) {
    const float* row = s.table + (long long)h * s.table_pitch + s.table_mid;
    if (lo >= s.n_dist - 1 || hi <= -(s.n_dist - 1)) b.base = row[s.n_dist - 1];
    else b.tab = row + dist0;
  }
  return b;
}

// Slopes with both signs, or a near table: the bias of column c in log2 units.
template <int kBias, int kSign>
__device__ __forceinline__ float column_bias(const TileBias& b, int c) {
  if constexpr (kBias == SCORE_SLOPES) return -b.slope * fabsf(b.dist0 + (float)(kSign * c));
  if constexpr (kBias == SCORE_TABLE) return b.tab[kSign * c];
  return 0.f;
}

}  // namespace score
}  // namespace cpattn
