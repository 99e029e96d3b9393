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
#pragma once
#include <stdint.h>

#include "ptx.cuh"
#include "tc.h"

namespace cpattn {
namespace score {

using namespace ptx;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPolyRange = 0.75f;
constexpr float kC1 = -0.33329880795843986f, kC2 = 0.13270406554292946f,
                kC3 = -0.050340821426050376f, kC4 = 0.013161359006389609f;

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a thread keeps for the whole launch.
template <bool kCap>
struct Cap {
  float limit = 0.f, cap2 = 0.f, inv = 0.f;
  uint64_t k[4] = {0, 0, 0, 0}, one = 0;
  __device__ __forceinline__ explicit Cap(const ScoreArgs& s) {
    if constexpr (kCap) {
      cap2 = s.cap_log2;
      inv = s.inv_cap_log2;
      limit = kPolyRange * cap2;
      const float i2 = inv * inv;
      k[0] = pack2(kC1 * i2, kC1 * i2);
      k[1] = pack2(kC2 * i2 * i2, kC2 * i2 * i2);
      k[2] = pack2(kC3 * i2 * i2 * i2, kC3 * i2 * i2 * i2);
      k[3] = pack2(kC4 * i2 * i2 * i2 * i2, kC4 * i2 * i2 * i2 * i2);
      one = pack2(1.f, 1.f);
    }
  }
  // cap2 tanh(a / cap2) of two scores, |a| <= limit
  __device__ __forceinline__ uint64_t poly(uint64_t a) const {
    const uint64_t v = mul2(a, a);
    uint64_t p = fma2(k[3], v, k[2]);
    p = fma2(p, v, k[1]);
    p = fma2(p, v, k[0]);
    p = fma2(p, v, one);
    return mul2(a, p);
  }
  // the same for any a: tanh z = 1 - 2 / (1 + e^(2z)), e^(2z) = 2^(2 z log2 e)
  __device__ __forceinline__ float any(float a) const {
    const float e = ex2(a * (inv * (2.f * kLog2e)));
    return fmaf(-2.f * cap2, rcp_approx(1.f + e), cap2);
  }
};

// The bias of one tile for one thread: columns run over keys (forward, the
// distance falls by one per column) or queries (backward, it rises).
struct TileBias {
  float base = 0.f;    // added to every column
  float step = 0.f;    // slopes: change per column
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

// Bias of column c that is not in `base`, added to y.
template <int kBias, int kSign>
__device__ __forceinline__ float add_column(const TileBias& b, int c, float y) {
  if constexpr (kBias == SCORE_SLOPES) {
    if (b.both) return fmaf(-b.slope, fabsf(b.dist0 + (float)(kSign * c)), y);
    return fmaf((float)c, b.step, y);
  }
  if constexpr (kBias == SCORE_TABLE) {
    if (b.tab) return y + b.tab[kSign * c];
  }
  return y;
}

}  // namespace score
}  // namespace cpattn
