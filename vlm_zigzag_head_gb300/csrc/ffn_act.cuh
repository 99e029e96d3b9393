// Activations of the gated feed-forward block and their derivatives.
#pragma once
#include <cuda_bf16.h>

#include "ffn.h"
#include "ptx.cuh"

namespace cpattn {

namespace {

__device__ __forceinline__ float inverse(float x) {   // 1 unit in the last place; 0 of infinity
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^-z); e^-z overflows to infinity, whose inverse is 0.  kFast, for bf16 results: the
// exponent's rounding and the approximations are off by about |z| 2^-24 and 2^-22 of the value.
// fp32 results take the math library's exponential and a rounded inverse: 1.9e-7 of the value down
// to z = -80, where the other way is off by 3.7e-6 (517 x 512 x 1360 with silu, forward 37 us with
// that and 39 so, backward 58 and 62).
template <bool kFast>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (!kFast) return __frcp_rn(1.f + expf(-z));
  return inverse(1.f + ptx::ex2(-1.4426950408889634f * z));
}

// The normal distribution at g, where e = e^(-g^2 / 2).  To the left of 0 it is e t P(t),
// t = 1 / (1 + 0.3 |g|), P of degree 7 fitted to the least relative error over |g| <= 14
// (1.5e-7, 3.5e-7 in fp32), so the far tail keeps its digits; to the right 1 minus that.
// kFast = false takes erfc of the math library, for fp32 results.
template <bool kFast>
__device__ __forceinline__ float normal(float g, float e) {
  if constexpr (!kFast) return 0.5f * erfcf(-0.70710678118654752f * g);
  constexpr float c[8] = {1.196293011e-01f, 1.207539588e-01f,
                          9.991349280e-02f, 1.285616159e-01f,
                          -5.368362367e-02f, 2.063534856e-01f,
                          -1.572030634e-01f, 3.567476943e-02f};
  const float t = inverse(fmaf(0.3f, fabsf(g), 1.f));
  float p = c[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) p = fmaf(p, t, c[i]);
  const float q = e * (p * t);
  return g < 0.f ? q : 1.f - q;
}

// a(g), and its derivative where asked for.
//   silu        g s(g),                 s the sigmoid
//   gelu        g F(g),                 F the normal distribution
//   gelu_tanh   g s(2 z),  z = sqrt(2 / pi) (g + 0.044715 g^3): 0.5 (1 + tanh z) is
//               s(2 z), without the difference of two ones at the left
// With a = g s: a' = s + a (1 - s) (2 z)'.
template <bool kDerivative, bool kFast>
__device__ __forceinline__ float activation(float g, int act, float& da) {
  if (act == ACT_GELU) {
    const float e = ptx::ex2(-0.72134752044448170f * (g * g));
    const float f = normal<kFast>(g, e);
    if constexpr (kDerivative) da = fmaf(g, 0.3989422804014327f * e, f);
    return g * f;
  }
  float s, slope;   // slope of the sigmoid's argument
  if (act == ACT_SILU) {
    s = sigmoid<kFast>(g);
    slope = 1.f;
  } else {
    constexpr float k = 1.5957691216057308f;   // 2 sqrt(2 / pi)
    const float g2 = g * g;
    s = sigmoid<kFast>(k * g * fmaf(0.044715f, g2, 1.f));
    // far out the slope's factor is 0, and an infinite slope would make it NaN
    slope = k * fmaf(0.134145f, fminf(g2, 1e6f), 1.f);
  }
  const float a = g * s;
  if constexpr (kDerivative) da = fmaf(a - a * s, slope, s);
  return a;
}

// Calls f with the activation as a compile-time constant, for loops over several values:
// a branch at every value keeps them from running side by side (fp32, silu, 517 x 512 x 1360:
// the backward 68 us with it, 62 without; bf16 hidden gradients, which wait for their loads, 1 %
// slower without).
template <int kAct>
struct Activation {
  static constexpr int value = kAct;
};
template <class F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  if (act == ACT_SILU) f(Activation<ACT_SILU>());
  else if (act == ACT_GELU) f(Activation<ACT_GELU>());
  else f(Activation<ACT_GELU_TANH>());
}

// The upper 24 bits of two or four fp32 values, in memory order: their upper halves
// (bf16 planes), and the bytes below them.  Byte permutations alone: rounding to 24
// bits instead took six instructions a value, and with it the gradient's epilogue
// longer than its products.
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ uint32_t next_bytes(float a, float b, float c, float d) {
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0051),
                     __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0051), 0x5410);
}
// Value i of a pair of upper halves, and its byte, number k of four.  The lowest eight
// bits, of which nothing was kept, repeat that byte: off by at most 2^-15 of the value,
// zeros and infinities are exact.
template <int i, int k>
__device__ __forceinline__ float rejoin(uint32_t halves, uint32_t bytes) {
  return __uint_as_float(
      __byte_perm(halves, bytes, (4 + k) | (4 + k) << 4 | (2 * i) << 8 | (2 * i + 1) << 12));
}

// Eight values from four pairs of halves and two words of bytes.
__device__ __forceinline__ void rejoin8(const uint32_t* halves, const uint32_t* bytes,
                                        float (&f)[8]) {
  f[0] = rejoin<0, 0>(halves[0], bytes[0]);
  f[1] = rejoin<1, 1>(halves[0], bytes[0]);
  f[2] = rejoin<0, 2>(halves[1], bytes[0]);
  f[3] = rejoin<1, 3>(halves[1], bytes[0]);
  f[4] = rejoin<0, 0>(halves[2], bytes[1]);
  f[5] = rejoin<1, 1>(halves[2], bytes[1]);
  f[6] = rejoin<0, 2>(halves[3], bytes[1]);
  f[7] = rejoin<1, 3>(halves[3], bytes[1]);
}

}  // namespace

}  // namespace cpattn
