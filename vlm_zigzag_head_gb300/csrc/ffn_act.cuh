// Activations of the gated feed-forward block and their derivatives.
#pragma once
#include <cuda_bf16.h>

#include "ffn.h"
#include "ptx.cuh"

namespace cpattn {

namespace {

// 1 / (1 + e^-z); e^-z overflows to infinity, whose inverse is 0.
__device__ __forceinline__ float sigmoid(float z) {
  return __fdividef(1.f, 1.f + ptx::ex2(-1.4426950408889634f * z));
}

// a(g), and its derivative where asked for.
//   silu        g s(g),                 s the sigmoid
//   gelu        g F(g),                 F the normal distribution, by erfc so that the
//               far left tail keeps its digits
//   gelu_tanh   g s(2 z),  z = sqrt(2 / pi) (g + 0.044715 g^3): 0.5 (1 + tanh z) is
//               s(2 z), without the difference of two ones at the left
template <bool kDerivative>
__device__ __forceinline__ float activation(float g, int act, float& da) {
  if (act == ACT_GELU) {
    const float f = 0.5f * erfcf(-0.70710678118654752f * g);
    if constexpr (kDerivative)
      da = fmaf(g, 0.3989422804014327f * ptx::ex2(-0.72134752044448170f * g * g), f);
    return g * f;
  }
  float s, slope;   // slope of the sigmoid's argument
  if (act == ACT_SILU) {
    s = sigmoid(g);
    slope = 1.f;
  } else {
    constexpr float k = 1.5957691216057308f;   // 2 sqrt(2 / pi)
    const float g2 = g * g;
    s = sigmoid(k * g * fmaf(0.044715f, g2, 1.f));
    slope = k * fmaf(0.134145f, g2, 1.f);
  }
  if constexpr (kDerivative) da = fmaf(g * s * (1.f - s), slope, s);
  return g * s;
}

// The 24 bits kept of v: a bf16 (rounded to nearest) and the rest in steps of 2^-8 of
// its step.  The sum of bit patterns carries across powers of two.
__device__ __forceinline__ void split24(float v, uint32_t& hi, uint32_t& lo) {
  const uint32_t r = __float_as_uint(v) + 0x80u;   // rounded to 24 bits
  hi = (r + 0x8000u) >> 16;
  lo = ((r - (hi << 16)) >> 8) & 0xffu;
  if (v != v) {
    hi = 0x7fc0u;
    lo = 0u;
  }
}
__device__ __forceinline__ float join24(uint32_t hi, uint32_t lo) {   // lo: any upper bits
  return __uint_as_float((hi << 16) + (uint32_t)((int32_t)(lo << 24) >> 16));
}

}  // namespace

}  // namespace cpattn
