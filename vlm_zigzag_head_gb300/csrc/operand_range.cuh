// Operand types of the scored backward, chosen for each sample and KV head.
//
// dS = P (dP - D) is rounded to 16 bits as the operand of dQ and dK.  bf16 has the range
// for any gradient but 8 bits, and in a short sample, where few terms meet, its half
// step shows beside the results' own (dq up to 2.1 of their rounding, 1.3 on average,
// over 120 packings of up to 1024 tokens; f16: 1.5 and 1.06).  f16 has three bits more
// and 30 binades: dS times one power of two, from
//     |dS_ij| <= P_ij 2 |dout_i| max_j |v_j|   (2-norms),
// which an ordinary dS / P stays about 2^4.5 below.  With the largest at 2^15, dS keeps
// f16's 11 bits down to P |dout_i| of 2^-24 of its largest, and at least bf16's 8 to
// 2^-27.  So a sample takes f16 where
//   - it has at most kF16Tokens tokens (P is 2^-10 or more on average), and
//   - its non-zero rows of dout lie within 2^8 of one another (a masked or weighted loss
//     may have them apart: then bf16 keeps the bits of the small ones), and
//   - all exponents lie in the middle of fp32's range.
// It depends on nothing outside the sample and the heads that share the KV head, so a
// sample gets the gradients that it gets alone.
#pragma once
#include <stdint.h>

#include "tc.h"

namespace cpattn {

struct Operands {
  int f16;             // K, Q (scaled copies) and dS are f16; else bf16 as they are
  int eq, ek;          // copies of Q and K: x 2^-e
  float qk_mul;        // S = (K Q^T) qk_mul
  float ds_inv;        // dS as an operand: dS ds_inv (below 2^15)
  float dq_mul, dk_mul;   // dQ = (dS K) dq_mul, dK = (dS^T Q) dk_mul
};

__device__ __forceinline__ int range_exp(uint32_t bits) { return (int)(bits >> 23) - 126; }
__device__ __forceinline__ float range_pow2(int k) { return __int_as_float((k + 127) << 23); }

__device__ __forceinline__ Operands choose_operands(const OperandRange& r) {
  constexpr float kLeast = 7.9e-31f, kMost = 1.26e30f;   // squares: 2^-100 and 2^100
  Operands o{0, 0, 0, 1.f, 1.f, 1.f, 1.f};
  const float v2 = __uint_as_float(r.v2), g2 = __uint_as_float(r.g2);
  const float least = __uint_as_float(~r.g2_least);   // (comparisons with NaN are false)
  if (!(v2 >= kLeast && v2 <= kMost && g2 >= kLeast && g2 <= kMost &&
        least >= g2 * (1.f / 65536.f)))
    return o;
  // the largest magnitude times 2^-e lies in [2^14, 2^15)
  const int eq = r.q >> 23 ? range_exp(r.q) - 15 : 0, ek = r.k >> 23 ? range_exp(r.k) - 15 : 0;
  // 2 sqrt(v2 g2) < 2^(1 + ceil((e_v + e_g) / 2))
  const int es = 1 + ((range_exp(r.v2) + range_exp(r.g2) + 1) >> 1) - 15;
  if (abs(eq) > 60 || abs(ek) > 60 || abs(es) > 60) return o;
  o.f16 = 1;
  o.eq = eq;
  o.ek = ek;
  o.qk_mul = range_pow2(eq + ek);
  o.ds_inv = range_pow2(-es);
  o.dq_mul = range_pow2(es + ek);
  o.dk_mul = range_pow2(es + eq);
  return o;
}

}  // namespace cpattn
