// Picks the kernel of a launch with modified scores: one translation unit per
// direction, head size and operand type.
#include "tc.h"

#include <algorithm>
#include <cmath>

namespace cpattn {

void fill_cap_polynomial(ScoreArgs* s, float scale_log2) {
  // |z| up to which the terms from this one on are below 3e-7
  constexpr float without[4] = {9e-4f, 0.038f, 0.13f, 0.26f};
  const float in = scale_log2 * s->inv_cap_log2;
  double a = scale_log2;
  float z = kCapPolyRange;
  s->cap_k[0] = scale_log2;
  for (int i = 0; i < 4; ++i) {
    a *= (double)in * in;
    const float k = (float)(a * kCapPoly[i]);
    const bool normal = std::fabs(k) >= 1e-36f && std::fabs(k) <= 1e36f;
    if (!normal) z = std::min(z, without[i]);
    s->cap_k[i + 1] = normal ? k : 0.f;
  }
  s->cap_reach = z / in;
}

#define CP_SCORED(name, Args) cudaError_t launch_##name(const Args&, int, cudaStream_t);
CP_SCORED(fwd_scored_64_bf16, TcFwdArgs)
CP_SCORED(fwd_scored_64_f16, TcFwdArgs)
CP_SCORED(fwd_scored_128_bf16, TcFwdArgs)
CP_SCORED(fwd_scored_128_f16, TcFwdArgs)
CP_SCORED(bwd_scored_64_bf16, TcBwdArgs)
CP_SCORED(bwd_scored_64_item, TcBwdArgs)
CP_SCORED(bwd_scored_128_bf16, TcBwdArgs)
CP_SCORED(bwd_scored_128_item, TcBwdArgs)
#undef CP_SCORED

cudaError_t launch_tc_fwd_scored(const TcFwdArgs& a, int bias, cudaStream_t st) {
  if (a.n_items == 0) return cudaSuccess;
  if (a.f16_pv && a.op_scales == nullptr) return cudaErrorInvalidValue;
  if (bias == SCORE_PLAIN && !(a.score.cap_log2 > 0.f)) return launch_tc_fwd(a, st);
  if (a.d == 64)
    return a.f16_pv ? launch_fwd_scored_64_f16(a, bias, st) : launch_fwd_scored_64_bf16(a, bias, st);
  return a.f16_pv ? launch_fwd_scored_128_f16(a, bias, st) : launch_fwd_scored_128_bf16(a, bias, st);
}

cudaError_t launch_tc_bwd_scored(const TcBwdArgs& a, int bias, cudaStream_t st) {
  if (a.n_items == 0) return cudaSuccess;
  if (a.runs == nullptr || a.kv_split < 1 || (a.H / a.Hkv) % a.kv_split != 0 ||
      a.f16)   // one choice for all items: the plain kernels'
    return cudaErrorInvalidValue;
  const bool item = a.ranges != nullptr;
  if (!item && bias == SCORE_PLAIN && !(a.score.cap_log2 > 0.f)) return launch_tc_bwd_q128(a, st);
  if (a.d == 64)
    return item ? launch_bwd_scored_64_item(a, bias, st) : launch_bwd_scored_64_bf16(a, bias, st);
  if (a.d != 128) return cudaErrorNotSupported;
  return item ? launch_bwd_scored_128_item(a, bias, st) : launch_bwd_scored_128_bf16(a, bias, st);
}

}  // namespace cpattn
