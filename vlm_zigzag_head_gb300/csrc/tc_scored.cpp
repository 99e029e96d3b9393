// Picks the kernel of a launch with modified scores: one translation unit per
// direction, head size and operand type.
#include "tc.h"

namespace cpattn {

#define CP_SCORED(dir, Args)                                                       \
  cudaError_t launch_##dir##_scored_64_bf16(const Args&, int, cudaStream_t);       \
  cudaError_t launch_##dir##_scored_64_f16(const Args&, int, cudaStream_t);        \
  cudaError_t launch_##dir##_scored_128_bf16(const Args&, int, cudaStream_t);      \
  cudaError_t launch_##dir##_scored_128_f16(const Args&, int, cudaStream_t);
CP_SCORED(fwd, TcFwdArgs)
CP_SCORED(bwd, TcBwdArgs)
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
      (a.f16 && a.op_scales == nullptr))
    return cudaErrorInvalidValue;
  if (bias == SCORE_PLAIN && !(a.score.cap_log2 > 0.f)) return launch_tc_bwd_q128(a, st);
  if (a.d == 64)
    return a.f16 ? launch_bwd_scored_64_f16(a, bias, st) : launch_bwd_scored_64_bf16(a, bias, st);
  if (a.d != 128) return cudaErrorNotSupported;
  return a.f16 ? launch_bwd_scored_128_f16(a, bias, st) : launch_bwd_scored_128_bf16(a, bias, st);
}

}  // namespace cpattn
