// Launches of the backward with modified scores (tc_bwd_q128.cuh) for one head size.
#pragma once
#include "tc_bwd_q128.cuh"

namespace cpattn {

// One instantiation serves key tiles of one CTA and shared ones: the epilogue asks
// add_dkdv.  kOps: OPS_BF16, or OPS_ITEM where some samples may take f16.
template <int D, int kOps>
cudaError_t launch_bwd_scored_d(const TcBwdArgs& a, int bias, cudaStream_t st) {
  if (a.score.cap_log2 > 0.f) {
    if (bias == SCORE_SLOPES) return launch_q128<D, kOps, true, true, SCORE_SLOPES>(a, st);
    if (bias == SCORE_TABLE) return launch_q128<D, kOps, true, true, SCORE_TABLE>(a, st);
    return launch_q128<D, kOps, true, true, SCORE_PLAIN>(a, st);
  }
  if (bias == SCORE_SLOPES) return launch_q128<D, kOps, true, false, SCORE_SLOPES>(a, st);
  if (bias == SCORE_TABLE) return launch_q128<D, kOps, true, false, SCORE_TABLE>(a, st);
  if constexpr (kOps == OPS_ITEM)
    return a.add_dkdv ? launch_q128<D, kOps, true, false, SCORE_PLAIN>(a, st)
                      : launch_q128<D, kOps, false, false, SCORE_PLAIN>(a, st);
  return cudaErrorInvalidValue;   // plain scores in bf16: launch_tc_bwd_q128
}

}  // namespace cpattn
