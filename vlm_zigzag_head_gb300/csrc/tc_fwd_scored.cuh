// Launches of the forward with modified scores (tc_fwd.cuh) for one head size.
#pragma once
#include "tc_fwd.cuh"

namespace cpattn {

template <int D, bool kF16P>
cudaError_t launch_fwd_scored_d(const TcFwdArgs& a, int bias, cudaStream_t st) {
  if (a.score.cap_log2 > 0.f) {
    if (bias == SCORE_SLOPES) return launch_d<D, kF16P, true, SCORE_SLOPES>(a, st);
    if (bias == SCORE_TABLE) return launch_d<D, kF16P, true, SCORE_TABLE>(a, st);
    return launch_d<D, kF16P, true, SCORE_PLAIN>(a, st);
  }
  if (bias == SCORE_SLOPES) return launch_d<D, kF16P, false, SCORE_SLOPES>(a, st);
  if (bias == SCORE_TABLE) return launch_d<D, kF16P, false, SCORE_TABLE>(a, st);
  return cudaErrorInvalidValue;   // plain scores: launch_tc_fwd
}

}  // namespace cpattn
