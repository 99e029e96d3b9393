// Modified scores, head size 64, bf16 operands.
#include "tc_fwd_scored.cuh"

namespace cpattn {

cudaError_t launch_fwd_scored_64_bf16(const TcFwdArgs& a, int bias, cudaStream_t st) {
  return launch_fwd_scored_d<64, false>(a, bias, st);
}

}  // namespace cpattn
