// Modified scores, head size 64, f16 operands.
#include "tc_bwd_scored.cuh"

namespace cpattn {

cudaError_t launch_bwd_scored_64_f16(const TcBwdArgs& a, int bias, cudaStream_t st) {
  return launch_bwd_scored_d<64, true>(a, bias, st);
}

}  // namespace cpattn
