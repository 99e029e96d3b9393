// Backward with modified scores, head size 64, f16 operands for the samples whose range allows them.
#include "tc_bwd_scored.cuh"

namespace cpattn {

cudaError_t launch_bwd_scored_64_item(const TcBwdArgs& a, int bias, cudaStream_t st) {
  return launch_bwd_scored_d<64, OPS_ITEM>(a, bias, st);
}

}  // namespace cpattn
