// Backward with modified scores, head size 128, bf16 operands.
#include "tc_bwd_scored.cuh"

namespace cpattn {

cudaError_t launch_bwd_scored_128_bf16(const TcBwdArgs& a, int bias, cudaStream_t st) {
  return launch_bwd_scored_d<128, OPS_BF16>(a, bias, st);
}

}  // namespace cpattn
