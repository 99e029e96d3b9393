// Modified scores, head size 128, bf16 operands.
#include "tc_fwd_scored.cuh"

namespace cpattn {

cudaError_t launch_fwd_scored_128_bf16(const TcFwdArgs& a, int bias, cudaStream_t st) {
  return launch_fwd_scored_d<128, false>(a, bias, st);
}

}  // namespace cpattn
