// Modified scores, head size 128, f16 operands.
#include "tc_fwd_scored.cuh"

namespace cpattn {

cudaError_t launch_fwd_scored_128_f16(const TcFwdArgs& a, int bias, cudaStream_t st) {
  return launch_fwd_scored_d<128, true>(a, bias, st);
}

}  // namespace cpattn
