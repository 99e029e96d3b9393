// The tensor-core forward with plain scores (the kernel: tc_fwd.cuh).
#include "tc_fwd.cuh"

namespace cpattn {

cudaError_t launch_tc_fwd(const TcFwdArgs& a, cudaStream_t st) {
  if (a.n_items == 0) return cudaSuccess;
  if (a.f16_pv) {
    if (a.op_scales == nullptr) return cudaErrorInvalidValue;
    return a.d == 64 ? launch_d<64, true, false, SCORE_PLAIN>(a, st)
                     : launch_d<128, true, false, SCORE_PLAIN>(a, st);
  }
  return a.d == 64 ? launch_d<64, false, false, SCORE_PLAIN>(a, st)
                   : launch_d<128, false, false, SCORE_PLAIN>(a, st);
}

}  // namespace cpattn
