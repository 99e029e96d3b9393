// The tensor-core backward with plain scores (the kernel: tc_bwd_q128.cuh).
#include "tc_bwd_q128.cuh"

namespace cpattn {

namespace {

template <int D, int kOps>
cudaError_t launch_plain(const TcBwdArgs& a, cudaStream_t st) {
  return a.add_dkdv ? launch_q128<D, kOps, true, false, SCORE_PLAIN>(a, st)
                    : launch_q128<D, kOps, false, false, SCORE_PLAIN>(a, st);
}

}  // namespace

cudaError_t launch_tc_bwd_q128(const TcBwdArgs& a, cudaStream_t st) {
  if (a.n_items == 0) return cudaSuccess;
  if (a.runs == nullptr) return cudaErrorInvalidValue;   // all-steps items only
  if (a.kv_split < 1 || (a.H / a.Hkv) % a.kv_split != 0) return cudaErrorInvalidValue;
  if (a.f16 && a.op_scales == nullptr) return cudaErrorInvalidValue;
  if (a.d == 128)
    return a.f16 ? launch_plain<128, OPS_F16>(a, st) : launch_plain<128, OPS_BF16>(a, st);
  if (a.d != 64) return cudaErrorNotSupported;
  return a.f16 ? launch_plain<64, OPS_F16>(a, st) : launch_plain<64, OPS_BF16>(a, st);
}

}  // namespace cpattn
