// C ABI of the rotation of query and key heads: argument checks and the launch.
#include <cuda_runtime.h>

#include <cmath>
#include <string>

#include "../../include/cpattn.h"
#include "entry.h"
#include "rope.h"
#include "rope_desc.h"

using namespace cpattn;

namespace {

cp_status_t check_desc(const cp_rope_t* p) {
  if (!p) return entry_fail(CP_ERR_INVALID_ARG, "desc is NULL");
  if (p->dtype != CP_F32 && p->dtype != CP_BF16)
    return entry_fail(CP_ERR_DTYPE, "dtype must be CP_F32 or CP_BF16");
  if (p->T < 0 || p->H < 1 || p->H_kv < 1)
    return entry_fail(CP_ERR_INVALID_ARG, "T >= 0, H >= 1, H_kv >= 1");
  if (p->H > (1 << 20) || p->H_kv > (1 << 20))
    return entry_fail(CP_ERR_SHAPE, "at most 2^20 heads");
  if (p->d != 64 && p->d != 128) return entry_fail(CP_ERR_SHAPE, "head_dim must be 64 or 128");
  if (!std::isfinite(p->amplitude))
    return entry_fail(CP_ERR_INVALID_ARG, "amplitude must be finite");
  return rope_check_angles(p);
}

cp_status_t rotate(const cp_rope_t* p, const void* q, const void* k, const int32_t* pos, void* qo,
                   void* ko, float sign, void* stream) {
  cp_status_t s = check_desc(p);
  if (s != CP_OK) return s;
  if (p->T == 0) return CP_OK;
  const bool bf16 = p->dtype == CP_BF16;
  const size_t elem = bf16 ? 2 : 4;
  if (!q || !k || !qo || !ko || (!pos && p->rot_dim > 0))
    return entry_fail(CP_ERR_INVALID_ARG, "a tensor or positions is NULL");
  RopeArgs a;
  a.x[0] = q;
  a.x[1] = k;
  a.y[0] = qo;
  a.y[1] = ko;
  a.st[0] = p->q_stride_t;
  a.st[1] = p->k_stride_t;
  a.sh[0] = p->q_stride_h;
  a.sh[1] = p->k_stride_h;
  a.yst[0] = p->q_out_stride_t;
  a.yst[1] = p->k_out_stride_t;
  a.ysh[0] = p->q_out_stride_h;
  a.ysh[1] = p->k_out_stride_h;
  a.heads[0] = p->H;
  a.heads[1] = p->H_kv;
  bool vec = true;
  for (int i = 0; i < 2; ++i) {
    if (!aligned_to(a.x[i], elem) || !aligned_to(a.y[i], elem))
      return entry_fail(CP_ERR_ALIGNMENT, "a pointer is not aligned to its element type");
    if (a.x[i] == a.y[i] && ((p->T > 1 && a.st[i] != a.yst[i]) ||
                             (a.heads[i] > 1 && a.sh[i] != a.ysh[i])))
      return entry_fail(CP_ERR_INVALID_ARG, "an output in place must have its input's strides");
    if ((p->T > 1 && a.yst[i] == 0) || (a.heads[i] > 1 && a.ysh[i] == 0))
      return entry_fail(CP_ERR_INVALID_ARG, "an output's rows must not share memory");
    // vector accesses where every group of four elements lies on a boundary of its size
    vec = vec && aligned_to(a.x[i], 4 * elem) && aligned_to(a.y[i], 4 * elem) &&
          a.st[i] % 4 == 0 && a.sh[i] % 4 == 0 && a.yst[i] % 4 == 0 && a.ysh[i] % 4 == 0;
  }
  if (!aligned_to(pos, 4))
    return entry_fail(CP_ERR_ALIGNMENT, "a pointer is not aligned to its element type");
  a.amp = p->amplitude;
  a.sin_amp = sign * p->amplitude;
  rope_fill_angles(p, pos, &a);
  int dev = 0, sms = 0;
  ENTRY_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  ENTRY_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "SM count");
  rope_split(p->T, p->H + p->H_kv, p->d, sms, &a.chunk, &a.n_chunks);
  ENTRY_CUDA(launch_rope(a, bf16, p->d, p->interleaved != 0, vec,
                         static_cast<cudaStream_t>(stream)),
             "rotation of heads");
  return CP_OK;
}

}  // namespace

extern "C" {

cp_status_t cp_rope_fwd(const cp_rope_t* desc, const void* q, const void* k,
                        const int32_t* positions, void* q_out, void* k_out, void* stream) {
  ENTRY_TRY
  return rotate(desc, q, k, positions, q_out, k_out, 1.f, stream);
  ENTRY_CATCH
}

cp_status_t cp_rope_bwd(const cp_rope_t* desc, const void* dq_out, const void* dk_out,
                        const int32_t* positions, void* dq, void* dk, void* stream) {
  ENTRY_TRY
  return rotate(desc, dq_out, dk_out, positions, dq, dk, -1.f, stream);
  ENTRY_CATCH
}

}  // extern "C"
