// C ABI of the query / key norm with rotation: argument checks, launch shapes
// and the launch sequence.
#include <cuda_runtime.h>

#include <cmath>
#include <string>

#include "../../include/cpattn.h"
#include "entry.h"
#include "norm_rope.h"
#include "rope_desc.h"

using namespace cpattn;

namespace {

struct Setup {
  NormRopeArgs a;
  bool bf16 = false, vec = false;
  int sms = 0;
};

// Everything that does not look at a tensor pointer.
cp_status_t check_desc(const cp_norm_rope_t* p) {
  if (!p) return entry_fail(CP_ERR_INVALID_ARG, "desc is NULL");
  if (p->dtype != CP_F32 && p->dtype != CP_BF16)
    return entry_fail(CP_ERR_DTYPE, "dtype must be CP_F32 or CP_BF16");
  if (p->weight_dtype != CP_F32 && p->weight_dtype != CP_BF16)
    return entry_fail(CP_ERR_DTYPE, "weight_dtype must be CP_F32 or CP_BF16");
  if (p->T < 0 || p->H < 1 || p->H_kv < 1)
    return entry_fail(CP_ERR_INVALID_ARG, "T >= 0, H >= 1, H_kv >= 1");
  if (p->H > (1 << 20) || p->H_kv > (1 << 20))
    return entry_fail(CP_ERR_SHAPE, "at most 2^20 heads");
  if (p->d != 64 && p->d != 128) return entry_fail(CP_ERR_SHAPE, "head_dim must be 64 or 128");
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps))
    return entry_fail(CP_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return rope_check_angles(p);
}

cp_status_t setup(const cp_norm_rope_t* p, const void* q, const void* k, const int32_t* pos,
                  const void* qw, const void* kw, Setup* o) {
  cp_status_t s = check_desc(p);
  if (s != CP_OK) return s;
  o->bf16 = p->dtype == CP_BF16;
  const size_t elem = o->bf16 ? 2 : 4;
  NormRopeArgs& a = o->a;
  if (p->T > 0) {
    if (!q || !k || (!pos && p->rot_dim > 0))
      return entry_fail(CP_ERR_INVALID_ARG, "q, k or positions is NULL");
    if (!aligned_to(q, elem) || !aligned_to(k, elem) || !aligned_to(pos, 4))
      return entry_fail(CP_ERR_ALIGNMENT, "a pointer is not aligned to its element type");
    const size_t wsize = p->weight_dtype == CP_BF16 ? 2 : 4;
    if (!aligned_to(qw, wsize) || !aligned_to(kw, wsize))
      return entry_fail(CP_ERR_ALIGNMENT, "a weight pointer is not aligned to its element type");
  }
  a.x[0] = q;
  a.x[1] = k;
  a.st[0] = p->q_stride_t;
  a.st[1] = p->k_stride_t;
  a.sh[0] = p->q_stride_h;
  a.sh[1] = p->k_stride_h;
  a.heads[0] = p->H;
  a.heads[1] = p->H_kv;
  a.w[0] = qw;
  a.w[1] = kw;
  a.w_bf16 = p->weight_dtype == CP_BF16;
  a.eps = p->eps;
  a.partial = nullptr;
  rope_fill_angles(p, pos, &a);
  // vector loads where every group of four elements lies on a boundary of its size
  o->vec = aligned_to(q, 4 * elem) && aligned_to(k, 4 * elem);
  for (int i = 0; i < 2; ++i) o->vec = o->vec && a.st[i] % 4 == 0 && a.sh[i] % 4 == 0;
  return CP_OK;
}

// The launch shape, once every argument has been checked.
cp_status_t shape_launch(const cp_norm_rope_t* p, Setup* o) {
  int dev = 0;
  ENTRY_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  ENTRY_CUDA(cudaDeviceGetAttribute(&o->sms, cudaDevAttrMultiProcessorCount, dev), "SM count");
  rope_split(p->T, p->H + p->H_kv, p->d, o->sms, &o->a.chunk, &o->a.n_chunks);
  return CP_OK;
}

cp_status_t check_out(const void* p) {
  if (!p) return entry_fail(CP_ERR_INVALID_ARG, "an output or gradient pointer is NULL");
  if (!aligned_to(p, 16))
    return entry_fail(CP_ERR_ALIGNMENT, "outputs and gradients must be 16-byte aligned");
  return CP_OK;
}

}  // namespace

extern "C" {

cp_status_t cp_qk_norm_rope_fwd(const cp_norm_rope_t* desc, const void* q, const void* k,
                                const int32_t* positions, const void* q_weight,
                                const void* k_weight, void* q_out, void* k_out, void* stream) {
  ENTRY_TRY
  Setup s;
  cp_status_t e = setup(desc, q, k, positions, q_weight, k_weight, &s);
  if (e != CP_OK) return e;
  if (desc->T == 0) return CP_OK;
  if ((e = check_out(q_out)) != CP_OK || (e = check_out(k_out)) != CP_OK ||
      (e = shape_launch(desc, &s)) != CP_OK)
    return e;
  s.a.y[0] = q_out;
  s.a.y[1] = k_out;
  ENTRY_CUDA(launch_norm_rope_fwd(s.a, s.bf16, desc->d, desc->interleaved != 0, s.vec,
                                  static_cast<cudaStream_t>(stream)),
             "query / key norm with rotation");
  return CP_OK;
  ENTRY_CATCH
}

size_t cp_qk_norm_rope_bwd_workspace_size(const cp_norm_rope_t* desc) {
  if (!desc || desc->d < 1) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return (size_t)norm_rope_bwd_max_blocks(sms) * 2 * desc->d * sizeof(float);
}

cp_status_t cp_qk_norm_rope_bwd(const cp_norm_rope_t* desc, const void* q, const void* k,
                                const int32_t* positions, const void* q_weight,
                                const void* k_weight, const void* dq_out, const void* dk_out,
                                void* dq, void* dk, float* dq_weight, float* dk_weight,
                                void* workspace, size_t ws_bytes, void* stream) {
  ENTRY_TRY
  Setup s;
  cp_status_t e = setup(desc, q, k, positions, q_weight, k_weight, &s);
  if (e != CP_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool weights = dq_weight || dk_weight;
  if (!aligned_to(dq_weight, 4) || !aligned_to(dk_weight, 4))
    return entry_fail(CP_ERR_ALIGNMENT, "a weight gradient is not aligned to its element type");
  if (desc->T == 0) {   // no rows: the weights' gradients are zero
    for (float* p : {dq_weight, dk_weight})
      if (p) ENTRY_CUDA(cudaMemsetAsync(p, 0, desc->d * sizeof(float), st), "clear gradients");
    return CP_OK;
  }
  for (const void* p : {dq_out, dk_out, (const void*)dq, (const void*)dk})
    if ((e = check_out(p)) != CP_OK) return e;
  if (weights && !aligned_to(workspace, 256))
    return entry_fail(CP_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  if (weights && !workspace) return entry_fail(CP_ERR_WORKSPACE, "workspace is NULL");
  if ((e = shape_launch(desc, &s)) != CP_OK) return e;
  const int blocks = norm_rope_bwd_blocks(desc->T, s.a.n_chunks, s.sms);
  if (weights) {
    if (ws_bytes < (size_t)blocks * 2 * desc->d * sizeof(float))
      return entry_fail(CP_ERR_WORKSPACE,
                        "workspace smaller than cp_qk_norm_rope_bwd_workspace_size()");
    s.a.partial = static_cast<float*>(workspace);
  }
  s.a.dy[0] = dq_out;
  s.a.dy[1] = dk_out;
  s.a.y[0] = dq;
  s.a.y[1] = dk;
  ENTRY_CUDA(launch_norm_rope_bwd(s.a, s.bf16, desc->d, desc->interleaved != 0, s.vec, blocks, st),
             "gradient of the query / key norm with rotation");
  if (weights)
    ENTRY_CUDA(launch_norm_rope_dw(s.a.partial, blocks, desc->d, dq_weight, dk_weight, st),
               "norm weight gradients");
  return CP_OK;
  ENTRY_CATCH
}

}  // extern "C"
