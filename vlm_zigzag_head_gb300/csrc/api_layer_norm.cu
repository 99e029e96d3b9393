// C ABI of the layer norm: argument checks, launch shapes and the launch sequence.
#include <cuda_runtime.h>

#include <cmath>
#include <string>

#include "../../include/cpattn.h"
#include "entry.h"
#include "layer_norm.h"

using namespace cpattn;

namespace {

cp_status_t check_desc(const cp_layer_norm_t* p) {
  if (!p) return entry_fail(CP_ERR_INVALID_ARG, "desc is NULL");
  if (p->dtype != CP_F32 && p->dtype != CP_BF16)
    return entry_fail(CP_ERR_DTYPE, "dtype must be CP_F32 or CP_BF16");
  if (p->weight_dtype != CP_F32 && p->weight_dtype != CP_BF16)
    return entry_fail(CP_ERR_DTYPE, "weight_dtype must be CP_F32 or CP_BF16");
  if (p->T < 0) return entry_fail(CP_ERR_INVALID_ARG, "T >= 0");
  if (p->D < 1 || p->D > kLayerNormMaxWidth)
    return entry_fail(CP_ERR_SHAPE, "D must be in [1, 16384]");
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps))
    return entry_fail(CP_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return CP_OK;
}

// A [D] weight or bias.
bool weight_ok(const cp_layer_norm_t* p, const void* w) {
  return aligned_to(w, p->weight_dtype == CP_BF16 ? 2 : 4);
}

void fill(const cp_layer_norm_t* p, const void* x, const void* w, const void* b,
          LayerNormArgs* a) {
  a->x = x;
  a->x_stride = p->x_stride;
  a->dy = nullptr;
  a->dy_stride = p->dy_stride;
  a->w = w;
  a->b = b;
  a->w_bf16 = p->weight_dtype == CP_BF16;
  a->y = nullptr;
  a->mean = a->rstd = a->partial = nullptr;
  a->T = p->T;
  a->D = p->D;
  a->eps = p->eps;
  a->inv_D = 1.f / (float)p->D;
}

}  // namespace

extern "C" {

cp_status_t cp_layer_norm_fwd(const cp_layer_norm_t* desc, const void* x, const void* weight,
                              const void* bias, void* y, float* mean, float* rstd, void* stream) {
  ENTRY_TRY
  cp_status_t e = check_desc(desc);
  if (e != CP_OK) return e;
  if (desc->T == 0) return CP_OK;
  const bool bf16 = desc->dtype == CP_BF16;
  const size_t elem = bf16 ? 2 : 4;
  if (!x || !y) return entry_fail(CP_ERR_INVALID_ARG, "x or y is NULL");
  if (!aligned_to(x, elem) || !weight_ok(desc, weight) || !weight_ok(desc, bias) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return entry_fail(CP_ERR_ALIGNMENT, "a pointer is not aligned to its element type");
  if (!aligned_to(y, 16)) return entry_fail(CP_ERR_ALIGNMENT, "y must be 16-byte aligned");
  LayerNormArgs a;
  fill(desc, x, weight, bias, &a);
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  const bool vec = aligned_to(x, 16) && (desc->T == 1 || desc->x_stride * elem % 16 == 0) &&
                   desc->D * elem % 16 == 0 && aligned_to(weight, 16) && aligned_to(bias, 16);
  int dev = 0, sms = 0;
  ENTRY_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  ENTRY_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "SM count");
  ENTRY_CUDA(launch_layer_norm_fwd(a, bf16, vec, sms, static_cast<cudaStream_t>(stream)),
             "layer norm");
  return CP_OK;
  ENTRY_CATCH
}

size_t cp_layer_norm_bwd_workspace_size(const cp_layer_norm_t* desc) {
  if (check_desc(desc) != CP_OK) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  const int blocks = layer_norm_bwd_blocks(desc->T, desc->D, desc->dtype == CP_BF16, sms);
  return (size_t)blocks * 2 * desc->D * sizeof(float);
}

cp_status_t cp_layer_norm_bwd(const cp_layer_norm_t* desc, const void* x, const void* dy,
                              const void* weight, const float* mean, const float* rstd, void* dx,
                              float* dweight, float* dbias, void* workspace, size_t ws_bytes,
                              void* stream) {
  ENTRY_TRY
  cp_status_t e = check_desc(desc);
  if (e != CP_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool sums = dweight || dbias;
  if (!aligned_to(dweight, 4) || !aligned_to(dbias, 4))
    return entry_fail(CP_ERR_ALIGNMENT, "a weight gradient is not aligned to its element type");
  if (desc->T == 0) {   // no rows: the gradients are zero
    for (float* p : {dweight, dbias})
      if (p) ENTRY_CUDA(cudaMemsetAsync(p, 0, desc->D * sizeof(float), st), "clear gradients");
    return CP_OK;
  }
  const bool bf16 = desc->dtype == CP_BF16;
  const size_t elem = bf16 ? 2 : 4;
  if (!x || !dy || !mean || !rstd)
    return entry_fail(CP_ERR_INVALID_ARG, "x, dy, mean or rstd is NULL");
  if (!aligned_to(x, elem) || !aligned_to(dy, elem) || !weight_ok(desc, weight) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return entry_fail(CP_ERR_ALIGNMENT, "a pointer is not aligned to its element type");
  if (!aligned_to(dx, 16)) return entry_fail(CP_ERR_ALIGNMENT, "dx must be 16-byte aligned");
  if (!dx && !sums) return CP_OK;   // nothing is wanted
  if (sums && !workspace) return entry_fail(CP_ERR_WORKSPACE, "workspace is NULL");
  if (sums && !aligned_to(workspace, 256))
    return entry_fail(CP_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  int dev = 0, sms = 0;
  ENTRY_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  ENTRY_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "SM count");
  const int blocks = layer_norm_bwd_blocks(desc->T, desc->D, bf16, sms);
  LayerNormArgs a;
  fill(desc, x, weight, nullptr, &a);
  if (sums) {
    if (ws_bytes < (size_t)blocks * 2 * desc->D * sizeof(float))
      return entry_fail(CP_ERR_WORKSPACE,
                        "workspace smaller than cp_layer_norm_bwd_workspace_size()");
    a.partial = static_cast<float*>(workspace);
  }
  a.dy = dy;
  a.y = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  const bool one = desc->T == 1;
  const bool vec = aligned_to(x, 16) && aligned_to(dy, 16) &&
                   (one || (desc->x_stride * elem % 16 == 0 && desc->dy_stride * elem % 16 == 0)) &&
                   desc->D * elem % 16 == 0 && aligned_to(weight, 16);
  ENTRY_CUDA(launch_layer_norm_bwd(a, bf16, vec, blocks, st), "gradient of the layer norm");
  if (sums)
    ENTRY_CUDA(launch_layer_norm_dw(a.partial, blocks, desc->D, dweight, dbias, st),
               "layer norm weight gradients");
  return CP_OK;
  ENTRY_CATCH
}

}  // extern "C"
