// Layer norm of token rows and its gradient (kernel launchers).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace cpattn {

constexpr int kLayerNormMaxWidth = 16384;

struct LayerNormArgs {
  const void* x;            // [T][D], row stride x_stride elements
  int64_t x_stride;
  const void* dy;           // backward: [T][D], row stride dy_stride elements
  int64_t dy_stride;
  const void* w;            // [D], nullable: ones
  const void* b;            // [D], nullable: zeros
  bool w_bf16;              // type of w and b
  void* y;                  // forward: output; backward: gradient of x (nullable); contiguous
  float* mean;              // [T]; forward: written where not null; backward: read
  float* rstd;
  float* partial;           // backward: [blocks][2][D] partial sums of dw, db (nullable)
  int64_t T;
  int D;
  float eps, inv_D;
};

// Blocks of the backward launch (rows of `partial`).
int layer_norm_bwd_blocks(int64_t T, int D, bool bf16, int sms);

// vec: rows, weights and outputs lie on 16-byte boundaries and D is whole 16-byte
// pieces (vector loads), else element loads.
cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, bool bf16, bool vec, int sms,
                                  cudaStream_t st);
cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, bool bf16, bool vec, int blocks,
                                  cudaStream_t st);
// dw[e], db[e]: sums of partial[b][0][e], partial[b][1][e] over the blocks, in a fixed order.
cudaError_t launch_layer_norm_dw(const float* partial, int blocks, int D, float* dw, float* db,
                                 cudaStream_t st);

}  // namespace cpattn
