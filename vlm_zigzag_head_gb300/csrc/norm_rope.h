// Norm of query and key heads with the position rotation (kernel launchers).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace cpattn {

constexpr int kRopeMaxAxes = 4;

struct NormRopeArgs {
  // [T][heads][d] inputs with token and head strides in elements (the last
  // dimension is contiguous): q, k forward; the same q, k backward
  const void* x[2];
  int64_t st[2], sh[2];
  const void* dy[2];        // backward: gradients of the outputs, contiguous
  void* y[2];               // forward: outputs; backward: gradients of q, k; contiguous
  int heads[2];             // query heads, KV heads
  const void* w[2];         // [d] norm weights (nullable: ones)
  bool w_bf16;
  const int32_t* pos;       // [n_axes][T]
  int sec_end[kRopeMaxAxes];   // rotated pairs of axes 0..a: pairs below sec_end[a]
  int n_axes;
  int64_t T;
  int rot;                  // rotated elements of each head (multiple of 16, <= d)
  float eps;
  int chunk;                // heads (queries and keys counted together) one warp takes
  int n_chunks;
  float* partial;           // backward: [blocks][2][d] partial weight gradients (nullable)
  // turns of pair p per position, as a fraction of 2^64
  uint64_t freq[64];
};

// Blocks of the backward launch (rows of `partial`), and the most there are.
int norm_rope_bwd_blocks(int64_t T, int n_chunks, int sms);
int norm_rope_bwd_max_blocks(int sms);
// Heads per warp and the number of such chunks.
void norm_rope_split(int64_t T, int heads, int d, int sms, int* chunk, int* n_chunks);

// vec: every group of four elements lies on a boundary of its size (vector
// loads), else element loads.
cudaError_t launch_norm_rope_fwd(const NormRopeArgs& a, bool bf16, int d, bool interleaved,
                                 bool vec, cudaStream_t st);
cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, bool bf16, int d, bool interleaved,
                                 bool vec, int blocks, cudaStream_t st);
// dw[s][e] = sum of partial[b][s][e] over the blocks, in a fixed order.
cudaError_t launch_norm_rope_dw(const float* partial, int blocks, int d, float* dqw, float* dkw,
                                cudaStream_t st);

}  // namespace cpattn
