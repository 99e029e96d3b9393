// Learned bias by bucket, laid out by distance for the attention kernels, and
// its gradient summed back.  Both are a few KB a head: bound by the launch.
#include <cuda_bf16.h>

#include "scored.h"

namespace cpattn {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    expand_bias_kernel(const void* bias, int bf16, int64_t sh, int64_t sb, const int32_t* buckets,
                       int n_dist, float mul, float* table, int mid, int pitch) {
  const int h = blockIdx.y;
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < pitch; i += gridDim.x * kThreads) {
    const int s = i - mid;
    const int64_t at = h * sh + buckets[min(s < 0 ? -s : s, n_dist - 1)] * sb;
    const float b = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(bias)[at])
                         : static_cast<const float*>(bias)[at];
    table[(int64_t)h * pitch + i] = b <= -1e37f ? -INFINITY : b * mul;
  }
}

// One block per head, one warp per bucket at a time; lanes take the distances
// 32 apart and meet in a fixed order.
__global__ void __launch_bounds__(kThreads)
    reduce_dbias_kernel(const float* dtable, const int32_t* buckets, int n_dist, int n_buckets,
                        float* dbias) {
  const int h = blockIdx.x, lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < n_buckets; b += kThreads / 32) {
    float v = 0.f;
    for (int t = lane; t < n_dist; t += 32)
      if (buckets[t] == b) v += dtable[(int64_t)h * n_dist + t];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) dbias[(int64_t)h * n_buckets + b] = v;
  }
}

}  // namespace

cudaError_t launch_expand_bias(const void* bias, bool bf16, int64_t stride_h, int64_t stride_b,
                               const int32_t* buckets, int n_dist, int H, float mul, float* table,
                               int mid, int pitch, cudaStream_t st) {
  expand_bias_kernel<<<dim3((pitch + kThreads - 1) / kThreads, H), kThreads, 0, st>>>(
      bias, bf16 ? 1 : 0, stride_h, stride_b, buckets, n_dist, mul, table, mid, pitch);
  return cudaGetLastError();
}

cudaError_t launch_reduce_dbias(const float* dtable, const int32_t* buckets, int n_dist,
                                int n_buckets, int H, float* dbias, cudaStream_t st) {
  reduce_dbias_kernel<<<H, kThreads, 0, st>>>(dtable, buckets, n_dist, n_buckets, dbias);
  return cudaGetLastError();
}

}  // namespace cpattn
