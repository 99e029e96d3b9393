// Rotation of query and key heads by their positions (kernel launchers).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace cpattn {

constexpr int kRopeMaxAxes = 4;

// What the angles of a token are worked out from.
struct RopeAngles {
  const int32_t* pos;       // [n_axes][T]
  int sec_end[kRopeMaxAxes];   // rotated pairs of axes 0..a: pairs below sec_end[a]
  int n_axes;
  int64_t T;
  int rot;                  // rotated elements of each head (multiple of 16, <= d)
  // turns of pair p per position, as a fraction of 2^64
  uint64_t freq[64];
};

struct RopeArgs : RopeAngles {
  // [T][heads][d] inputs and outputs with token and head strides in elements (the
  // last dimension is contiguous): queries, keys
  const void* x[2];
  int64_t st[2], sh[2];
  void* y[2];
  int64_t yst[2], ysh[2];
  int heads[2];             // query heads, KV heads
  float amp, sin_amp;       // factors of the cosines and of the sines
  int chunk;                // heads (queries and keys counted together) one warp takes
  int n_chunks;
};

// vec: every group of four elements lies on a boundary of its size (vector
// accesses), else element accesses.  y may be x (in place).
cudaError_t launch_rope(const RopeArgs& a, bool bf16, int d, bool interleaved, bool vec,
                        cudaStream_t st);

// Heads per warp and the number of such chunks.
void rope_split(int64_t T, int heads, int d, int sms, int* chunk, int* n_chunks);

}  // namespace cpattn
