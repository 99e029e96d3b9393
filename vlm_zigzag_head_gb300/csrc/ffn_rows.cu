// The gated feed-forward block for up to eight rows (decoding: a token of each request).
//
// Bound by the weights, which are read once: 6 D F bytes in bf16.  A CTA takes 16 rows
// of each of two matrices (16 hidden units of gate and up, or 32 output columns),
// which are the M side of mma.sync; the eight tokens are its N side.  (The tiles of 256
// rows of the large products take 41 us for one token, 2048 x 6144; this takes 12 from
// memory and 11 where L2 holds the weights, whose bytes are 11.3 at a copy's rate.  From
// nine tokens on the older matrix instructions are what bounds it: 83 us for 16 tokens,
// 4096 x 12288, where ffn_tokens.cu takes 54.)  Two launches, the second's first loads in
// flight while the first ends.
//
// Operands go from memory straight into fragments: k may be permuted as long as both
// operands agree, so a lane takes 16 consecutive bytes of a row, eight k, as its
// fragments of two MMAs.  The warps of a CTA, and the CTAs of a cluster where there are
// too few rows of weights to fill the GPU, share k; their sums meet in shared memory in
// a fixed order.
#include <cuda_bf16.h>

#include "ffn.h"
#include "ffn_act.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 64;      // k of one step of a warp: 128 bytes of a row
constexpr int kResident = 4;   // CTAs an SM holds

__device__ __forceinline__ uint4 load_weight(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float peer_load(const float* p, int rank) {   // of another CTA
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

template <bool kGlu>
__global__ void __launch_bounds__(kThreads, kResident)
    ffn_rows_kernel(const __grid_constant__ FfnRowsArgs a) {
  __shared__ float red[kWarps][2][kFewRows][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane & 3, group = lane >> 2;
  const int shares = (int)gridDim.y, share = (int)blockIdx.y;
  const int n0 = blockIdx.x * (kGlu ? 16 : 32);
  if (kGlu) griddep_launch_dependents();
  if (kGlu && blockIdx.x == 0 && share == 0 && threadIdx.x < 2)
    a.status[threadIdx.x] = 0;   // no wait here can give up

  // rows group and group + 8 of both matrices, 8 k at quad * 8 and 32 further
  const __nv_bfloat16* row[2][2];
  bool in[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int n = n0 + group + 8 * r + (kGlu ? 0 : 16 * m);
      in[m][r] = n < a.N;
      row[m][r] = static_cast<const __nv_bfloat16*>(a.w[m]) + (int64_t)n * a.w_stride[m] + quad * 8;
    }
  const int steps = (a.K + kStep - 1) / kStep;
  const int parts = shares * kWarps, part = share * kWarps + warp;
  const int s0 = (int)((int64_t)steps * part / parts);
  const int s1 = (int)((int64_t)steps * (part + 1) / parts);
  uint4 w[2][2][2][2];   // step parity, half, matrix, row
  auto load = [&](int s, uint4 (&v)[2][2][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = s * kStep + h * 32;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          v[h][m][r] = in[m][r] && k + quad * 8 < a.K ? load_weight(row[m][r] + k)
                                                      : make_uint4(0, 0, 0, 0);
    }
  };
  const __nv_bfloat16* x =
      static_cast<const __nv_bfloat16*>(a.x) + (group < a.T ? group * a.x_stride : 0) + quad * 8;
  auto load_token = [&](int s, uint4 (&v)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = s * kStep + h * 32;
      v[h] = group < a.T && k + quad * 8 < a.K ? *reinterpret_cast<const uint4*>(x + k)
                                               : make_uint4(0, 0, 0, 0);
    }
  };
  float acc[2][4] = {};
  uint4 b[2][2];
  if (s0 < s1) load(s0, w[0]);
  if (s0 + 1 < s1) load(s0 + 1, w[1]);
  if (!kGlu) griddep_wait();   // the tokens' rows come from the launch before
  if (s0 < s1) load_token(s0, b[0]);
  if (s0 + 1 < s1) load_token(s0 + 1, b[1]);
  auto multiply = [&](const uint4 (&v)[2][2][2], const uint4 (&t)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint4 &p = v[h][m][0], &q = v[h][m][1];
        mma(acc[m], p.x, q.x, p.y, q.y, t[h].x, t[h].y);
        mma(acc[m], p.z, q.z, p.w, q.w, t[h].z, t[h].w);
      }
  };
  for (int s = s0; s < s1; s += 2) {
    multiply(w[0], b[0]);
    if (s + 2 < s1) {
      load(s + 2, w[0]);
      load_token(s + 2, b[0]);
    }
    if (s + 1 >= s1) break;
    multiply(w[1], b[1]);
    if (s + 3 < s1) {
      load(s + 3, w[1]);
      load_token(s + 3, b[1]);
    }
  }
  // a fragment's sums: rows group and group + 8, tokens 2 quad and 2 quad + 1
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      red[warp][m][quad * 2 + (i & 1)][group + (i >> 1) * 8] = acc[m][i];
  __syncthreads();
  if (shares > 1) cluster_sync();
  // a thread has a row of a token; the CTAs of a cluster take tokens in turn
  const int token = threadIdx.x / 16, r = threadIdx.x % 16;
  if (token < a.T && token % shares == share) {
    float v0 = 0.f, v1 = 0.f;
    if (shares == 1) {
#pragma unroll
      for (int q = 0; q < kWarps; ++q) {
        v0 += red[q][0][token][r];
        v1 += red[q][1][token][r];
      }
    } else {
#pragma unroll
      for (int c = 0; c < 8; c += 2) {   // 16 on their way before the first is added
        float p[2][2][kWarps];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < kWarps; ++q)
              p[i][m][q] = c + i < shares ? peer_load(&red[q][m][token][r], c + i) : 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = 0; q < kWarps; ++q) {
            v0 += p[i][0][q];
            v1 += p[i][1][q];
          }
      }
    }
    if constexpr (kGlu) {
      if (n0 + r < a.N) {
        const int64_t at = (int64_t)token * a.N + n0 + r;
        float unused;
        static_cast<__nv_bfloat16*>(a.out)[at] =
            __float2bfloat16_rn(activation<false, true>(v0, a.act, unused) * v1);
        if (a.gate != nullptr) {
          const int64_t low = kept_low(a.T, a.N) + token * kept_pitch(a.N) + n0 + r;
          const uint32_t g = __float_as_uint(v0), u = __float_as_uint(v1);
          static_cast<uint16_t*>(a.gate)[at] = (uint16_t)(g >> 16);
          static_cast<uint16_t*>(a.up)[at] = (uint16_t)(u >> 16);
          static_cast<uint8_t*>(a.gate)[low] = (uint8_t)(g >> 8);
          static_cast<uint8_t*>(a.up)[low] = (uint8_t)(u >> 8);
        }
      }
    } else {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (int64_t)token * a.N + n0 + r;
      if (n0 + r < a.N) out[0] = __float2bfloat16_rn(v0);
      if (n0 + 16 + r < a.N) out[16] = __float2bfloat16_rn(v1);
    }
  }
  __syncwarp();
  if (shares > 1) cluster_sync();   // the others have read this CTA's sums
}

template <bool kGlu>
cudaError_t launch(const FfnRowsArgs& a, int sms, cudaStream_t st) {
  const int groups = (a.N + (kGlu ? 15 : 31)) / (kGlu ? 16 : 32);
  const int steps = (a.K + kStep - 1) / kStep;
  // as many shares of k as run at once, a step or more for each warp
  int shares = 1;
  while (shares < 8 && 2 * shares * groups <= kResident * sms && 2 * shares * kWarps <= steps)
    shares *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)groups, (unsigned)shares);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = (unsigned)shares;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kGlu ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, ffn_rows_kernel<kGlu>, a);
}

}  // namespace

static_assert(kThreads == kFewRows * 16, "a thread for every row of every token");

cudaError_t launch_ffn_rows(const FfnRowsArgs& a, bool glu, int sms, cudaStream_t st) {
  if (a.T > kFewRows) return cudaErrorInvalidValue;
  return glu ? launch<true>(a, sms, st) : launch<false>(a, sms, st);
}

}  // namespace cpattn
