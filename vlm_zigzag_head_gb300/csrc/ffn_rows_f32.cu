// The gated feed-forward block in fp32 for up to kFewRowsF32 rows: forward.
//
// Bound by the weights, 12 D F bytes, while tokens are few; on CUDA cores, two
// multiply-adds an instruction.  A CTA takes four or eight rows of weights (half of
// gate and half of up, or output columns) and up to eight tokens; its warps, and the CTAs
// of a cluster where there are too few rows to fill the GPU, share k.  Weights go from
// memory to registers past L1, which the tokens' rows stay in.  Groups of eight tokens lie
// beside each other in the grid, so the second to read a weight finds it in L2.  Sums meet
// in a fixed order.
//
// 2048 x 6144, whose bytes take 22.6 us: one token 28 us, four 32, eight 45 (the tokens'
// rows from L1: 56 with four rows of weights to a CTA instead of eight), then 32 us for
// every eight (24 tokens 109, 32 tokens 141).  The tiles that take more rows need 125 to
// 129 us for 1 to 32.
#include <cuda_bf16.h>

#include "ffn.h"
#include "ffn_act.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 128;     // k of one step of a warp: 512 bytes of a row
constexpr int rows_of(int tokens) { return tokens > 4 ? 8 : 4; }        // of weights
constexpr int ahead_of(int tokens) { return tokens > 4 ? 1 : tokens > 2 ? 2 : 4; }
constexpr int resident(int tokens) { return tokens > 4 ? 2 : 4; }       // CTAs an SM holds

struct Four {   // two pairs of fp32
  uint64_t a, b;
};
__device__ __forceinline__ Four load_weight(const float* p) {
  Four v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.b64 {%0, %1}, [%2];"
               : "=l"(v.a), "=l"(v.b)
               : "l"(p));
  return v;
}
__device__ __forceinline__ Four load_token(const float* p) {   // kept in L1
  Four v;
  asm volatile("ld.global.v2.b64 {%0, %1}, [%2];" : "=l"(v.a), "=l"(v.b) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void fma2(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
__device__ __forceinline__ float peer_load(const float* p, int rank) {   // of another CTA
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// Sums of kValues values over the lanes: lane i ends with value i / (32 / kValues).
template <int kValues>
__device__ __forceinline__ float spread_sum(float (&v)[kValues], int lane) {
  int left = kValues;
#pragma unroll
  for (int bit = 16; bit > 0; bit /= 2) {
    if (left > 1) {
      left /= 2;
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < kValues / 2; ++i) {
        if (i >= left) break;
        const float give = up ? v[i] : v[i + left];
        v[i] = (up ? v[i + left] : v[i]) + __shfl_xor_sync(0xffffffffu, give, bit);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
    }
  }
  return v[0];
}

// Grid: groups of kT tokens, fastest, times groups of rows; shares of k.
template <bool kGlu, int kT>
__global__ void __launch_bounds__(kThreads, resident(kT))
    ffn_rows_f32_kernel(const __grid_constant__ FfnRowsArgs a) {
  constexpr int kRows = rows_of(kT);
  constexpr int kValues = kRows * kT;       // [row][token]
  constexpr int kAhead = ahead_of(kT);      // steps whose weights are on their way
  __shared__ float red[kWarps][kValues];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shares = (int)gridDim.y, share = (int)blockIdx.y;
  const int token_groups = (a.T + kT - 1) / kT;
  const int t0 = (int)(blockIdx.x % token_groups) * kT;
  const int n0 = (int)(blockIdx.x / token_groups) * (kGlu ? kRows / 2 : kRows);
  if (kGlu) griddep_launch_dependents();
  if (kGlu && blockIdx.x == 0 && share == 0 && threadIdx.x < 2)
    a.status[threadIdx.x] = 0;   // no wait here can give up

  const float* row[kRows];   // N is a multiple of 8: all are there
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int m = kGlu ? r / (kRows / 2) : 0, n = n0 + (kGlu ? r % (kRows / 2) : r);
    row[r] = static_cast<const float*>(a.w[m]) + (int64_t)n * a.w_stride[m] + lane * 4;
  }
  const float* token[kT];   // past the last: the last, whose sums are not stored
#pragma unroll
  for (int t = 0; t < kT; ++t)
    token[t] = static_cast<const float*>(a.x) + min(t0 + t, a.T - 1) * a.x_stride + lane * 4;

  const int steps = (a.K + kStep - 1) / kStep;
  const int parts = shares * kWarps, part = share * kWarps + warp;
  const int s0 = (int)((int64_t)steps * part / parts);
  const int s1 = (int)((int64_t)steps * (part + 1) / parts);
  Four w[kAhead][kRows];
  auto load = [&](int s, Four (&v)[kRows]) {
    const int k = s * kStep;
    const bool in = k + lane * 4 < a.K;
#pragma unroll
    for (int r = 0; r < kRows; ++r) v[r] = in ? load_weight(row[r] + k) : Four{0, 0};
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (s0 + i < s1) load(s0 + i, w[i]);
  if (!kGlu) griddep_wait();   // the tokens' rows come from the launch before
  uint64_t acc[kRows][kT] = {};
  for (int s = s0; s < s1; s += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s + i >= s1) break;
      const int k = (s + i) * kStep;
      const bool in = k + lane * 4 < a.K;
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const Four x = in ? load_token(token[t] + k) : Four{0, 0};
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          fma2(acc[r][t], w[i][r].a, x.a);
          fma2(acc[r][t], w[i][r].b, x.b);
        }
      }
      if (s + i + kAhead < s1) load(s + i + kAhead, w[i]);
    }
  }
  constexpr int kSpread = kValues < 32 ? kValues : 32;
#pragma unroll
  for (int first = 0; first < kValues; first += kSpread) {
    float v[kSpread];
#pragma unroll
    for (int i = 0; i < kSpread; ++i) {
      float lo, hi;
      unpack2(acc[(first + i) / kT][(first + i) % kT], lo, hi);
      v[i] = lo + hi;
    }
    const float sum = spread_sum(v, lane);
    if (lane % (32 / kSpread) == 0) red[warp][first + lane / (32 / kSpread)] = sum;
  }
  __syncthreads();
  if (shares > 1) cluster_sync();
  // a thread has a row of a token, of gate and of up
  constexpr int kTake = kGlu ? kValues / 2 : kValues;
  if (share == 0 && threadIdx.x < kTake) {
    const int i = threadIdx.x, r = i / kT, t = t0 + i % kT;
    auto total = [&](int value) {
      float f = 0.f;
      if (shares == 1) {
#pragma unroll
        for (int q = 0; q < kWarps; ++q) f += red[q][value];
        return f;
      }
      float p[8][kWarps];   // on their way before the first is added
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int q = 0; q < kWarps; ++q) p[c][q] = c < shares ? peer_load(&red[q][value], c) : 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int q = 0; q < kWarps; ++q) f += p[c][q];
      return f;
    };
    const float gate = total(i);
    const int64_t at = (int64_t)t * a.N + n0 + r;
    float* out = static_cast<float*>(a.out);
    if constexpr (kGlu) {
      const float up = total(kTake + i);
      if (t < a.T) {
        float unused;
        out[at] = activation<false, false>(gate, a.act, unused) * up;
        if (a.gate != nullptr) {
          static_cast<float*>(a.gate)[at] = gate;
          static_cast<float*>(a.up)[at] = up;
        }
      }
    } else if (t < a.T) {
      out[at] = gate;
    }
  }
  __syncwarp();
  if (shares > 1) cluster_sync();   // the first has read this CTA's sums
}

template <bool kGlu, int kT>
cudaError_t launch(const FfnRowsArgs& a, int sms, cudaStream_t st) {
  constexpr int kRows = rows_of(kT);
  const int64_t groups = (int64_t)(a.N / (kGlu ? kRows / 2 : kRows)) * ((a.T + kT - 1) / kT);
  if (groups > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int steps = (a.K + kStep - 1) / kStep;
  // as many shares of k as run at once, a step or more for each warp
  int shares = 1;
  while (shares < 8 && 2 * shares * groups <= (int64_t)resident(kT) * sms &&
         2 * shares * kWarps <= steps)
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
  return cudaLaunchKernelEx(&cfg, ffn_rows_f32_kernel<kGlu, kT>, a);
}

template <bool kGlu>
cudaError_t launch_t(const FfnRowsArgs& a, int sms, cudaStream_t st) {
  if (a.T == 1) return launch<kGlu, 1>(a, sms, st);
  if (a.T == 2) return launch<kGlu, 2>(a, sms, st);
  if (a.T <= 4) return launch<kGlu, 4>(a, sms, st);
  return launch<kGlu, 8>(a, sms, st);
}

}  // namespace

cudaError_t launch_ffn_rows_f32(const FfnRowsArgs& a, bool glu, int sms, cudaStream_t st) {
  if (a.T > kFewRowsF32) return cudaErrorInvalidValue;
  return glu ? launch_t<true>(a, sms, st) : launch_t<false>(a, sms, st);
}

}  // namespace cpattn
