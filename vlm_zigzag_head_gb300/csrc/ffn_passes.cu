// The gated feed-forward block beside its tensor-core products: sums of the shares of
// a product with what its epilogue does, and the fp32 products on CUDA cores.
#include <cuda_bf16.h>

#include "ffn.h"
#include "ffn_act.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

template <typename T>
__device__ __forceinline__ float4 load4(const void* p, int64_t i) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
}
template <typename T>
__device__ __forceinline__ void store4(void* p, int64_t i, float4 v) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Four elements, from column c of row m on, of a kept projection.
template <typename T>
__device__ __forceinline__ void keep4(void* p, int64_t m, int c, int64_t M, int N, float4 v) {
  if constexpr (sizeof(T) == 4) {
    store4<float>(p, m * N + c, v);
  } else {
    uint32_t hi[4], lo[4];
    split24(v.x, hi[0], lo[0]);
    split24(v.y, hi[1], lo[1]);
    split24(v.z, hi[2], lo[2]);
    split24(v.w, hi[3], lo[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + m * N + c) =
        make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + kept_low(M, N) + m * kept_pitch(N) +
                                 c) = lo[0] | lo[1] << 8 | lo[2] << 16 | lo[3] << 24;
  }
}
template <typename T>
__device__ __forceinline__ float4 kept4(const void* p, int64_t m, int c, int64_t M, int N) {
  if constexpr (sizeof(T) == 4) {
    return load4<float>(p, m * N + c);
  } else {
    const uint2 h =
        *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + m * N + c);
    const uint32_t l = *reinterpret_cast<const uint32_t*>(
        static_cast<const uint8_t*>(p) + kept_low(M, N) + m * kept_pitch(N) + c);
    return make_float4(join24(h.x & 0xffffu, l), join24(h.x >> 16, l >> 8),
                       join24(h.y & 0xffffu, l >> 16), join24(h.y >> 16, l >> 24));
  }
}

// Bound by memory: reads every share once.  Shares are added in order, so the sums do
// not depend on timing.
template <typename T, int kEpi>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs j) {
  const int64_t n = j.M * j.N, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;   // N is a multiple of 8
  const int64_t row = i / j.N;
  const int col = (int)(i - row * j.N);
  auto sum = [&](const float* p) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < j.splits; ++s) {
      const float4 w = *reinterpret_cast<const float4*>(p + s * n + i);
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    return v;
  };
  float4 x = sum(j.partial);
  if constexpr (kEpi == GEMM_STORE) {
    store4<T>(j.out, i, x);
  } else if constexpr (kEpi == GEMM_GLU) {
    const float4 u = sum(j.partial + j.splits * n);
    if (j.gate != nullptr) {
      keep4<T>(j.gate, row, col, j.M, j.N, x);
      keep4<T>(j.up, row, col, j.M, j.N, u);
    }
    float d;
    x.x = activation<false>(x.x, j.act, d) * u.x;
    x.y = activation<false>(x.y, j.act, d) * u.y;
    x.z = activation<false>(x.z, j.act, d) * u.z;
    x.w = activation<false>(x.w, j.act, d) * u.w;
    store4<T>(j.out, i, x);
  } else {
    const float4 g = kept4<T>(j.gate, row, col, j.M, j.N);
    const float4 u = kept4<T>(j.up, row, col, j.M, j.N);
    const float gs[4] = {g.x, g.y, g.z, g.w}, us[4] = {u.x, u.y, u.z, u.w};
    const float dh[4] = {x.x, x.y, x.z, x.w};
    float h[4], dg[4], du[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float da;
      const float a = activation<true>(gs[e], j.act, da);
      h[e] = a * us[e];
      dg[e] = dh[e] * us[e] * da;
      du[e] = dh[e] * a;
    }
    store4<T>(j.dgate, i, make_float4(dg[0], dg[1], dg[2], dg[3]));
    store4<T>(j.dup, i, make_float4(du[0], du[1], du[2], du[3]));
    store4<T>(j.out, i, make_float4(h[0], h[1], h[2], h[3]));
  }
}

// 128 x 128 tiles, 256 threads of 8 x 8 sums, k by 16 through shared memory; two
// multiply-adds an instruction.
constexpr int kTile = 128, kStep = 16, kPitch = kTile + 4;

__global__ void __launch_bounds__(256) gemm_f32_kernel(const __grid_constant__ GemmF32Args g) {
  __shared__ __align__(16) float as[2][kStep][kPitch], bs[2][kStep][kPitch];
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
  const int steps = (g.K + kStep - 1) / kStep;
  const int s0 = (int)((int64_t)steps * blockIdx.z / g.splits);
  const int s1 = (int)((int64_t)steps * (blockIdx.z + 1) / g.splits);
  float ra[8], rb[8];
  // eight elements of one operand's tile: neighbouring threads along its contiguous
  // direction
  auto load = [&](const float* p, int64_t sr, int64_t sk, int r0, int rows, int k0, float (&r)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = tid + i * 256;
      const int k = sk == 1 ? e % kStep : e / kTile, row = sk == 1 ? e / kStep : e % kTile;
      r[i] = row < rows - r0 && k0 + k < g.K ? p[(int64_t)(r0 + row) * sr + (int64_t)(k0 + k) * sk] : 0.f;
    }
  };
  auto store = [&](float (*t)[kPitch], int64_t sk, const float (&r)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = tid + i * 256;
      const int k = sk == 1 ? e % kStep : e / kTile, row = sk == 1 ? e / kStep : e % kTile;
      t[k][row] = r[i];
    }
  };
  uint64_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[i][c] = 0ull;
  if (s0 < s1) {
    load(g.a, g.sam, g.sak, m0, g.M, s0 * kStep, ra);
    load(g.b, g.sbn, g.sbk, n0, g.N, s0 * kStep, rb);
    store(as[0], g.sak, ra);
    store(bs[0], g.sbk, rb);
  }
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    const int cur = (s - s0) & 1;
    if (s + 1 < s1) {
      load(g.a, g.sam, g.sak, m0, g.M, (s + 1) * kStep, ra);
      load(g.b, g.sbn, g.sbk, n0, g.N, (s + 1) * kStep, rb);
    }
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      // rows ty * 4 and 64 + ty * 4 on, columns tx * 4 and 64 + tx * 4 on
      const float4 a0 = *reinterpret_cast<const float4*>(&as[cur][k][ty * 4]);
      const float4 a1 = *reinterpret_cast<const float4*>(&as[cur][k][64 + ty * 4]);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(&bs[cur][k][tx * 4]);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(&bs[cur][k][64 + tx * 4]);
      const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
      const uint64_t bv[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t a2 = pack2(av[i], av[i]);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] = fma2(a2, bv[c], acc[i][c]);
      }
    }
    if (s + 1 < s1) {
      store(as[cur ^ 1], g.sak, ra);
      store(bs[cur ^ 1], g.sbk, rb);
    }
    __syncthreads();
  }
  float* out = g.out + (int64_t)blockIdx.z * g.M * g.N;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + (i / 4) * 64 + ty * 4 + i % 4;
    if (m >= g.M) continue;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = n0 + c * 64 + tx * 4;
      if (n >= g.N) continue;   // N is a multiple of 4
      float4 v;
      unpack2(acc[i][2 * c], v.x, v.y);
      unpack2(acc[i][2 * c + 1], v.z, v.w);
      float4* p = reinterpret_cast<float4*>(out + (int64_t)m * g.N + n);
      if (g.accumulate) {
        const float4 w = *p;
        v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
      }
      *p = v;
    }
  }
}

template <typename T>
cudaError_t join_t(const JoinArgs& j, int epilogue, cudaStream_t st) {
  const int64_t blocks = (j.M * j.N / 4 + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (epilogue == GEMM_STORE) join_kernel<T, GEMM_STORE><<<(unsigned)blocks, 256, 0, st>>>(j);
  else if (epilogue == GEMM_GLU) join_kernel<T, GEMM_GLU><<<(unsigned)blocks, 256, 0, st>>>(j);
  else join_kernel<T, GEMM_DGLU><<<(unsigned)blocks, 256, 0, st>>>(j);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ffn_join(const JoinArgs& j, int epilogue, bool bf16, cudaStream_t st) {
  return bf16 ? join_t<__nv_bfloat16>(j, epilogue, st) : join_t<float>(j, epilogue, st);
}

cudaError_t launch_gemm_f32(const GemmF32Args& g, cudaStream_t st) {
  const int64_t nt = ((int64_t)g.N + kTile - 1) / kTile;
  if (nt > 65535 || g.splits > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(((int64_t)g.M + kTile - 1) / kTile), (unsigned)nt, (unsigned)g.splits);
  gemm_f32_kernel<<<grid, 256, 0, st>>>(g);
  return cudaGetLastError();
}

}  // namespace cpattn
