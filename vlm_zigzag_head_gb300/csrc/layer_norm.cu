// Layer norm of whole token rows and its gradient.
//
//   mu = mean_e x_e,  r = 1 / sqrt(mean_e (x_e - mu)^2 + eps),  n = (x - mu) r
//   y = n w + b
// Gradient, with g = dy w:
//   dx = r (g - mean_e g_e - n mean_e(g_e n_e)),  dw_e = sum_t dy_e n_e,  db_e = sum_t dy_e.
//
// The passes are bound by memory: forward reads x and writes y, backward reads x
// and dy and writes dx.  A row therefore lives in the registers of its threads:
// the variance is taken about the mean itself (no difference of large sums), and
// nothing is read twice.  All sums are fp32.
//
// A row belongs to one warp where its lanes can hold it, else to a block: a warp
// needs no barrier for its sums.  In the backward a thread owns the same columns
// of every row it meets and keeps their sums of dw and db; blocks walk rows
// gridDim.x apart, write one row of partial sums each, and a second small launch
// adds those in block order, so the sums do not depend on timing.
#include <cuda_bf16.h>

#include <type_traits>

#include "layer_norm.h"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

template <typename T>
constexpr int kPiece = 16 / (int)sizeof(T);   // elements of a 16-byte piece

// A thread's elements of a row: NV pieces.  Vector loads: piece i is the row's
// piece i * TPR + t; element loads take element (i * E + j) * TPR + t instead, so
// that neighbouring lanes read neighbouring elements.
template <typename T, int TPR, bool kVec>
__device__ __forceinline__ int column(int t, int i, int j) {
  constexpr int E = kPiece<T>;
  return kVec ? (i * TPR + t) * E + j : (i * E + j) * TPR + t;
}

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void widen(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // a bf16 is the upper half of its fp32
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const uint4& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 narrow(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}

// One piece of a row as stored (16 bytes); elements past the row are zero.
template <typename T, int TPR, bool kVec>
__device__ __forceinline__ uint4 load_piece(const T* row, int t, int i, int D) {
  constexpr int E = kPiece<T>;
  if constexpr (kVec) {
    const int c = column<T, TPR, true>(t, i, 0);
    return c < D ? load_once(row + c) : make_uint4(0, 0, 0, 0);
  } else {
    float f[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int c = column<T, TPR, false>(t, i, j);
      f[j] = c < D ? as_float(row[c]) : 0.f;
    }
    return narrow(f);   // exact: the values come from this type
  }
}

template <typename T, int TPR, bool kVec>
__device__ __forceinline__ void store_piece(T* row, int t, int i, int D,
                                            const float (&f)[kPiece<T>]) {
  constexpr int E = kPiece<T>;
  if constexpr (kVec) {
    const int c = column<T, TPR, true>(t, i, 0);
    if (c < D) *reinterpret_cast<uint4*>(row + c) = narrow(f);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int c = column<T, TPR, false>(t, i, j);
      if (c < D) {
        if constexpr (sizeof(T) == 2) row[c] = __float2bfloat16_rn(f[j]);
        else row[c] = f[j];
      }
    }
  }
}

// Weights or biases of one piece's columns (`none` where the pointer is null).
template <typename T, int TPR, bool kVec>
__device__ __forceinline__ void load_weights(const void* w, bool bf16, float none, int t, int i,
                                             int D, float (&f)[kPiece<T>]) {
  constexpr int E = kPiece<T>;
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < E; ++j) f[j] = none;
    return;
  }
  const int c0 = column<T, TPR, kVec>(t, i, 0);
  if (kVec && c0 < D) {   // pieces lie within the row
    if (bf16) {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(w) + c0;
      if constexpr (E == 8) {
        widen(*reinterpret_cast<const uint4*>(p), f);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        f[0] = __uint_as_float(v.x << 16);
        f[1] = __uint_as_float(v.x & 0xffff0000u);
        f[2] = __uint_as_float(v.y << 16);
        f[3] = __uint_as_float(v.y & 0xffff0000u);
      }
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c0);
#pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        const float4 v = p[j];
        f[4 * j] = v.x;
        f[4 * j + 1] = v.y;
        f[4 * j + 2] = v.z;
        f[4 * j + 3] = v.w;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int c = column<T, TPR, kVec>(t, i, j);
    f[j] = c >= D  ? 0.f
           : bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c])
                  : static_cast<const float*>(w)[c];
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, int TPR, int NV, bool kVec>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR)
    layer_norm_fwd_kernel(const __grid_constant__ LayerNormArgs a) {
  constexpr int E = kPiece<T>;
  constexpr int kWarps = TPR / 32;
  __shared__ float red[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = TPR == 32 ? lane : threadIdx.x;
  const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
  if (row >= a.T) return;   // whole warps, and only where a row is one warp's
  auto row_sum = [&](float v, int which) {
    v = warp_sum(v);
    if constexpr (kWarps > 1) {
      if (lane == 0) red[which][warp] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += red[which][i];
    }
    return v;
  };
  const T* src = static_cast<const T*>(a.x) + row * a.x_stride;
  uint4 raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) raw[i] = load_piece<T, TPR, kVec>(src, t, i, a.D);
  float x[NV][E];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    widen(raw[i], x[i]);
#pragma unroll
    for (int j = 0; j < E; ++j) sum += x[i][j];
  }
  const float mean = row_sum(sum, 0) * a.inv_D;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < E; ++j) {
      x[i][j] -= mean;
      if (column<T, TPR, kVec>(t, i, j) < a.D) ss = fmaf(x[i][j], x[i][j], ss);
    }
  const float r = rsqrtf(row_sum(ss, 1) * a.inv_D + a.eps);
  T* dst = static_cast<T*>(a.y) + row * a.D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[E], b[E];
    load_weights<T, TPR, kVec>(a.w, a.w_bf16, 1.f, t, i, a.D, w);
    load_weights<T, TPR, kVec>(a.b, a.w_bf16, 0.f, t, i, a.D, b);
#pragma unroll
    for (int j = 0; j < E; ++j) x[i][j] = fmaf(x[i][j] * r, w[j], b[j]);
    store_piece<T, TPR, kVec>(dst, t, i, a.D, x[i]);
  }
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = r;
  }
}

constexpr int kBwdThreads = 256;   // of a block whose rows take fewer

// kWide (rows of more than 1024 threads' 8 elements): sums of dw and db in shared
// memory and no row read ahead, so that a thread's row fits 64 registers.
template <typename T, int TPR, int NV, bool kVec, bool kWide>
__global__ void __launch_bounds__(TPR > kBwdThreads ? TPR : kBwdThreads)
    layer_norm_bwd_kernel(const __grid_constant__ LayerNormArgs a) {
  constexpr int E = kPiece<T>;
  constexpr int kThreads = TPR > kBwdThreads ? TPR : kBwdThreads;
  constexpr int G = kThreads / TPR;        // rows of one pass
  constexpr int kWarps = TPR / 32;         // of one row
  constexpr int kCols = TPR * NV * E;
  extern __shared__ float acc[];           // kWide: [2][kCols]; else [G][2][kCols] at the end
  __shared__ float2 red[2][G][kWarps];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int warp = t >> 5, lane = threadIdx.x & 31;
  float dw[kWide ? 1 : NV][E], db[kWide ? 1 : NV][E], w[kWide ? 1 : NV][E];
  if constexpr (kWide) {
    for (int c = threadIdx.x; c < 2 * kCols; c += kThreads) acc[c] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_weights<T, TPR, kVec>(a.w, a.w_bf16, 1.f, t, i, a.D, w[i]);
#pragma unroll
      for (int j = 0; j < E; ++j) dw[i][j] = db[i][j] = 0.f;
    }
  }
  uint4 rx[NV], rd[NV];
  float mean = 0.f, r = 0.f;
  auto load = [&](int64_t row) {
    if (row < a.T) {
      const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
      const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        rx[i] = load_piece<T, TPR, kVec>(x, t, i, a.D);
        rd[i] = load_piece<T, TPR, kVec>(dy, t, i, a.D);
      }
      mean = a.mean[row];
      r = a.rstd[row];
    } else {   // a group without a row in the last pass adds nothing
#pragma unroll
      for (int i = 0; i < NV; ++i) rx[i] = rd[i] = make_uint4(0, 0, 0, 0);
      mean = r = 0.f;
    }
  };
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t row = (int64_t)blockIdx.x * G + grp;
  if constexpr (!kWide) load(row);
  int slot = 0;
  for (int64_t first = (int64_t)blockIdx.x * G; first < a.T; first += step, row += step) {
    if constexpr (kWide) load(row);
    float s1 = 0.f, s2 = 0.f;
    float n[kWide ? 1 : NV][E], g[kWide ? 1 : NV][E];
    const float rc = r, mc = mean;
    auto widen_piece = [&](int i, float (&ni)[E], float (&gi)[E], const float (&wi)[E], bool sums) {
      float d[E];
      widen(rx[i], ni);
      widen(rd[i], d);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const bool in = column<T, TPR, kVec>(t, i, j) < a.D;
        ni[j] = in ? (ni[j] - mc) * rc : 0.f;
        gi[j] = in ? d[j] * wi[j] : 0.f;
        if (!sums) continue;
        s1 += gi[j];
        s2 = fmaf(gi[j], ni[j], s2);
        if constexpr (kWide) {
          if (in && a.partial) {
            const int c = (i * E + j) * TPR + t;   // no two lanes on one bank
            acc[c] = fmaf(d[j], ni[j], acc[c]);
            acc[kCols + c] += d[j];
          }
        } else {
          dw[i][j] = fmaf(d[j], ni[j], dw[i][j]);
          db[i][j] += d[j];
        }
      }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (kWide) {
        float wi[E];
        load_weights<T, TPR, kVec>(a.w, a.w_bf16, 1.f, t, i, a.D, wi);
        widen_piece(i, n[0], g[0], wi, true);
      } else {
        widen_piece(i, n[i], g[i], w[i], true);
      }
    }
    if constexpr (!kWide) load(row + step);   // in flight during the sums
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (kWarps > 1) {
      if (lane == 0) red[slot][grp][warp] = make_float2(s1, s2);
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        s1 += red[slot][grp][i].x;
        s2 += red[slot][grp][i].y;
      }
      slot ^= 1;   // the next pass writes the other slot: one barrier a pass
    }
    if (a.y != nullptr && row < a.T) {
      const float c1 = s1 * a.inv_D, c2 = s2 * a.inv_D;
      T* dst = static_cast<T*>(a.y) + row * a.D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        constexpr int kOne = 0;
        const int k = kWide ? kOne : i;
        if constexpr (kWide) {
          float wi[E];
          load_weights<T, TPR, kVec>(a.w, a.w_bf16, 1.f, t, i, a.D, wi);
          widen_piece(i, n[0], g[0], wi, false);
        }
        float dx[E];
#pragma unroll
        for (int j = 0; j < E; ++j) dx[j] = rc * (fmaf(-n[k][j], c2, g[k][j]) - c1);
        store_piece<T, TPR, kVec>(dst, t, i, a.D, dx);
      }
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.D;
  if constexpr (kWide) {   // a thread's own columns: no barrier
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int c = column<T, TPR, kVec>(t, i, j), s = (i * E + j) * TPR + t;
        if (c < a.D) {
          out[c] = acc[s];
          out[a.D + c] = acc[kCols + s];
        }
      }
  } else if constexpr (G == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int c = column<T, TPR, kVec>(t, i, j);
        if (c < a.D) {
          out[c] = dw[i][j];
          out[a.D + c] = db[i][j];
        }
      }
  } else {
    float* mine = acc + grp * 2 * kCols;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int c = column<T, TPR, kVec>(t, i, j);
        mine[c] = dw[i][j];
        mine[kCols + c] = db[i][j];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * kCols; c += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < G; ++k) v += acc[k * 2 * kCols + c];
      const int e = c % kCols;
      if (e < a.D) out[(c / kCols) * a.D + e] = v;
    }
  }
}

// 32 columns per block; a warp adds the rows of its share, then the warps' sums
// meet in warp order.
constexpr int kDwWarps = 32;
__global__ void __launch_bounds__(kDwWarps * 32)
    layer_norm_dw_kernel(const float* partial, int blocks, int D, float* dw, float* db) {
  __shared__ float red[kDwWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (col < 2 * D) {
#pragma unroll 4
    for (int b = warp; b < blocks; b += kDwWarps) v += partial[(int64_t)b * 2 * D + col];
  }
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && col < 2 * D) {
#pragma unroll
    for (int g = 1; g < kDwWarps; ++g) v += red[g][lane];
    if (col < D) { if (dw) dw[col] = v; }
    else if (db) db[col - D] = v;
  }
}

template <int V>
using Int = std::integral_constant<int, V>;

// f(threads per row, pieces per thread) for a row of `pieces` 16-byte pieces
template <typename F>
cudaError_t by_width_fwd(int pieces, F f) {
  if (pieces <= 32) return f(Int<32>{}, Int<1>{});
  if (pieces <= 64) return f(Int<32>{}, Int<2>{});
  if (pieces <= 128) return f(Int<32>{}, Int<4>{});
  if (pieces <= 256) return f(Int<32>{}, Int<8>{});
  if (pieces <= 512) return f(Int<128>{}, Int<4>{});
  if (pieces <= 1024) return f(Int<256>{}, Int<4>{});
  if (pieces <= 2048) return f(Int<512>{}, Int<4>{});
  return f(Int<1024>{}, Int<4>{});
}
template <typename F>
cudaError_t by_width_bwd(int pieces, F f) {
  if (pieces <= 32) return f(Int<32>{}, Int<1>{}, Int<0>{});
  if (pieces <= 64) return f(Int<32>{}, Int<2>{}, Int<0>{});
  if (pieces <= 128) return f(Int<64>{}, Int<2>{}, Int<0>{});
  if (pieces <= 256) return f(Int<128>{}, Int<2>{}, Int<0>{});
  if (pieces <= 512) return f(Int<256>{}, Int<2>{}, Int<0>{});
  if (pieces <= 1024) return f(Int<512>{}, Int<2>{}, Int<0>{});
  if (pieces <= 2048) return f(Int<1024>{}, Int<2>{}, Int<1>{});
  return f(Int<1024>{}, Int<4>{}, Int<1>{});
}

int pieces_of(int D, bool bf16) { return bf16 ? (D + 7) / 8 : (D + 3) / 4; }

template <typename T, bool kVec>
cudaError_t fwd_t(const LayerNormArgs& a, cudaStream_t st) {
  return by_width_fwd(pieces_of(a.D, sizeof(T) == 2), [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    const int64_t blocks = TPR == 32 ? (a.T + 7) / 8 : a.T;
    layer_norm_fwd_kernel<T, TPR, NV, kVec>
        <<<(unsigned)blocks, TPR == 32 ? 256 : TPR, 0, st>>>(a);
    return cudaGetLastError();
  });
}

template <typename T, bool kVec>
cudaError_t bwd_t(const LayerNormArgs& a, int blocks, cudaStream_t st) {
  return by_width_bwd(pieces_of(a.D, sizeof(T) == 2), [&](auto tpr, auto nv, auto wide) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr bool kWide = decltype(wide)::value != 0;
    constexpr int kThreads = TPR > kBwdThreads ? TPR : kBwdThreads;
    constexpr int G = kThreads / TPR;
    constexpr int smem = (kWide || G > 1) ? G * 2 * TPR * NV * kPiece<T> * 4 : 0;
    auto kernel = layer_norm_bwd_kernel<T, TPR, NV, kVec, kWide>;
    if (smem > 48 * 1024) {
      cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
    }
    kernel<<<(unsigned)blocks, kThreads, smem, st>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace

int layer_norm_bwd_blocks(int64_t T, int D, bool bf16, int sms) {
  const int pieces = pieces_of(D, bf16);
  int64_t rows = 1, per_sm = 1;   // rows of one pass, blocks that fit an SM
  if (pieces <= 64) rows = 8;
  else if (pieces <= 128) rows = 4;
  else if (pieces <= 256) rows = 2;
  if (pieces <= 512) per_sm = 2;
  const int64_t need = (T + rows - 1) / rows;
  const int64_t most = per_sm * sms;
  return (int)(need < most ? need : most);
}

cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, bool bf16, bool vec, cudaStream_t st) {
  if (bf16) return vec ? fwd_t<__nv_bfloat16, true>(a, st) : fwd_t<__nv_bfloat16, false>(a, st);
  return vec ? fwd_t<float, true>(a, st) : fwd_t<float, false>(a, st);
}

cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, bool bf16, bool vec, int blocks,
                                  cudaStream_t st) {
  if (bf16)
    return vec ? bwd_t<__nv_bfloat16, true>(a, blocks, st)
               : bwd_t<__nv_bfloat16, false>(a, blocks, st);
  return vec ? bwd_t<float, true>(a, blocks, st) : bwd_t<float, false>(a, blocks, st);
}

cudaError_t launch_layer_norm_dw(const float* partial, int blocks, int D, float* dw, float* db,
                                 cudaStream_t st) {
  layer_norm_dw_kernel<<<(2 * D + 31) / 32, kDwWarps * 32, 0, st>>>(partial, blocks, D, dw, db);
  return cudaGetLastError();
}

}  // namespace cpattn
