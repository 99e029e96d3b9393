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

// A piece's elements as pairs of floats.
template <typename T>
__device__ __forceinline__ void widen(const uint4& v, uint64_t (&f)[kPiece<T> / 2]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i)   // a bf16 is the upper half of its fp32
      f[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      f[i] = pack2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
  }
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const uint64_t (&f)[kPiece<T> / 2]) {
  uint32_t u[4];
  float a, b;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unpack2(f[i], a, b);
      u[i] = pack_bf16x2(a, b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      unpack2(f[i], a, b);
      u[2 * i] = __float_as_uint(a);
      u[2 * i + 1] = __float_as_uint(b);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float sum2(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}

// One piece of a row as stored (16 bytes); elements past the row are zero.
template <typename T, int TPR, bool kVec>
__device__ __forceinline__ uint4 load_piece(const T* row, int t, int i, int D) {
  constexpr int E = kPiece<T>;
  if constexpr (kVec) {
    const int c = column<T, TPR, true>(t, i, 0);
    return c < D ? load_once(row + c) : make_uint4(0, 0, 0, 0);
  } else {
    uint64_t f[E / 2];
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      const int c = column<T, TPR, false>(t, i, j), d = column<T, TPR, false>(t, i, j + 1);
      f[j / 2] = pack2(c < D ? as_float(row[c]) : 0.f, d < D ? as_float(row[d]) : 0.f);
    }
    return narrow<T>(f);   // exact: the values come from this type
  }
}

template <typename T, int TPR, bool kVec>
__device__ __forceinline__ void store_piece(T* row, int t, int i, int D,
                                            const uint64_t (&f)[kPiece<T> / 2]) {
  constexpr int E = kPiece<T>;
  if constexpr (kVec) {
    const int c = column<T, TPR, true>(t, i, 0);
    if (c < D) *reinterpret_cast<uint4*>(row + c) = narrow<T>(f);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int c = column<T, TPR, false>(t, i, j);
      float v[2];
      unpack2(f[j / 2], v[0], v[1]);
      if (c < D) {
        if constexpr (sizeof(T) == 2) row[c] = __float2bfloat16_rn(v[j & 1]);
        else row[c] = v[j & 1];
      }
    }
  }
}

// Weights or biases of one piece's columns (`none` where the pointer is null, zero
// past the row).
template <typename T, int TPR, bool kVec>
__device__ __forceinline__ void load_weights(const void* w, bool bf16, float none, int t, int i,
                                             int D, uint64_t (&f)[kPiece<T> / 2]) {
  constexpr int E = kPiece<T>;
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) f[j] = pack2(none, none);
    return;
  }
  const int c0 = column<T, TPR, kVec>(t, i, 0);
  if (kVec && c0 < D) {   // pieces lie within the row
    if (bf16) {
      const uint32_t* p =
          reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(w) + c0);
#pragma unroll
      for (int j = 0; j < E / 2; ++j)
        f[j] = pack2(__uint_as_float(p[j] << 16), __uint_as_float(p[j] & 0xffff0000u));
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c0);
#pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        const float4 v = p[j];
        f[2 * j] = pack2(v.x, v.y);
        f[2 * j + 1] = pack2(v.z, v.w);
      }
    }
    return;
  }
  float v[E];
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int c = column<T, TPR, kVec>(t, i, j);
    v[j] = c >= D  ? 0.f
           : bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c])
                  : static_cast<const float*>(w)[c];
  }
#pragma unroll
  for (int j = 0; j < E / 2; ++j) f[j] = pack2(v[2 * j], v[2 * j + 1]);
}

constexpr int kMinThreads = 256;   // of a block whose rows take fewer

// The next row's pieces are copied asynchronously into shared memory by the thread that
// will use them (so no barrier) while it works on a row: forward 186 us with them held
// in registers, 183 so (131072 x 2048, bf16; fp32 x 1000 169 and 159), backward 275 and
// 243, as the registers go to the sums.  More rows ahead gained nothing.
constexpr int block_threads(int tpr) { return tpr > kMinThreads ? tpr : kMinThreads; }
__device__ __forceinline__ void copy_async(uint4* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(in ? 16 : 0)   // zeros past the row
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copy_wait() {   // all rows but the last are there
  asm volatile("cp.async.wait_group 1;" ::: "memory");
}

// Sum over each kLanes neighbouring lanes.
template <int kLanes = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}


// Persistent blocks: a group of TPR threads takes rows gridDim.x * G apart with its
// columns' weights in registers (read per row they were twice the traffic of bf16
// rows, from L1) and the next row's loads in flight.  A warp takes the squares about
// its own mean, and the warps' means and squares are then joined: one barrier a row.
template <typename T, int TPR, int NV, bool kVec, int kBlocks>
__global__ void __launch_bounds__(block_threads(TPR), kBlocks)
    layer_norm_fwd_kernel(const __grid_constant__ LayerNormArgs a) {
  constexpr int E2 = kPiece<T> / 2;
  constexpr int G = block_threads(TPR) / TPR;   // rows of one pass
  constexpr int kWarps = TPR / 32;              // of one row
  __shared__ float2 red[2][G][kWarps];          // a warp's mean, sum of squares about it
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int warp = t >> 5, lane = threadIdx.x & 31;
  // columns of warp w of the row
  auto columns_of = [&](int w) {
    int n = 0;
    for (int i = 0; i < NV; ++i) {
      if (kVec) {
        const int c = (i * TPR + w * 32) * 2 * E2;
        n += min(max(a.D - c, 0), 32 * 2 * E2);
      } else {
        for (int j = 0; j < 2 * E2; ++j) n += min(max(a.D - (i * 2 * E2 + j) * TPR - w * 32, 0), 32);
      }
    }
    return n;
  };
  const int mine = columns_of(warp);
  const float inv_mine = mine > 0 ? 1.f / (float)mine : 0.f;
  const float lane_cols = kWarps > 1 ? (float)columns_of(lane % kWarps) : 0.f;
  uint64_t w[NV][E2], b[NV][E2];
  uint4 raw[NV];
  extern __shared__ uint4 ring[];   // [2][NV][threads]
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t row = (int64_t)blockIdx.x * G + grp;
  int stage = 0;   // of the row to be taken
  auto stage_at = [&](int s, int i) {
    return ring + (s * NV + i) * block_threads(TPR) + threadIdx.x;
  };
  auto load = [&](int64_t r, int to) {
    const T* src = static_cast<const T*>(a.x) + r * a.x_stride;
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = column<T, TPR, true>(t, i, 0);
        if (r < a.T) copy_async(stage_at(to, i), src + (c < a.D ? c : 0), c < a.D);
      }
      copy_commit();
    } else if (r < a.T) {
#pragma unroll
      for (int i = 0; i < NV; ++i) raw[i] = load_piece<T, TPR, false>(src, t, i, a.D);
    }
  };
  // the row's pieces, and the loads of one to come
  auto take = [&](uint64_t (&x)[NV][E2]) {
    if constexpr (kVec) {
      load(row + step, stage ^ 1);
      copy_wait();
#pragma unroll
      for (int i = 0; i < NV; ++i) raw[i] = *stage_at(stage, i);
      stage ^= 1;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) widen<T>(raw[i], x[i]);
    if constexpr (!kVec) load(row + step, 0);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) raw[i] = make_uint4(0, 0, 0, 0);
  load(row, 0);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_weights<T, TPR, kVec>(a.w, a.w_bf16, 1.f, t, i, a.D, w[i]);
    load_weights<T, TPR, kVec>(a.b, a.w_bf16, 0.f, t, i, a.D, b[i]);
  }
  int slot = 0;
  // a warp that is a row's only one leaves when its rows are done; with several the
  // whole block walks alike
  for (int64_t first = (int64_t)blockIdx.x * G; kWarps > 1 ? first < a.T : row < a.T;
       first += step, row += step) {
    uint64_t x[NV][E2];
    uint64_t s2 = 0ull;
    take(x);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < E2; ++j) s2 = add2(s2, x[i][j]);
    float mean = warp_sum(sum2(s2)) * inv_mine;
    const uint64_t neg = pack2(-mean, -mean);
    uint64_t ss = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < E2; ++j) {
        const uint64_t d = add2(x[i][j], neg);
        if constexpr (kVec) {   // elements past the row have no square
          if (column<T, TPR, true>(t, i, 0) < a.D) ss = fma2(d, d, ss);
        } else {
          float p, q;
          unpack2(d, p, q);
          p = column<T, TPR, false>(t, i, 2 * j) < a.D ? p : 0.f;
          q = column<T, TPR, false>(t, i, 2 * j + 1) < a.D ? q : 0.f;
          const uint64_t e = pack2(p, q);
          ss = fma2(e, e, ss);
        }
      }
    float squares = warp_sum(sum2(ss));
    if constexpr (kWarps > 1) {
      if (lane == 0) red[slot][grp][warp] = make_float2(mean, squares);
      __syncthreads();
      // a lane has a warp's: the mean of all, then the squares about that (each
      // thread adding all warps' from shared memory measured 3 to 15 % slower)
      const float2 v = red[slot][grp][lane % kWarps];
      mean = warp_sum<kWarps>(v.x * lane_cols) * a.inv_D;
      const float d = v.x - mean;
      squares = warp_sum<kWarps>(lane_cols > 0.f ? fmaf(lane_cols * d, d, v.y) : 0.f);
      slot ^= 1;   // the next pass writes the other slot: one barrier a pass
    }
    const float r = __frsqrt_rn(squares * a.inv_D + a.eps);
    if (row < a.T) {
      T* dst = static_cast<T*>(a.y) + row * a.D;
      const uint64_t m2 = pack2(-mean, -mean), r2 = pack2(r, r);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < E2; ++j)
          x[i][j] = fma2(mul2(add2(x[i][j], m2), r2), w[i][j], b[i][j]);
        store_piece<T, TPR, kVec>(dst, t, i, a.D, x[i]);
      }
      if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = r;
      }
    }
  }
}

// bf16 rows of one block of 512 threads come through registers all the same: 282 us for
// 32768 x 8192, 394 through shared memory (fp32, half the elements a thread: 32768 x 4096
// 268 and 252).  The widest rows leave no room.
constexpr bool bwd_ring(int tpr, int elem, bool vec) {
  return vec && (tpr <= 256 || (tpr == 512 && elem == 4));
}

// kWide (rows of more than 1024 threads' 8 elements): sums of dw and db in shared
// memory and no row read ahead, so that a thread's row fits 64 registers.
template <typename T, int TPR, int NV, bool kVec, bool kWide, int kBlocks>
__global__ void __launch_bounds__(block_threads(TPR), kBlocks)
    layer_norm_bwd_kernel(const __grid_constant__ LayerNormArgs a) {
  constexpr int E = kPiece<T>, E2 = E / 2;
  constexpr int kThreads = block_threads(TPR);
  constexpr int G = kThreads / TPR;        // rows of one pass
  constexpr int kWarps = TPR / 32;         // of one row
  constexpr int kCols = TPR * NV * E;
  constexpr int kHeld = kWide ? 1 : NV;
  extern __shared__ __align__(16) float acc[];   // kWide: [2][kCols]; else [G][2][kCols] at the end
  __shared__ float2 red[2][G][kWarps];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int warp = t >> 5, lane = threadIdx.x & 31;
  uint64_t dw[kHeld][E2], db[kHeld][E2], w[kHeld][E2];
  uint4 rx[NV], rd[NV];
  float mean = 0.f, r = 0.f;
  constexpr bool kRing = bwd_ring(TPR, sizeof(T), kVec);   // else rows come straight into registers
  uint4* ring = reinterpret_cast<uint4*>(acc);   // [2][x, dy][NV][threads]
  const int64_t step = (int64_t)gridDim.x * G;
  int64_t row = (int64_t)blockIdx.x * G + grp;
  int stage = 0;
  auto stage_at = [&](int s, int which, int i) {
    return ring + ((s * 2 + which) * NV + i) * kThreads + threadIdx.x;
  };
  auto load = [&](int64_t q, int to) {
    const T* x = static_cast<const T*>(a.x) + q * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + q * a.dy_stride;
    if constexpr (kRing) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = column<T, TPR, true>(t, i, 0);
        if (q < a.T) {
          copy_async(stage_at(to, 0, i), x + (c < a.D ? c : 0), c < a.D);
          copy_async(stage_at(to, 1, i), dy + (c < a.D ? c : 0), c < a.D);
        }
      }
      copy_commit();
    } else {   // a group without a row in the last pass adds nothing
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        rx[i] = q < a.T ? load_piece<T, TPR, kVec>(x, t, i, a.D) : make_uint4(0, 0, 0, 0);
        rd[i] = q < a.T ? load_piece<T, TPR, kVec>(dy, t, i, a.D) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  auto load_stats = [&](int64_t q) {
    mean = q < a.T ? a.mean[q] : 0.f;
    r = q < a.T ? a.rstd[q] : 0.f;
  };
  if constexpr (!kWide) load(row, 0);
  load_stats(row);
  if constexpr (kWide) {
    for (int c = threadIdx.x; c < 2 * kCols; c += kThreads) acc[c] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_weights<T, TPR, kVec>(a.w, a.w_bf16, 1.f, t, i, a.D, w[i]);
#pragma unroll
      for (int j = 0; j < E2; ++j) dw[i][j] = db[i][j] = 0ull;
    }
  }
  int slot = 0;
  for (int64_t first = (int64_t)blockIdx.x * G; first < a.T; first += step, row += step) {
    if constexpr (kWide) load(row, 0);
    if constexpr (kRing) {
      load(row + step, stage ^ 1);
      copy_wait();
      const bool in = row < a.T;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        rx[i] = in ? *stage_at(stage, 0, i) : make_uint4(0, 0, 0, 0);
        rd[i] = in ? *stage_at(stage, 1, i) : make_uint4(0, 0, 0, 0);
      }
      stage ^= 1;
    }
    uint64_t s1 = 0ull, s2 = 0ull;
    uint64_t n[kHeld][E2], g[kHeld][E2];
    const uint64_t r2 = pack2(r, r), m2 = pack2(-mean, -mean);
    // n and g of a piece; the first time its share of the sums too
    auto take = [&](int i, uint64_t (&ni)[E2], uint64_t (&gi)[E2], const uint64_t (&wi)[E2],
                    bool sums) {
      uint64_t d[E2];
      widen<T>(rx[i], ni);
      widen<T>(rd[i], d);
#pragma unroll
      for (int j = 0; j < E2; ++j) {
        ni[j] = mul2(add2(ni[j], m2), r2);
        gi[j] = mul2(d[j], wi[j]);   // past the row: zeros, in all sums
        if (!sums) continue;
        s1 = add2(s1, gi[j]);
        s2 = fma2(gi[j], ni[j], s2);
        if constexpr (kWide) {
          if (a.partial) {
            uint64_t* p = reinterpret_cast<uint64_t*>(acc) + (i * E2 + j) * TPR + t;
            p[0] = fma2(d[j], ni[j], p[0]);
            p[kCols / 2] = add2(p[kCols / 2], d[j]);
          }
        } else {
          dw[i][j] = fma2(d[j], ni[j], dw[i][j]);
          db[i][j] = add2(db[i][j], d[j]);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (kWide) {
        uint64_t wi[E2];
        load_weights<T, TPR, kVec>(a.w, a.w_bf16, 1.f, t, i, a.D, wi);
        take(i, n[0], g[0], wi, true);
      } else {
        take(i, n[i], g[i], w[i], true);
      }
    }
    const float rc = r;
    if constexpr (!kWide && !kRing) load(row + step, 0);   // in flight during the sums
    load_stats(row + step);
    float c1 = warp_sum(sum2(s1)), c2 = warp_sum(sum2(s2));
    if constexpr (kWarps > 1) {
      if (lane == 0) red[slot][grp][warp] = make_float2(c1, c2);
      __syncthreads();
      c1 = c2 = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        c1 += red[slot][grp][i].x;
        c2 += red[slot][grp][i].y;
      }
      slot ^= 1;   // the next pass writes the other slot: one barrier a pass
    }
    if (a.y != nullptr && row < a.T) {
      c1 *= -a.inv_D * rc;
      c2 *= -a.inv_D;
      const uint64_t k1 = pack2(c1, c1), k2 = pack2(c2, c2), kr = pack2(rc, rc);
      T* dst = static_cast<T*>(a.y) + row * a.D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int k = kWide ? 0 : i;
        if constexpr (kWide) {
          uint64_t wi[E2];
          load_weights<T, TPR, kVec>(a.w, a.w_bf16, 1.f, t, i, a.D, wi);
          take(i, n[0], g[0], wi, false);
        }
        uint64_t dx[E2];
#pragma unroll
        for (int j = 0; j < E2; ++j) dx[j] = fma2(fma2(n[k][j], k2, g[k][j]), kr, k1);
        store_piece<T, TPR, kVec>(dst, t, i, a.D, dx);
      }
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.D;
  if constexpr (kWide || G == 1) {   // a thread's own columns: no barrier
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < E2; ++j) {
        uint64_t vw, vb;
        if constexpr (kWide) {
          const uint64_t* p = reinterpret_cast<const uint64_t*>(acc) + (i * E2 + j) * TPR + t;
          vw = p[0];
          vb = p[kCols / 2];
        } else {
          vw = dw[i][j];
          vb = db[i][j];
        }
        float fw[2], fb[2];
        unpack2(vw, fw[0], fw[1]);
        unpack2(vb, fb[0], fb[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = column<T, TPR, kVec>(t, i, 2 * j + e);
          if (c < a.D) {
            out[c] = fw[e];
            out[a.D + c] = fb[e];
          }
        }
      }
  } else {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();   // the ring's place is free
    float* own = acc + grp * 2 * kCols;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < E2; ++j) {
        float fw[2], fb[2];
        unpack2(dw[i][j], fw[0], fw[1]);
        unpack2(db[i][j], fb[0], fb[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = column<T, TPR, kVec>(t, i, 2 * j + e);
          own[c] = fw[e];
          own[kCols + c] = fb[e];
        }
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

// Threads per row, 16-byte pieces per thread and blocks per SM of a launch.
struct Shape {
  int tpr, nv, blocks;
};
constexpr Shape kFwdShapes[] = {{32, 1, 4},  {32, 2, 3},  {64, 2, 3}, {128, 2, 3},
                                {256, 2, 3}, {256, 4, 2}, {512, 4, 1}};
// fp32: half the elements a piece, so fewer registers
constexpr Shape kFwdShapesF32[] = {{32, 1, 4},  {32, 2, 4},  {64, 2, 4},   {128, 2, 4},
                                   {256, 2, 4}, {512, 2, 2}, {1024, 2, 1}, {1024, 4, 1}};
constexpr Shape kBwdShapes[] = {{32, 1, 3},  {32, 2, 2},  {64, 2, 2},   {128, 2, 2},
                                {256, 2, 2}, {512, 2, 1}, {1024, 2, 1}, {1024, 4, 1}};   // last: fp32
constexpr int kBwdWideFrom = 6;   // shapes with sums in shared memory

// The shape of rows of `pieces` 16-byte pieces: 32, 64, 128, ... at most.
constexpr int shape_of(int pieces) {
  int i = 0;
  while ((32 << i) < pieces) ++i;
  return i;
}

constexpr int pieces_of(int D, bool bf16) { return bf16 ? (D + 7) / 8 : (D + 3) / 4; }

// The shapes that rows of a type reach.
template <typename T>
constexpr int kShapes = shape_of(pieces_of(kLayerNormMaxWidth, sizeof(T) == 2)) + 1;
template <typename A>
constexpr int entries(const A&) { return sizeof(A) / sizeof(Shape); }
static_assert(kShapes<__nv_bfloat16> == entries(kFwdShapes) && kShapes<float> == entries(kFwdShapesF32) &&
              kShapes<float> == entries(kBwdShapes), "no shape without rows, none missing");

// f(the shape's number as an integral constant)
template <typename T, int I = 0, typename F>
cudaError_t by_shape(int i, F f) {
  if constexpr (I < kShapes<T>)
    return i == I ? f(std::integral_constant<int, I>{}) : by_shape<T, I + 1>(i, f);
  else return cudaErrorInvalidValue;
}

int blocks_of(const Shape& s, int64_t T, int sms) {
  const int rows = block_threads(s.tpr) / s.tpr;
  const int64_t need = (T + rows - 1) / rows, most = (int64_t)s.blocks * sms;
  return (int)(need < most ? need : most);
}

constexpr int ring_bytes(const Shape& s, int arrays) {
  return 2 * arrays * s.nv * block_threads(s.tpr) * 16;
}

// 48 KB are there unasked, static ones among them.
template <typename F>
cudaError_t more_shared(F kernel, int bytes) {
  if (bytes <= 40 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, bool kVec>
cudaError_t fwd_t(const LayerNormArgs& a, int sms, cudaStream_t st) {
  return by_shape<T>(shape_of(pieces_of(a.D, sizeof(T) == 2)), [&](auto i) {
    constexpr Shape s = sizeof(T) == 2 ? kFwdShapes[decltype(i)::value]
                                       : kFwdShapesF32[decltype(i)::value];
    auto kernel = layer_norm_fwd_kernel<T, s.tpr, s.nv, kVec, s.blocks>;
    constexpr int smem = kVec ? ring_bytes(s, 1) : 0;
    cudaError_t e = more_shared(kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<blocks_of(s, a.T, sms), block_threads(s.tpr), smem, st>>>(a);
    return cudaGetLastError();
  });
}

template <typename T, bool kVec>
cudaError_t bwd_t(const LayerNormArgs& a, int blocks, cudaStream_t st) {
  return by_shape<T>(shape_of(pieces_of(a.D, sizeof(T) == 2)), [&](auto i) {
    constexpr Shape s = kBwdShapes[decltype(i)::value];
    constexpr bool kWide = decltype(i)::value >= kBwdWideFrom;
    constexpr int kThreads = block_threads(s.tpr), G = kThreads / s.tpr;
    constexpr int sums = (kWide || G > 1) ? G * 2 * s.tpr * s.nv * kPiece<T> * 4 : 0;
    constexpr int ring = bwd_ring(s.tpr, sizeof(T), kVec) ? ring_bytes(s, 2) : 0;
    constexpr int smem = sums > ring ? sums : ring;
    auto kernel = layer_norm_bwd_kernel<T, s.tpr, s.nv, kVec, kWide, s.blocks>;
    cudaError_t e = more_shared(kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)blocks, kThreads, smem, st>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace

int layer_norm_bwd_blocks(int64_t T, int D, bool bf16, int sms) {
  return blocks_of(kBwdShapes[shape_of(pieces_of(D, bf16))], T, sms);
}

cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, bool bf16, bool vec, int sms,
                                  cudaStream_t st) {
  if (bf16)
    return vec ? fwd_t<__nv_bfloat16, true>(a, sms, st) : fwd_t<__nv_bfloat16, false>(a, sms, st);
  return vec ? fwd_t<float, true>(a, sms, st) : fwd_t<float, false>(a, sms, st);
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
