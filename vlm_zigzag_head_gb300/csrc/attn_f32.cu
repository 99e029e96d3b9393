// Attention with modified scores on fp32 inputs, forward and backward, on the
// CUDA cores (fp32 throughout, accurate exp, log and tanh).
//
// One block of 256 threads takes a 64-row tile of one sample and head and walks
// the 64-row tiles it meets.  Operands are staged transposed in shared memory,
// [element][row], and a thread owns a 4 x 4 piece of the 64 x 64 score tile and
// 4 rows x d / 16 elements of the output tile:
//   scores   16 fused multiply-adds per two 16-byte shared loads,
//   outputs  4 d / 4 of them per d / 16 + 4 such loads (contraction in fours),
// so the products are bound by fp32 arithmetic, not by shared memory.
// Backward: one kernel per output side (dQ by query tiles; dK, dV by key tiles and
// query heads).  These inputs are short as a rule, so a tile's walk is what bounds
// a launch: several blocks share it (f32_splits), forward by the log-sum-exp merge
// of their partial results, backward by fp32 adds into zeroed gradients, as for
// the query heads that share a KV head.
#include "scored.h"

namespace cpattn {

namespace {

constexpr int kThreads = 256;
constexpr int kT = kTile32;
constexpr int kPad = kT + 4;     // row pitch of staged tiles (16-byte rows)

template <int D>
constexpr int tile_floats() { return D * kPad; }
constexpr int kPFloats = kT * kPad;

// dst[e][row] = src[row][e] for row < rows, 0 beyond.  A warp takes 8 rows x 64
// bytes at a time: half as many lines per load as one row per lane, at the price of
// two-way conflicts among its stores.
template <int D>
__device__ __forceinline__ void stage(float* dst, const float* src, int rows, int64_t stride) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = warp * 8 + (lane >> 2);
#pragma unroll
  for (int e = (lane & 3) * 4; e < D; e += 16) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows) v = *reinterpret_cast<const float4*>(src + row * stride + e);
    dst[e * kPad + row] = v.x;
    dst[(e + 1) * kPad + row] = v.y;
    dst[(e + 2) * kPad + row] = v.z;
    dst[(e + 3) * kPad + row] = v.w;
  }
}
static_assert(kThreads == 8 * 32 && kT == 64, "eight warps stage eight rows each");

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// c[i][j] = sum_e A[e][4 ty + i] B[e][4 tx + j]
template <int D>
__device__ __forceinline__ void outer(const float* A, const float* B, int ty, int tx,
                                      float (&c)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
#pragma unroll 8
  for (int e = 0; e < D; ++e) {
    const float4 a = ld4(A + e * kPad + 4 * ty), b = ld4(B + e * kPad + 4 * tx);
    const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[i][j] = fmaf(av[i], bv[j], c[i][j]);
  }
}

// acc[i][j] += sum_u P[u][4 ty + i] B[tx + 16 j][u]
template <int D>
__device__ __forceinline__ void accumulate(const float* P, const float* B, int ty, int tx,
                                           float (&acc)[4][D / 16]) {
#pragma unroll 2
  for (int u = 0; u < kT; u += 4) {
    float4 p[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) p[x] = ld4(P + (u + x) * kPad + 4 * ty);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const float4 b = ld4(B + (tx + 16 * j) * kPad + u);
      const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        acc[0][j] = fmaf(p[x].x, bv[x], acc[0][j]);
        acc[1][j] = fmaf(p[x].y, bv[x], acc[1][j]);
        acc[2][j] = fmaf(p[x].z, bv[x], acc[2][j]);
        acc[3][j] = fmaf(p[x].w, bv[x], acc[3][j]);
      }
    }
  }
}

// P[4 tx + j][4 ty + i] = c[i][j]
__device__ __forceinline__ void put(float* P, int ty, int tx, const float (&c)[4][4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<float4*>(P + (4 * tx + j) * kPad + 4 * ty) =
        make_float4(c[0][j], c[1][j], c[2][j], c[3][j]);
}

// Score of query position i and key position j from their product; tanh's value
// in t (0 without a cap).  -inf where the pair is hidden.
__device__ __forceinline__ float score(const F32Args& a, int h, float s, int i, int j, int prefix,
                                       float& t) {
  float x = s * a.scale;
  t = 0.f;
  if (a.softcap > 0.f) {
    t = tanhf(x * a.inv_cap);
    x = a.softcap * t;
  }
  const int dist = i - j;
  if (a.slopes) x -= a.slopes[h] * (float)(dist < 0 ? -dist : dist);
  if (a.table) {
    const int lim = a.n_dist - 1;
    x += a.table[(int64_t)h * a.table_pitch + a.table_mid + max(-lim, min(dist, lim))];
  }
  const bool seen = dist >= 0 || (i < prefix && j < prefix);
  return seen ? x : -INFINITY;
}

__device__ __forceinline__ float row_max(float v) {   // over the 16 threads of a row
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The tiles [first, last) of a walk of n that fall to this block.
__device__ __forceinline__ void my_tiles(const F32Args& a, int n, int& first, int& last) {
  first = (int)((int64_t)n * blockIdx.z / a.splits);
  last = (int)((int64_t)n * (blockIdx.z + 1) / a.splits);
}

// Keys a query tile sees: up to its last row, or the whole both-way prefix.
__device__ __forceinline__ int visible_keys(const Tile32& tl) {
  const int t0 = tl.row0 - tl.seq0;
  return t0 < tl.prefix ? max(tl.prefix, t0 + tl.len) : t0 + tl.len;
}

template <int D>
__global__ void __launch_bounds__(kThreads) f32_fwd_kernel(const F32Args a) {
  extern __shared__ float sm[];
  float* Q = sm;
  float* K = Q + tile_floats<D>();
  float* V = K + tile_floats<D>();
  float* P = V + tile_floats<D>();
  const Tile32 tl = a.tiles[gridDim.x - 1 - blockIdx.x];   // longest walks first
  const int h = blockIdx.y, hk = h / (a.H / a.Hkv);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int t0 = tl.row0 - tl.seq0, nkeys = visible_keys(tl);
  const int64_t qs = (int64_t)a.H * D, ks = (int64_t)a.Hkv * D;
  stage<D>(Q, a.q + tl.row0 * qs + h * D, tl.len, qs);
  float o[4][D / 16], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[i][j] = 0.f;
  }
  int first, last;
  my_tiles(a, (nkeys + kT - 1) / kT, first, last);
  for (int u0 = first * kT; u0 < last * kT; u0 += kT) {
    const int n = min(kT, nkeys - u0);
    __syncthreads();
    stage<D>(K, a.k + (tl.seq0 + u0) * ks + hk * D, n, ks);
    stage<D>(V, a.v + (tl.seq0 + u0) * ks + hk * D, n, ks);
    __syncthreads();
    float c[4][4];
    outer<D>(Q, K, ty, tx, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY, t;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int u = u0 + 4 * tx + j;
        c[i][j] = u < nkeys ? score(a, h, c[i][j], t0 + 4 * ty + i, u, tl.prefix, t) : -INFINITY;
        top = fmaxf(top, c[i][j]);
      }
      top = fmaxf(m[i], row_max(top));
      const float base = top == -INFINITY ? 0.f : top;   // nothing seen yet: all terms are 0
      const float old = expf(m[i] - base);
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[i][j] = expf(c[i][j] - base);
        sum += c[i][j];
      }
      l[i] = l[i] * old + row_sum(sum);
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[i][j] *= old;
    }
    put(P, ty, tx, c);
    __syncthreads();
    accumulate<D>(P, V, ty, tx, o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= tl.len) continue;
    // 0: no key seen; NaN: a score was, or overflowed, and out and lse are too
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    float* dst = a.out + (blockIdx.z * a.T + tl.row0 + r) * qs + h * D;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) dst[tx + 16 * j] = o[i][j] * inv;
    if (tx == 0)
      a.lse[((int64_t)blockIdx.z * a.H + h) * a.T + tl.row0 + r] =
          l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) f32_dq_kernel(const F32Args a) {
  extern __shared__ float sm[];
  float* Q = sm;
  float* dO = Q + tile_floats<D>();
  float* K = dO + tile_floats<D>();
  float* V = K + tile_floats<D>();
  float* P = V + tile_floats<D>();
  const Tile32 tl = a.tiles[gridDim.x - 1 - blockIdx.x];   // longest walks first
  const int h = blockIdx.y, hk = h / (a.H / a.Hkv);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int t0 = tl.row0 - tl.seq0, nkeys = visible_keys(tl);
  const int64_t qs = (int64_t)a.H * D, ks = (int64_t)a.Hkv * D;
  stage<D>(Q, a.q + tl.row0 * qs + h * D, tl.len, qs);
  stage<D>(dO, a.dout + tl.row0 * qs + h * D, tl.len, qs);
  float dq[4][D / 16], lse[4], Dr[4], far_sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    lse[i] = r < tl.len ? a.lse_in[h * a.T + tl.row0 + r] : -INFINITY;
    Dr[i] = r < tl.len ? a.D[h * a.pitch_d + tl.row0 + r] : 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) dq[i][j] = 0.f;
  }
  int first, last;
  my_tiles(a, (nkeys + kT - 1) / kT, first, last);
  if (first >= last) return;
  for (int u0 = first * kT; u0 < last * kT; u0 += kT) {
    const int n = min(kT, nkeys - u0);
    __syncthreads();
    stage<D>(K, a.k + (tl.seq0 + u0) * ks + hk * D, n, ks);
    stage<D>(V, a.v + (tl.seq0 + u0) * ks + hk * D, n, ks);
    __syncthreads();
    float c[4][4], g[4][4];
    outer<D>(Q, K, ty, tx, c);
    outer<D>(dO, V, ty, tx, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int pos = t0 + 4 * ty + i, u = u0 + 4 * tx + j;
        float t;
        const float x = score(a, h, c[i][j], pos, u, tl.prefix, t);
        // rows without a key, rows past the tile and hidden pairs have no share
        const bool live = lse[i] != -INFINITY && u < nkeys && x != -INFINITY;
        const float ds = live ? expf(x - lse[i]) * (g[i][j] - Dr[i]) : 0.f;
        if (a.dtable && live) {   // pairs past the table's last distance meet in a register
          const int dist = pos > u ? pos - u : u - pos;
          if (dist >= a.n_dist - 1) far_sum += ds;
          else atomicAdd(a.dtable + (int64_t)h * a.n_dist + dist, ds);
        }
        c[i][j] = ds * (1.f - t * t) * a.scale;
      }
    }
    put(P, ty, tx, c);
    __syncthreads();
    accumulate<D>(P, K, ty, tx, dq);
  }
  if (a.dtable) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) far_sum += __shfl_xor_sync(0xffffffffu, far_sum, o);
    if ((threadIdx.x & 31) == 0)
      atomicAdd(a.dtable + (int64_t)h * a.n_dist + a.n_dist - 1, far_sum);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= tl.len) continue;
    float* dst = a.dq + (tl.row0 + r) * qs + h * D;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      if (a.add_dq) atomicAdd(dst + tx + 16 * j, dq[i][j]);
      else dst[tx + 16 * j] = dq[i][j];
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) f32_dkdv_kernel(const F32Args a) {
  extern __shared__ float sm[];
  float* K = sm;
  float* V = K + tile_floats<D>();
  float* Q = V + tile_floats<D>();
  float* dO = Q + tile_floats<D>();
  float* P = dO + tile_floats<D>();
  float* S = P + kPFloats;
  const Tile32 tl = a.tiles[blockIdx.x];
  const int h = blockIdx.y, hk = h / (a.H / a.Hkv);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int u0 = tl.row0 - tl.seq0;
  const int64_t qs = (int64_t)a.H * D, ks = (int64_t)a.Hkv * D;
  stage<D>(K, a.k + tl.row0 * ks + hk * D, tl.len, ks);
  stage<D>(V, a.v + tl.row0 * ks + hk * D, tl.len, ks);
  float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < D / 16; ++j) dk[i][j] = dv[i][j] = 0.f;
  // queries that see this tile: its own rows on, or all for a both-way prefix
  const int start = u0 < tl.prefix ? 0 : u0;
  int first, last;
  my_tiles(a, (tl.seq_len - start + kT - 1) / kT, first, last);
  if (first >= last) return;
  for (int t0 = start + first * kT; t0 < start + last * kT; t0 += kT) {
    const int n = min(kT, tl.seq_len - t0);
    __syncthreads();
    stage<D>(Q, a.q + (tl.seq0 + t0) * qs + h * D, n, qs);
    stage<D>(dO, a.dout + (tl.seq0 + t0) * qs + h * D, n, qs);
    __syncthreads();
    float c[4][4], g[4][4];        // [key][query]
    outer<D>(K, Q, ty, tx, c);
    outer<D>(V, dO, ty, tx, g);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * tx + j, pos = t0 + r;
      const float lse = r < n ? a.lse_in[h * a.T + tl.seq0 + pos] : -INFINITY;
      const float Dr = r < n ? a.D[h * a.pitch_d + tl.seq0 + pos] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = u0 + 4 * ty + i;
        float t;
        const float x = score(a, h, c[i][j], pos, u, tl.prefix, t);
        const bool live = lse != -INFINITY && 4 * ty + i < tl.len && x != -INFINITY;
        const float p = live ? expf(x - lse) : 0.f;
        c[i][j] = p;
        g[i][j] = live ? p * (g[i][j] - Dr) * (1.f - t * t) * a.scale : 0.f;
      }
    }
    put(P, ty, tx, c);
    put(S, ty, tx, g);
    __syncthreads();
    accumulate<D>(P, dO, ty, tx, dv);
    accumulate<D>(S, Q, ty, tx, dk);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= tl.len) continue;
    const int64_t at = (tl.row0 + r) * ks + hk * D;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      if (a.add_dkdv) {
        atomicAdd(a.dk + at + tx + 16 * j, dk[i][j]);
        atomicAdd(a.dv + at + tx + 16 * j, dv[i][j]);
      } else {
        a.dk[at + tx + 16 * j] = dk[i][j];
        a.dv[at + tx + 16 * j] = dv[i][j];
      }
    }
  }
}

template <typename K>
cudaError_t run(K kernel, int floats, const F32Args& a, cudaStream_t st) {
  const int bytes = floats * (int)sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(a.n_tiles, a.H, a.splits), kThreads, bytes, st>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd_d(const F32Args& a, cudaStream_t st) {
  constexpr int t = tile_floats<D>();
  static_assert((4 * t + 2 * kPFloats) * 4 <= 227 * 1024, "shared memory budget");
  cudaError_t e = run(f32_dq_kernel<D>, 4 * t + kPFloats, a, st);
  if (e != cudaSuccess) return e;
  return run(f32_dkdv_kernel<D>, 4 * t + 2 * kPFloats, a, st);
}

}  // namespace

cudaError_t launch_f32_fwd(const F32Args& a, int d, cudaStream_t st) {
  if (a.n_tiles == 0) return cudaSuccess;
  return d == 64 ? run(f32_fwd_kernel<64>, 3 * tile_floats<64>() + kPFloats, a, st)
                 : run(f32_fwd_kernel<128>, 3 * tile_floats<128>() + kPFloats, a, st);
}

cudaError_t launch_f32_bwd(const F32Args& a, int d, cudaStream_t st) {
  if (a.n_tiles == 0) return cudaSuccess;
  return d == 64 ? bwd_d<64>(a, st) : bwd_d<128>(a, st);
}

}  // namespace cpattn
