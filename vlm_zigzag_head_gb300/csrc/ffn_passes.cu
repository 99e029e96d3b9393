// The gated feed-forward block: work split of its products, and in fp32 the products of
// up to kSimtRows rows on CUDA cores with the passes between them.
#include <cuda_bf16.h>

#include <algorithm>

#include "ffn.h"
#include "ffn_act.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

__device__ __forceinline__ void add4(float4& v, const float4& w) {
  v.x += w.x;
  v.y += w.y;
  v.z += w.z;
  v.w += w.w;
}

template <int kEpi>
__global__ void __launch_bounds__(256) f32_join_kernel(const __grid_constant__ F32JoinArgs j) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= j.n) return;   // n is a multiple of 8
  auto sum = [&](const float* p) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < j.splits; ++s) add4(v, *reinterpret_cast<const float4*>(p + s * j.n + i));
    return v;
  };
  auto put = [&](float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p + i) = make_float4(f[0], f[1], f[2], f[3]);
  };
  const float4 v = sum(j.partial);
  const float x[4] = {v.x, v.y, v.z, v.w};
  if constexpr (kEpi == GEMM_STORE) {
    put(j.out, x);
  } else if constexpr (kEpi == GEMM_GLU) {
    const float4 w = sum(j.partial + j.splits * j.n);
    const float u[4] = {w.x, w.y, w.z, w.w};
    if (j.gate != nullptr) {
      put(j.gate, x);
      put(j.up, u);
    }
    float h[4], unused;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = activation<false, false>(x[e], j.act, unused) * u[e];
    put(j.out, h);
  } else {
    const float4 a4 = *reinterpret_cast<const float4*>(j.gate + i);
    const float4 u4 = *reinterpret_cast<const float4*>(j.up + i);
    const float gs[4] = {a4.x, a4.y, a4.z, a4.w}, us[4] = {u4.x, u4.y, u4.z, u4.w};
    float h[4], dg[4], du[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float da;
      const float a = activation<true, false>(gs[e], j.act, da);
      h[e] = a * us[e];
      dg[e] = x[e] * us[e] * da;
      du[e] = x[e] * a;
    }
    put(j.dgate, dg);
    put(j.dup, du);
    put(j.out, h);
  }
}

// Tiles of 64 x 64 (64 threads), 8 x 8 sums a thread, k by 16 through shared memory, two
// multiply-adds an instruction.  Bound by the loads from shared memory, whose 64 bytes a
// thread and k take as long as its 64 multiply-adds: 64 rows, forward with the joins, 36
// TFLOP/s (2048 x 6144, 134 us) and 42 (4096 x 12288, 456 us).  Tiles of 128 x 128 where
// they fill the GPU gained up to 1 % in weights' gradients of 64 rows (4096 x 12288: 562 us,
// 560 so) and lost 7 to 10 % for 1 to 32 (32 rows 365 and 395) and, half empty, 40 % of the
// forward beside wide hidden layers (64 x 8192 x 28672: 2063 and 2916).  Calls of more than
// kSimtRows rows take the tensor cores instead.
constexpr int kStep = 16;

constexpr int kTile = 64, kSide = kTile / 8, kThreads = kSide * kSide;

__global__ void __launch_bounds__(kThreads, 8)
    gemm_f32_kernel(const __grid_constant__ GemmF32Args g) {
  constexpr int kPitch = kTile + 4;
  constexpr int kLoads = kTile * kStep / 4 / kThreads;   // 16-byte pieces a thread loads
  __shared__ __align__(16) float as[2][kStep][kPitch], bs[2][kStep][kPitch];
  const int tid = threadIdx.x, tx = tid % kSide, ty = tid / kSide;
  const int m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
  const int output = blockIdx.z / g.splits, share = blockIdx.z % g.splits;
  const int steps = (g.K + kStep - 1) / kStep, all = steps * g.phases;
  const int s0 = (int)((int64_t)all * share / g.splits);
  const int s1 = (int)((int64_t)all * (share + 1) / g.splits);
  float4 ra[kLoads], rb[kLoads];
  // pieces of one operand's tile along its contiguous direction; a piece lies wholly
  // inside the matrix or outside (widths are multiples of 8)
  auto load = [&](const float* p, int64_t sr, int64_t sk, int r0, int rows, int k0,
                  float4 (&r)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = tid + i * kThreads;
      const int k = sk == 1 ? e % 4 * 4 : e / (kTile / 4);
      const int row = sk == 1 ? e / 4 : e % (kTile / 4) * 4;
      r[i] = row < rows - r0 && k0 + k < g.K
                 ? *reinterpret_cast<const float4*>(p + (int64_t)(r0 + row) * sr +
                                                    (int64_t)(k0 + k) * sk)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  auto store = [&](float (*t)[kPitch], int64_t sk, const float4 (&r)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = tid + i * kThreads;
      if (sk == 1) {
        const int k = e % 4 * 4, row = e / 4;
        t[k][row] = r[i].x;
        t[k + 1][row] = r[i].y;
        t[k + 2][row] = r[i].z;
        t[k + 3][row] = r[i].w;
      } else {
        *reinterpret_cast<float4*>(&t[e / (kTile / 4)][e % (kTile / 4) * 4]) = r[i];
      }
    }
  };
  auto fetch = [&](int s) {
    const int phase = s >= steps, k = (s - phase * steps) * kStep, i = output + phase;
    load(g.a[i], g.sam, g.sak, m0, g.M, k, ra);
    load(g.b[i], g.sbn[i], g.sbk[i], n0, g.N, k, rb);
  };
  uint64_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[i][c] = 0ull;
  if (s0 < s1) {
    fetch(s0);
    store(as[0], g.sak, ra);
    store(bs[0], g.sbk[0], rb);
  }
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    const int cur = (s - s0) & 1;
    if (s + 1 < s1) fetch(s + 1);
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      // rows ty * 4 and half a tile further on, columns tx * 4 and half a tile on
      const float4 a0 = *reinterpret_cast<const float4*>(&as[cur][k][ty * 4]);
      const float4 a1 = *reinterpret_cast<const float4*>(&as[cur][k][kTile / 2 + ty * 4]);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(&bs[cur][k][tx * 4]);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(&bs[cur][k][kTile / 2 + tx * 4]);
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
      store(bs[cur ^ 1], g.sbk[0], rb);   // both phases' run the same way
    }
    __syncthreads();
  }
  float* out = g.out[output] + (int64_t)share * g.M * g.N;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + (i / 4) * (kTile / 2) + ty * 4 + i % 4;
    if (m >= g.M) continue;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = n0 + c * (kTile / 2) + tx * 4;
      if (n >= g.N) continue;   // N is a multiple of 8
      float4 v;
      unpack2(acc[i][2 * c], v.x, v.y);
      unpack2(acc[i][2 * c + 1], v.z, v.w);
      *reinterpret_cast<float4*>(out + (int64_t)m * g.N + n) = v;
    }
  }
}

}  // namespace

// A tile half as wide reads three quarters of the operands for half the products.
GemmCost gemm_cost(int epilogue, int tile_n) {
  return {tile_n, tile_n == 256 ? 0.29 : 0.22,
          (epilogue == GEMM_STORE ? 2. : 4.) * tile_n / 256, 4};
}
// Six products a k tile.
GemmCost split_cost(int epilogue) {
  return {kSplitN, 0.95, epilogue == GEMM_STORE ? 2. : 6., 2};
}

// Adding up the shares of a tile: each writes its sums and one reads them all, through L2
// (taken as half of that, forward of 2048 x 2048 x 6144 shares its last tiles: 99 -> 104 us).
static double unit_time(const GemmCut& c, const GemmCost& cost) {
  return (c.k_tiles + c.shares - 1) / c.shares * cost.step +
         (c.shares > 1 ? 1.5 + 0.4 * c.shares * cost.tile_n / 64 : 0.);
}

// About the time of a launch, its units dealt out to the pairs to and fro.
static double launch_time(const GemmCut* p, int n, int pairs, const GemmCost& cost) {
  struct {
    int64_t end;
    double time;
  } run[2 * kGemmProblems];   // of equal units
  int runs = 0;
  int64_t units = 0;
  double sum = 0, longest = 0;
  auto add = [&](int64_t count, double time) {
    if (count == 0) return;
    units += count;
    run[runs++] = {units, time};
    sum += count * time;
    longest = std::max(longest, time);
  };
  for (int i = 0; i < n; ++i) {
    add(p[i].whole, p[i].k_tiles * cost.step);
    if (p[i].shares > 1)
      add((p[i].tiles - p[i].whole) * p[i].shares, unit_time(p[i], cost));
  }
  if (units <= pairs) return longest + cost.epilogue;
  double time = sum / pairs;
  if (units <= 2 * pairs) {
    auto at = [&](int64_t u) {
      int i = 0;
      while (i < runs && u >= run[i].end) ++i;
      return i < runs ? run[i].time : 0.;
    };
    auto pair = [&](int64_t i) {   // its first unit and its second
      if (i >= 0 && i < pairs) time = std::max(time, at(i) + at(2 * pairs - 1 - i));
    };
    pair(0);
    for (int i = 0; i < runs; ++i) {   // where one of the two changes
      pair(run[i].end);
      pair(2 * pairs - run[i].end);
    }
  } else if (units % pairs != 0) {
    time += run[runs - 1].time * (1. - (double)(units % pairs) / pairs);
  }
  return std::max(time, longest) + cost.epilogue;
}

double cut_products(GemmCut* p, int n, int pairs, const GemmCost& cost) {
  int64_t total = 0, work = 0;
  for (int i = 0; i < n; ++i) {
    total += p[i].tiles;
    work += p[i].tiles * p[i].k_tiles;
    p[i].whole = p[i].tiles;
    p[i].shares = 1;
  }
  double best = launch_time(p, n, pairs, cost);
  if (work == 0) return best;   // no rows: nothing to cut
  auto consider = [&](const GemmCut* q) {
    const double t = launch_time(q, n, pairs, cost);
    if (t >= best) return;
    best = t;
    std::copy(q, q + n, p);
  };
  GemmCut q[kGemmProblems];

  // The last round's tiles: the product whose units are longest is cut further while that
  // pays and there are pairs left and enough k tiles a share.
  std::copy(p, p + n, q);
  int tail[kGemmProblems] = {}, left = (int)(total % pairs), free = pairs - left;
  for (int i = n - 1; i >= 0; --i) {
    tail[i] = (int)(p[i].tiles < left ? p[i].tiles : left);
    left -= tail[i];
  }
  for (;;) {
    int i = -1;
    for (int j = 0; j < n; ++j)
      if (tail[j] && (i < 0 || unit_time(q[j], cost) > unit_time(q[i], cost))) i = j;
    if (i < 0 || tail[i] > free || q[i].k_tiles / (q[i].shares + 1) < cost.least_k) break;
    GemmCut more = q[i];
    ++more.shares;
    more.whole = more.tiles - tail[i];
    if (unit_time(more, cost) >= unit_time(q[i], cost)) break;
    free -= tail[i];
    q[i] = more;
  }
  consider(q);

  // Or every product with more k than a pair's part of the whole work (so that these are
  // fewer tiles than pairs).
  const int part = (int)std::min<int64_t>((work + pairs - 1) / pairs, 1 << 30);
  bool any = false;
  for (int i = 0; i < n; ++i) {
    q[i].whole = p[i].tiles;
    q[i].shares = 1;
    const int most = std::min((p[i].k_tiles + part - 1) / part, p[i].k_tiles / cost.least_k);
    for (GemmCut more = q[i]; more.shares < most;) {
      more.whole = 0;
      ++more.shares;
      if (unit_time(more, cost) >= unit_time(q[i], cost)) break;
      q[i] = more;
      any = true;
    }
  }
  if (any) consider(q);
  return best;
}

cudaError_t launch_f32_join(const F32JoinArgs& j, int epilogue, cudaStream_t st) {
  const int64_t blocks = (j.n / 4 + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (epilogue == GEMM_STORE) f32_join_kernel<GEMM_STORE><<<(unsigned)blocks, 256, 0, st>>>(j);
  else if (epilogue == GEMM_GLU) f32_join_kernel<GEMM_GLU><<<(unsigned)blocks, 256, 0, st>>>(j);
  else f32_join_kernel<GEMM_DGLU><<<(unsigned)blocks, 256, 0, st>>>(j);
  return cudaGetLastError();
}

int share_f32(int64_t M, int64_t N, int64_t K, int outputs, int phases, int sms) {
  const int64_t tiles = ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile) * outputs;
  if (tiles == 0) return 1;
  // eight blocks of 64 threads an SM, of four steps at least
  const int64_t steps = (K + kStep - 1) / kStep * phases;
  int64_t s = 8 * (int64_t)sms / tiles;
  if (s > steps / 4) s = steps / 4;
  if (s > 64) s = 64;
  return s > 1 ? (int)s : 1;
}

cudaError_t launch_gemm_f32(const GemmF32Args& g, cudaStream_t st) {
  const int64_t nt = ((int64_t)g.N + kTile - 1) / kTile;
  if (nt > 65535 || g.splits * g.outputs > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(((int64_t)g.M + kTile - 1) / kTile), (unsigned)nt,
                  (unsigned)(g.splits * g.outputs));
  gemm_f32_kernel<<<grid, kThreads, 0, st>>>(g);
  return cudaGetLastError();
}

}  // namespace cpattn
