// Matrix products of the gated feed-forward block in fp32 on the 5th-generation tensor
// cores (sm_103a), with its activation in their epilogues.
//
//   C[m][n] = sum_k A(m, k) B(n, k),  every operand x = hi + mid + lo, three bf16 values
//
// fp32 has 24 bits and bf16 has 8: hi is x cut off, mid the rest rounded, lo what is
// left, exactly (down to about 2^-110, where lo leaves bf16's range).  Of the nine
// products of parts the six largest are taken,
//   hi hi + hi mid + mid hi + mid mid + hi lo + lo hi;
// the others are below 2^-23 of |A| |B| and of random sign (2^-26 in the mean).  The
// tensor cores cut their sums off at each step, which grows with k: a chain of 4096 was
// off by 4e-6 of the result, ordered fp32 sums by 1e-6.  So a chain ends after kChain k,
// and its sums are added in fp32 registers: 2.3e-7.
//
// Six bf16 products take a third of the time that CUDA cores need at their peak, which
// shared memory keeps them from (45 TFLOP/s here): see the figures at the launch.
//
// Pairs of CTAs as in gemm_bf16.cu, tiles of 256 x 128 (gate and up: 64 columns of each).
// A slot of shared memory holds a 64 deep tile of one plane of A and of B; each of the
// three pairs of slots of a k tile is loaded once and used by the terms that it completes.
// Epilogue warps hold 64 sums a thread, a row of 64 columns or 32 of gate and of up, and
// read and write memory directly: a lane's 128 bytes are a line of its own, and with six
// products to a k tile there is time for it.
#include <cuda_bf16.h>

#include "check.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "gemm_units.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kN = kSplitN;
constexpr int kRows = kGemmM / 2, kRowsB = kN / 2;   // of A and B in one CTA
constexpr int kTileA = kRows * kGemmK * 2, kTileB = kRowsB * kGemmK * 2;
constexpr int kSlot = kTileA + kTileB;
constexpr int kDepth = 3;                            // k tiles in shared memory
constexpr int kChain = 4;                            // k tiles of one accumulation
constexpr int kBarsAt = 3 * kDepth * kSlot;
constexpr int kSmem = kBarsAt + 256 + 1024;          // slack for alignment
static_assert(kSmem <= 227 * 1024, "shared memory budget");
constexpr uint32_t kTmemCols = 2 * kN;               // two accumulators

struct Bars {
  uint64_t full[3 * kDepth];   // first CTA: both CTAs' loads of a slot have landed
  uint64_t empty[kDepth];      // both: the MMAs of a k tile are done
  uint64_t acc_full[2];        // both: a chain's products are done
  uint64_t acc_empty[2];       // first CTA: both CTAs' epilogues have read them
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// Eight values as three planes' 16-byte pieces.
__device__ __forceinline__ void split8(const float (&f)[8], uint4 (&plane)[3]) {
  uint32_t w[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = f[2 * i], b = f[2 * i + 1];
    w[0][i] = upper_halves(a, b);
    const float ra = a - __uint_as_float(w[0][i] << 16);
    const float rb = b - __uint_as_float(w[0][i] & 0xffff0000u);
    w[1][i] = pack_bf16x2(ra, rb);
    w[2][i] = pack_bf16x2(ra - __uint_as_float(w[1][i] << 16),
                          rb - __uint_as_float(w[1][i] & 0xffff0000u));
  }
#pragma unroll
  for (int p = 0; p < 3; ++p) plane[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

template <int kEpi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    split_gemm_kernel(const __grid_constant__ SplitArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + kBarsAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int units = g.units;
  // the units are dealt out to and fro: the longest come first
  auto unit_of = [&](int r) { return r * pairs + (r & 1 ? pairs - 1 - pair : pair); };
  griddep_launch_dependents();   // the next product waits for this one
  volatile int* abort = &bars->abort;
  const long long lim = g.wait_limit;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 3 * kDepth; ++s) mbar_init(&bars->full[s], 1);
    for (int s = 0; s < kDepth; ++s) mbar_init(&bars->empty[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->acc_full[s], 1);
      mbar_init(&bars->acc_empty[s], 2 * kEpiWarps);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&bars->tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the other CTA's barriers are ready too
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // What the launch before wrote; and the waits below are bounded, so none may begin
  // while that launch still runs.
  griddep_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int j = 0;   // k tiles so far, across units
      for (int r = 0; unit_of(r) < units && !*abort; ++r) {
        const Unit t = unit_at(g, unit_of(r));
        const SplitProblem& p = g.p[t.p];
        const bool second = t.m >= p.m_split, a_mn = p.a_mn, b_mn = p.b_mn;
        const int k_split = p.k_split;
        int m0 = (t.m - (second ? p.m_split : 0)) * kGemmM + rank * kRows;
        int n0 = kEpi == GEMM_GLU ? t.n * kRowsB : t.n * kN + rank * kRowsB;
        if (!CP_IN_RANGE(m0, 0, p.M + kRows, g.status, 311)) m0 = 0;
        if (!CP_IN_RANGE(n0, 0, p.N + kRows, g.status, 312)) n0 = 0;
        for (int k = t.k0; k < t.k1; ++k, ++j) {
          const int st = j % kDepth;
          if (j >= kDepth &&
              !mbar_wait_cluster(&bars->empty[st], ((j / kDepth) - 1) & 1, lim, abort)) {
            record_timeout(g.status, abort, 41);
            break;
          }
          const bool next = k >= k_split;
          const int kk = (k - (next ? k_split : 0)) * kGemmK;
          const CUtensorMap* ma = &p.a[second || next];
          const CUtensorMap* mb = &p.b[kEpi == GEMM_GLU ? rank : next];   // gate or up
          for (int plane = 0; plane < 3; ++plane) {
            const int slot = st * 3 + plane;
            uint8_t* dst = smem + slot * kSlot;
            const uint32_t full = in_first_cta(&bars->full[slot]);
            if (rank == 0) mbar_expect_tx(&bars->full[slot], 2 * kSlot);   // both CTAs' parts
            if (a_mn) {
#pragma unroll
              for (int i = 0; i < kRows / 64; ++i)
                tma_load_3d_pair(ma, full, dst + i * 64 * kGemmK * 2, m0 + i * 64, kk, plane);
            } else {
              tma_load_3d_pair(ma, full, dst, kk, m0, plane);
            }
            if (b_mn) tma_load_3d_pair(mb, full, dst + kTileA, n0, kk, plane);
            else tma_load_3d_pair(mb, full, dst + kTileA, kk, n0, plane);
          }
        }
      }
      // no load may be on its way when the CTA exits
      int zero = 0;
      for (int x = j - kDepth; x < j; ++x)
        if (x >= 0)
          mbar_wait_cluster(&bars->empty[x % kDepth], (x / kDepth) & 1, kLandLimit, &zero);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      bool ok = true;
      int j = 0, n = 0;   // k tiles and chains so far
      Work t = work_at(g, pair), next = t;
      for (int r = 0; ok && unit_of(r) < units; ++r, t = next) {
        if (unit_of(r + 1) < units) next = work_at(g, unit_of(r + 1));
        const int a_mn = g.p[t.p].a_mn, b_mn = g.p[t.p].b_mn;
        const uint32_t idesc = idesc_bf16(kGemmM, kN, a_mn, b_mn);
        // 16 k further: 32 bytes along a K-major row, 16 rows of an MN-major box
        const uint32_t a_step = a_mn ? 2048 : 32, b_step = b_mn ? 2048 : 32;
        const uint32_t a_lbo = a_mn ? 64 * kGemmK * 2 : 16, b_lbo = b_mn ? 64 * kGemmK * 2 : 16;
        for (int k = t.k0; ok && k < t.k1; ++k, ++j) {
          const int st = j % kDepth, s = n & 1;
          const bool starts = (k - t.k0) % kChain == 0;
          if (starts) {
            if (n >= 2 &&
                !mbar_wait_cluster(&bars->acc_empty[s], ((n >> 1) - 1) & 1, lim, abort)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          const uint32_t base = smem_u32(smem + st * 3 * kSlot);
          auto term = [&](int a, int b, bool first) {
            const uint32_t pa = base + a * kSlot, pb = base + b * kSlot + kTileA;
#pragma unroll
            for (int i = 0; i < kGemmK / 16; ++i)
              mma_bf16_pair(tmem + s * kN, sdesc_sw128(pa + i * a_step, a_lbo, 1024),
                            sdesc_sw128(pb + i * b_step, b_lbo, 1024), idesc,
                            first && i == 0 ? 0u : 1u);
          };
          for (int plane = 0; plane < 3; ++plane) {
            if (!mbar_wait_cluster(&bars->full[st * 3 + plane], (j / kDepth) & 1, lim, abort)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (plane == 0) {
              term(0, 0, starts);
            } else if (plane == 1) {
              term(0, 1, false);
              term(1, 0, false);
              term(1, 1, false);
            } else {
              term(0, 2, false);
              term(2, 0, false);
            }
          }
          if (!ok) break;
          mma_commit_pair(&bars->empty[st]);
          if (k + 1 == t.k1 || (k + 1 - t.k0) % kChain == 0) {
            mma_commit_pair(&bars->acc_full[s]);
            ++n;
          }
        }
      }
      if (!ok) {
        record_timeout(g.status, abort, 42);
        // nothing issued by this thread may still be running at exit
        mma_commit_pair(&bars->drain);
        int zero = 0;
        mbar_wait_cluster(&bars->drain, 0, kDrainLimit, &zero);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    // a thread's two runs of 32 columns in the accumulator
    const int col0 = half * (kEpi == GEMM_GLU ? 32 : 64);
    const int col1 = kEpi == GEMM_GLU ? kN / 2 + col0 : col0 + 32;
    const int tile_row = rank * kRows + quarter * 32 + lane;
    int n = 0;   // chains so far
    bool ok = true;
    for (int r = 0; ok && unit_of(r) < units; ++r) {
      const Unit t = unit_at(g, unit_of(r));
      const SplitProblem& p = g.p[t.p];
      const bool second = t.m >= p.m_split;
      const int row = (t.m - (second ? p.m_split : 0)) * kGemmM + tile_row;
      const bool in = row < p.M;
      float x[2][32];
#pragma unroll
      for (int i = 0; i < 32; ++i) x[0][i] = x[1][i] = 0.f;
      for (int k = t.k0; k < t.k1; k += kChain, ++n) {
        const int s = n & 1;
        if (!__all_sync(0xffffffffu,
                        mbar_wait_cluster(&bars->acc_full[s], (n >> 1) & 1, lim, abort))) {
          if (lane == 0) record_timeout(g.status, abort, 43);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + s * kN;
        float f[32];
        load_acc(acc + col0, f);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[0][i] += f[i];
        load_acc(acc + col1, f);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[1][i] += f[i];
        tc_fence_before();   // the next products may overwrite the accumulator
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(in_first_cta(&bars->acc_empty[s]));
      }
      if (!ok) break;
      if (t.slot >= 0) {
        if (in) {
          store_partial<kN>(g.partial, t.slot, col0, tile_row, x[0]);
          store_partial<kN>(g.partial, t.slot, col1, tile_row, x[1]);
        }
        // this warp's rows of all shares: the last to get here goes on with them
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0) {
          int32_t* ticket = g.tickets + t.ticket * kTickets + rank * kEpiWarps + warp - 4;
          last = atomicAdd(ticket, 1) == p.shares - 1;
          if (last) *ticket = 0;
          __threadfence();
        }
        if (!__shfl_sync(0xffffffffu, last, 0)) continue;
        if (in) {
          load_partials<kN>(g.partial, t.slot - t.share, p.shares, col0, tile_row, x[0]);
          load_partials<kN>(g.partial, t.slot - t.share, p.shares, col1, tile_row, x[1]);
        }
      }
      if (in) {
        const int64_t line = (int64_t)row * p.N, plane = (int64_t)p.M * p.N;
        auto eight = [](const float* f, float (&v)[8]) {
  #pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = f[e];
        };
        auto put = [](float* q, const float (&v)[8]) {
          reinterpret_cast<float4*>(q)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(q)[1] = make_float4(v[4], v[5], v[6], v[7]);
        };
        auto put_planes = [&](__nv_bfloat16* q, const float (&v)[8]) {
          uint4 w[3];
          split8(v, w);
  #pragma unroll
          for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4*>(q + i * plane) = w[i];
        };
        if constexpr (kEpi == GEMM_GLU) {
          const int first = t.n * (kN / 2) + half * 32;
  #pragma unroll
          for (int q = 0; q < 4; ++q) {   // eight columns at a time; N is a multiple of 8
            if (first + 8 * q >= p.N) break;
            const int64_t at = line + first + 8 * q;
            float gate[8], up[8], unused;
            eight(x[0] + 8 * q, gate);
            eight(x[1] + 8 * q, up);
            if (g.gate != nullptr) {
              put(g.gate + at, gate);
              put(g.up + at, up);
            }
  #pragma unroll
            for (int e = 0; e < 8; ++e)
              gate[e] = activation<false, false>(gate[e], g.act, unused) * up[e];
            put_planes(g.h + at, gate);
          }
        } else {
  #pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int col = t.n * kN + half * 64 + 8 * q;
            if (col >= p.N) break;
            const int64_t at = line + col;
            float v[8];
            eight(x[q / 4] + 8 * (q % 4), v);
            if constexpr (kEpi == GEMM_STORE) {
              put(p.out[second] + at, v);
            } else {
              float gate[8], up[8];
              *reinterpret_cast<float4*>(gate) = *reinterpret_cast<const float4*>(g.gate + at);
              *reinterpret_cast<float4*>(gate + 4) = *reinterpret_cast<const float4*>(g.gate + at + 4);
              *reinterpret_cast<float4*>(up) = *reinterpret_cast<const float4*>(g.up + at);
              *reinterpret_cast<float4*>(up + 4) = *reinterpret_cast<const float4*>(g.up + at + 4);
              float h[8];
  #pragma unroll
              for (int e = 0; e < 8; ++e) {
                float da;
                const float a = activation<true, false>(gate[e], g.act, da), dh = v[e];
                h[e] = a * up[e];
                gate[e] = dh * up[e] * da;
                up[e] = dh * a;
              }
              put_planes(g.dgate + at, gate);
              put_planes(g.dup + at, up);
              put_planes(g.h + at, h);
            }
          }
        }
      }
      __syncwarp();   // the next loads of an accumulator are the whole warp's
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the other CTA's MMAs and arrivals no longer need this one
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// 10 bytes an element, eight elements a thread.
constexpr int kSplitThreads = 256;
__global__ void __launch_bounds__(kSplitThreads) split_kernel(const __grid_constant__ SplitPass s) {
  griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < s.clear; i += kSplitThreads) s.status[i] = 0;
  const auto& m = s.m[blockIdx.y];
  const int pieces = m.cols / 8;
  const int64_t n = m.rows * pieces;
  for (int64_t i = (int64_t)blockIdx.x * kSplitThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kSplitThreads) {
    int64_t at = i * 8;
    if (m.stride != m.cols) {
      const int64_t row = i / pieces;
      at = row * m.stride + (i - row * pieces) * 8;
    }
    float f[8];
    *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(m.src + at);
    *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(m.src + at + 4);
    uint4 w[3];
    split8(f, w);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint4*>(m.planes + p * n * 8 + i * 8) = w[p];
  }
}

template <int kEpi>
cudaError_t launch_t(const SplitArgs& g, int sms, cudaStream_t st) {
  auto kernel = split_gemm_kernel<kEpi>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int pairs = g.units < sms / 2 ? g.units : sms / 2;
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, g);
}

}  // namespace

cudaError_t launch_gemm_split(const SplitArgs& g, int epilogue, int sms, cudaStream_t st) {
  if (epilogue == GEMM_GLU) return launch_t<GEMM_GLU>(g, sms, st);
  if (epilogue == GEMM_DGLU) return launch_t<GEMM_DGLU>(g, sms, st);
  return launch_t<GEMM_STORE>(g, sms, st);
}

cudaError_t launch_split(const SplitPass& s, cudaStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < s.n; ++i) {
    const int64_t n = s.m[i].rows * (s.m[i].cols / 8);
    if (n > most) most = n;
  }
  int64_t blocks = (most + kSplitThreads - 1) / kSplitThreads;
  if (blocks > 2048) blocks = 2048;
  if (blocks < 1 || s.n < 1) return cudaErrorInvalidConfiguration;
  split_kernel<<<dim3((unsigned)blocks, (unsigned)s.n), kSplitThreads, 0, st>>>(s);
  return cudaGetLastError();
}

}  // namespace cpattn
