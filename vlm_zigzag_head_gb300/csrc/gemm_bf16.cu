// Matrix products of the gated feed-forward block on the 5th-generation tensor
// cores (sm_103a), with its activation in their epilogues.
//
//   C[m][n] = sum_k A(m, k) B(n, k),  bf16 operands, fp32 sums in tensor memory
//
// A tile is 128 x 256 (gate and up: 128 x 128 of each, so that both halves of a pair
// meet in one epilogue), k goes by 64.  Operands come by TMA in the 128-byte swizzle,
// K-major or MN-major as they lie in memory: no product needs a transposed copy.  The
// kernel is persistent: CTAs walk (tile, share of k) units, and the two accumulators
// in tensor memory let a tile's epilogue run under the next one's products.
//
// Warp roles (384 threads):
//   warp 0       TMA producer (one lane)
//   warp 1       TMEM allocation; lane 0 issues every tcgen05.mma
//   warps 4..11  epilogue: TMEM lane quarter w % 4, column half (w - 4) / 4
//
// Rows and columns past the matrices' ends are zeros by TMA's fill and are not
// stored.
#include <cuda_bf16.h>

#include "check.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kStages = 4;
constexpr int kEpiWarps = 8;
constexpr int kTileA = kGemmM * kGemmK * 2, kTileB = kGemmN * kGemmK * 2;   // bytes
constexpr int kStage = kTileA + kTileB;
constexpr int kSmem = kStages * kStage + 256 + 1024;   // barriers; slack for alignment
constexpr uint32_t kTmemCols = 512;
constexpr long long kDrainLimit = 1LL << 24;
// m tiles whose n tiles are walked together: about square patches of tiles run at a
// time, which reads the least of A and B
constexpr int kGroupM = 16;
static_assert(kSmem <= 227 * 1024, "shared memory budget");

struct Bars {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

struct Unit {
  int m, n, split, k0, k1;   // tile, share of k, its k tiles
};
__device__ __forceinline__ Unit unit_at(const GemmArgs& g, int u) {
  Unit r;
  const int tile = u / g.splits;
  r.split = u % g.splits;
  const int per_group = kGroupM * g.n_tiles;
  const int first = tile / per_group * kGroupM, in = tile % per_group;
  const int rows = min(kGroupM, g.m_tiles - first);
  r.m = first + in % rows;
  r.n = in / rows;
  r.k0 = (int)((long long)g.k_tiles * r.split / g.splits);
  r.k1 = (int)((long long)g.k_tiles * (r.split + 1) / g.splits);
  return r;
}

__device__ __forceinline__ void record_timeout(int32_t* status, volatile int* abort, int site) {
  if (atomicCAS(&status[0], 0, 1) == 0) status[1] = site;
  *abort = 1;
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// 32 columns of one row, from column n on (N is a multiple of 8).
__device__ __forceinline__ void store_bf16(void* out, int64_t at, int n, int N, const float* f) {
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(out) + at;
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    if (n + i < N) *reinterpret_cast<uint4*>(p + i) = pack8(f + i);
}
__device__ __forceinline__ void store_f32(float* out, int64_t at, int n, int N, const float* f) {
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    if (n + i < N)
      *reinterpret_cast<float4*>(out + at + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}

__device__ __forceinline__ void load_acc(uint32_t taddr, float (&f)[32]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_ld_wait();
  reg_fence32(r);
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
}

// dgate, dup and h of 32 columns of one row, from dh and the kept gate and up.
__device__ __forceinline__ void hidden_gradients(const GemmArgs& g, int64_t at, int n,
                                                 const float* dh) {
  const __nv_bfloat16* pg = static_cast<const __nv_bfloat16*>(g.gate) + at;
  const __nv_bfloat16* pu = static_cast<const __nv_bfloat16*>(g.up) + at;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    if (n + i >= g.N) continue;
    float gate[8], up[8], h[8];
    unpack8(*reinterpret_cast<const uint4*>(pg + i), gate);
    unpack8(*reinterpret_cast<const uint4*>(pu + i), up);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float da;
      const float a = activation<true>(gate[e], g.act, da), d = dh[i + e];
      h[e] = a * up[e];
      gate[e] = d * up[e] * da;
      up[e] = d * a;
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.dgate) + at + i) = pack8(gate);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.dup) + at + i) = pack8(up);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.out[0]) + at + i) = pack8(h);
  }
}

template <bool kAMN, bool kBMN, int kEpi>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + kStages * kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = g.m_tiles * g.n_tiles * g.splits;
  volatile int* abort = &bars->abort;
  const long long lim = g.wait_limit;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->acc_full[s], 1);
      mbar_init(&bars->acc_empty[s], kEpiWarps);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int j = 0;   // k tiles so far, across units
      for (int u = blockIdx.x; u < units && !*abort; u += gridDim.x) {
        const Unit t = unit_at(g, u);
        const bool second = t.m >= g.m_split;
        const int m0 = (t.m - (second ? g.m_split : 0)) * kGemmM;
        const int n0 = t.n * (kEpi == GEMM_GLU ? kGemmN / 2 : kGemmN);
        if (!CP_IN_RANGE(m0, 0, g.M, g.status, 301) || !CP_IN_RANGE(n0, 0, g.N, g.status, 302)) {
          *abort = 1;
          break;
        }
        for (int k = t.k0; k < t.k1; ++k, ++j) {
          const int st = j % kStages;
          if (j >= kStages && !mbar_wait(&bars->empty[st], ((j / kStages) - 1) & 1, lim, abort)) {
            record_timeout(g.status, abort, 31);
            break;
          }
          const int src = k >= g.k_split;
          const int kk = (k - (src ? g.k_split : 0)) * kGemmK;
          const CUtensorMap* ma = &g.a[second || src];
          const CUtensorMap* mb = &g.b[src];
          uint8_t* pa = smem + st * kStage;
          uint8_t* pb = pa + kTileA;
          uint64_t* full = &bars->full[st];
          mbar_expect_tx(full, kStage);
          if constexpr (kAMN) {
            for (int i = 0; i < kGemmM / 64; ++i)
              tma_load_2d(ma, full, pa + i * 64 * kGemmK * 2, m0 + i * 64, kk);
          } else {
            tma_load_2d(ma, full, pa, kk, m0);
          }
          if constexpr (kEpi == GEMM_GLU) {   // 128 rows of each weight
            tma_load_2d(&g.b[0], full, pb, kk, n0);
            tma_load_2d(&g.b[1], full, pb + kTileB / 2, kk, n0);
          } else if constexpr (kBMN) {
            for (int i = 0; i < kGemmN / 64; ++i)
              tma_load_2d(mb, full, pb + i * 64 * kGemmK * 2, n0 + i * 64, kk);
          } else {
            tma_load_2d(mb, full, pb, kk, n0);
            tma_load_2d(mb, full, pb + kTileB / 2, kk, n0 + kGemmN / 2);
          }
        }
      }
      // every load must land before the CTA exits (normally they have: the MMA
      // issuer waited for them)
      int zero = 0;
      for (int x = j - kStages; x < j; ++x)
        if (x >= 0) mbar_wait(&bars->full[x % kStages], (x / kStages) & 1, kDrainLimit, &zero);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(kGemmM, kGemmN, kAMN, kBMN);
      bool ok = true;
      int j = 0, n = 0;   // k tiles and units so far
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++n) {
        const Unit t = unit_at(g, u);
        const int s = n & 1;
        if (n >= 2 && !mbar_wait(&bars->acc_empty[s], ((n >> 1) - 1) & 1, lim, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int k = t.k0; k < t.k1; ++k, ++j) {
          const int st = j % kStages;
          if (!mbar_wait(&bars->full[st], (j / kStages) & 1, lim, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t pa = smem_u32(smem + st * kStage), pb = pa + kTileA;
#pragma unroll
          for (int i = 0; i < kGemmK / 16; ++i) {
            // 16 k further: 32 bytes along a K-major row, 16 rows of an MN-major box
            const uint64_t da = kAMN ? sdesc_sw128(pa + i * 2048, 64 * kGemmK * 2, 1024)
                                     : sdesc_sw128(pa + i * 32, 16, 1024);
            const uint64_t db = kBMN ? sdesc_sw128(pb + i * 2048, 64 * kGemmK * 2, 1024)
                                     : sdesc_sw128(pb + i * 32, 16, 1024);
            mma_bf16(tmem + s * kGemmN, da, db, idesc, (k > t.k0 || i > 0) ? 1u : 0u);
          }
          mma_commit(&bars->empty[st]);
        }
        if (!ok) break;
        mma_commit(&bars->acc_full[s]);
      }
      if (!ok) {
        record_timeout(g.status, abort, 32);
        // nothing issued by this thread may still be running at exit
        mma_commit(&bars->drain);
        int zero = 0;
        mbar_wait(&bars->drain, 0, kDrainLimit, &zero);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    int n = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++n) {
      const Unit t = unit_at(g, u);
      const int s = n & 1;
      if (!mbar_wait(&bars->acc_full[s], (n >> 1) & 1, lim, abort)) {
        if (lane == 0) record_timeout(g.status, abort, 33);
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + s * kGemmN;
      const bool second = t.m >= g.m_split;
      const int row = (t.m - (second ? g.m_split : 0)) * kGemmM + quarter * 32 + lane;
      const bool in = row < g.M;
      const int64_t at = (int64_t)row * g.N;
      if constexpr (kEpi == GEMM_GLU) {
        const int64_t share = (int64_t)g.M * g.N;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int col = half * 64 + c * 32, nc = t.n * (kGemmN / 2) + col;
          float x[32], v[32];
          load_acc(acc + col, x);
          load_acc(acc + kGemmN / 2 + col, v);
          if (in && g.splits > 1) {
            store_f32(g.partial + t.split * share, at + nc, nc, g.N, x);
            store_f32(g.partial + (g.splits + t.split) * share, at + nc, nc, g.N, v);
          } else if (in) {
            if (g.gate != nullptr) {
              store_bf16(g.gate, at + nc, nc, g.N, x);
              store_bf16(g.up, at + nc, nc, g.N, v);
            }
            float unused;
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = activation<false>(x[i], g.act, unused) * v[i];
            store_bf16(g.out[0], at + nc, nc, g.N, x);
          }
          __syncwarp();   // the next load of the accumulator is the whole warp's
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int col = half * 128 + c * 32, nc = t.n * kGemmN + col;
          float x[32];
          load_acc(acc + col, x);
          if (in && g.splits > 1) {
            store_f32(g.partial + (int64_t)(t.split + (second ? g.splits : 0)) * g.M * g.N, at + nc,
                      nc, g.N, x);
          } else if (in && kEpi == GEMM_STORE) {
            if (g.out_f32) store_f32(static_cast<float*>(g.out[second]), at + nc, nc, g.N, x);
            else store_bf16(g.out[second], at + nc, nc, g.N, x);
          } else if (in) {
            hidden_gradients(g, at + nc, nc, x);
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->acc_empty[s]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool kAMN, bool kBMN, int kEpi>
cudaError_t launch_t(const GemmArgs& g, int sms, cudaStream_t st) {
  auto kernel = gemm_kernel<kAMN, kBMN, kEpi>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)g.m_tiles * g.n_tiles * g.splits;
  if (units < 1 || units > 0x3fffffff) return cudaErrorInvalidConfiguration;
  kernel<<<(unsigned)(units < sms ? units : sms), kThreads, kSmem, st>>>(g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_bf16(const GemmArgs& g, int epilogue, bool a_mn, bool b_mn, int sms,
                             cudaStream_t st) {
  if (epilogue == GEMM_GLU) return launch_t<false, false, GEMM_GLU>(g, sms, st);
  if (epilogue == GEMM_DGLU) return launch_t<false, true, GEMM_DGLU>(g, sms, st);
  if (a_mn) return launch_t<true, true, GEMM_STORE>(g, sms, st);
  return b_mn ? launch_t<false, true, GEMM_STORE>(g, sms, st)
              : launch_t<false, false, GEMM_STORE>(g, sms, st);
}

}  // namespace cpattn
