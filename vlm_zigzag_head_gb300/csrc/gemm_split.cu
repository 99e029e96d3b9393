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
// tensor cores cut their sums off at each step, which grows with the steps: a chain of 4096
// k was off by 4e-6 of the result, fp32 sums by 1e-6.  So a chain ends after kChain k tiles,
// and its sums are added in fp32 registers; and the five small products, whose steps would
// cut off the large one's sum, have sums of their own (together 2.3e-6 at 512 k, apart 2.4e-7, fp32 sums 4e-7; at 4096 k 2.6e-7 and 1.2e-6).
//
// Six bf16 products are quicker than one on CUDA cores: 2048 x 2048 x 6144 forward 761 us
// (1219 TFLOP/s of bf16, 203 of fp32), on CUDA cores 3364.  Up to kSimtRows rows the planes
// of the weights cost the forward more than that saves (2048 x 6144, 64 rows: 163 us, on
// CUDA cores 134; 128 rows: 165 and 238); its backward is about as long either way (64 rows:
// 229 and 240; 128 rows: 268 and 442).
//
// Pairs of CTAs as in gemm_bf16.cu, tiles of 256 x 128 (gate and up: 64 columns of each).
// A slot of shared memory holds a 64 deep tile of one plane of A and of B; each of the
// three pairs of slots of a k tile is loaded once and used by the terms that it completes.
// Epilogue warps hold 64 sums a thread, a row of 64 columns or 32 of gate and of up.  Shared
// memory is full, so rows go to memory from registers: four lanes exchange their pieces,
// and write 64 bytes of a row at a time.  (Each lane its own row instead, 16 bytes in each
// of 32 lines: hidden gradients of 2048 x 2048 x 6144 466 us, 324 so.)
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
constexpr uint32_t kTmemCols = 4 * kN;   // two accumulators of hi hi, and of the rest

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

// Eight values as a 16-byte piece of their next plane, which is taken off them: cut off
// (the first) or rounded.
template <bool kCut>
__device__ __forceinline__ uint4 next_plane(float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = kCut ? upper_halves(f[2 * i], f[2 * i + 1]) : pack_bf16x2(f[2 * i], f[2 * i + 1]);
    f[2 * i] -= __uint_as_float(w[i] << 16);
    f[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Piece j of lane i (of four) and piece i of lane j change places.
__device__ __forceinline__ void exchange4(uint4 (&v)[4], int lane) {
  auto swap = [&](uint4& low, uint4& high, int bit) {
    const bool up = lane & bit;
    uint4 s = up ? low : high;
    s.x = __shfl_xor_sync(0xffffffffu, s.x, bit);
    s.y = __shfl_xor_sync(0xffffffffu, s.y, bit);
    s.z = __shfl_xor_sync(0xffffffffu, s.z, bit);
    s.w = __shfl_xor_sync(0xffffffffu, s.w, bit);
    (up ? low : high) = s;
  };
  swap(v[0], v[1], 1);
  swap(v[2], v[3], 1);
  swap(v[0], v[2], 2);
  swap(v[1], v[3], 2);
}

// A store of some lanes without a branch: behind one, the lanes of a warp that has rows
// past the end went on in two groups (33 x 512 x 1360, hidden gradients 89 us, 64 rows 33).
__device__ __forceinline__ void store_if(bool on, void* p, const uint4& v) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(p),
      "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"((uint32_t)on)
      : "memory");
}

// A warp's 32 rows and 16 columns of a matrix [M][N], a row in each lane's registers.
struct Rows {
  int row, col, M, N, lane;   // row: the first of the lane's four
  __device__ __forceinline__ void load(const float* p, float (&f)[16]) const {
    uint4 v[4];
    const int c = min(col + 4 * (lane & 3), N - 4);   // what lies past the ends is not used
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = *reinterpret_cast<const uint4*>(p + (int64_t)min(row + j, M - 1) * N + c);
    exchange4(v, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[4 * j] = __uint_as_float(v[j].x);
      f[4 * j + 1] = __uint_as_float(v[j].y);
      f[4 * j + 2] = __uint_as_float(v[j].z);
      f[4 * j + 3] = __uint_as_float(v[j].w);
    }
  }
  __device__ __forceinline__ void store(float* p, const float* f) const {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = make_uint4(__float_as_uint(f[4 * j]), __float_as_uint(f[4 * j + 1]),
                        __float_as_uint(f[4 * j + 2]), __float_as_uint(f[4 * j + 3]));
    exchange4(v, lane);
    const int c = col + 4 * (lane & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      store_if(row + j < M && c < N, p + (int64_t)(row + j) * N + c, v[j]);
  }
  // pieces 0, 1 and 2, 3 of the rows into one plane each (the second nullable)
  __device__ __forceinline__ void store_pieces(__nv_bfloat16* p0, __nv_bfloat16* p1,
                                               uint4 (&v)[4]) const {
    exchange4(v, lane);
    __nv_bfloat16* p = lane & 2 ? p1 : p0;
    const int c = col + 8 * (lane & 1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      store_if(p != nullptr && row + j < M && c < N, p + (int64_t)(row + j) * N + c, v[j]);
  }
  // the first two planes, the last one's pieces in lo; f is used up
  __device__ __forceinline__ void store_planes(__nv_bfloat16* p, float* f, uint4* lo) const {
    uint4 v[4] = {next_plane<true>(f), next_plane<true>(f + 8)};
    v[2] = next_plane<false>(f);
    v[3] = next_plane<false>(f + 8);
    store_pieces(p, p + (int64_t)M * N, v);
    lo[0] = next_plane<false>(f);
    lo[1] = next_plane<false>(f + 8);
  }
};

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
            record_timeout(g.status, abort, 51);
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
          const uint32_t large = tmem + s * 2 * kN, small = large + kN;
          auto term = [&](uint32_t acc, int a, int b, bool first) {
            const uint32_t pa = base + a * kSlot, pb = base + b * kSlot + kTileA;
#pragma unroll
            for (int i = 0; i < kGemmK / 16; ++i)
              mma_bf16_pair(acc, sdesc_sw128(pa + i * a_step, a_lbo, 1024),
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
              term(large, 0, 0, starts);
            } else if (plane == 1) {
              term(small, 0, 1, starts);
              term(small, 1, 0, false);
              term(small, 1, 1, false);
            } else {
              term(small, 0, 2, false);
              term(small, 2, 0, false);
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
        record_timeout(g.status, abort, 52);
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
      const bool any = row - lane < p.M;   // of the warp's rows
      float x[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) x[i] = 0.f;
      for (int k = t.k0; k < t.k1; k += kChain, ++n) {
        const int s = n & 1;
        if (!__all_sync(0xffffffffu,
                        mbar_wait_cluster(&bars->acc_full[s], (n >> 1) & 1, lim, abort))) {
          if (lane == 0) record_timeout(g.status, abort, 53);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + s * 2 * kN;
#pragma unroll
        for (int part = kN; part >= 0; part -= kN) {
          float f[32];
          load_acc(acc + part + col0, f);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] += f[i];
          load_acc(acc + part + col1, f);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[32 + i] += f[i];
        }
        tc_fence_before();   // the next products may overwrite the accumulator
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(in_first_cta(&bars->acc_empty[s]));
      }
      if (!ok) break;
      auto& x0 = *reinterpret_cast<float(*)[32]>(x);
      auto& x1 = *reinterpret_cast<float(*)[32]>(x + 32);
      if (t.slot >= 0) {
        if (any) {
          store_partial<kN>(g.partial, t.slot, col0, tile_row, x0);
          store_partial<kN>(g.partial, t.slot, col1, tile_row, x1);
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
        if (any) {
          load_partials<kN>(g.partial, t.slot - t.share, p.shares, col0, tile_row, x0);
          load_partials<kN>(g.partial, t.slot - t.share, p.shares, col1, tile_row, x1);
        }
      }
      if (!any) continue;
      // 16 columns at a time; rolled up, since code that runs once per launch and warp is
      // waited for line by line
      Rows to = {row - (lane & 3), t.n * kN + half * 64, p.M, p.N, lane};
      if (kEpi == GEMM_GLU) to.col = t.n * (kN / 2) + half * 32;
      constexpr int kRounds = kEpi == GEMM_GLU ? 2 : 4;
#pragma unroll 1
      for (int c = 0; c < kRounds; ++c, to.col += 16) {
        if constexpr (kEpi == GEMM_GLU) {
          if (g.gate != nullptr) {
            to.store(g.gate, x);
            to.store(g.up, x + 32);
          }
          with_activation(g.act, [&](auto act) {
            float unused;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              x[i] = activation<false, false>(x[i], act.value, unused) * x[32 + i];
          });
          uint4 lo[4] = {};
          to.store_planes(g.h, x, lo);
          to.store_pieces(g.h + 2 * (int64_t)p.M * p.N, nullptr, lo);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] = x[16 + i];
            x[32 + i] = x[48 + i];
          }
        } else {
          if constexpr (kEpi == GEMM_STORE) {
            to.store(p.out[second], x);
          } else {
            float gate[16], up[16];
            to.load(g.gate, gate);
            to.load(g.up, up);
            with_activation(g.act, [&](auto act) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float da;
                const float a = activation<true, false>(gate[i], act.value, da), dh = x[i];
                x[i] = a * up[i];
                gate[i] = dh * up[i] * da;
                up[i] = dh * a;
              }
            });
            const int64_t last_plane = 2 * (int64_t)p.M * p.N;
            uint4 lo[4];
            to.store_planes(g.dgate, gate, lo);
            to.store_planes(g.dup, up, lo + 2);
            to.store_pieces(g.dgate + last_plane, g.dup + last_plane, lo);
            to.store_planes(g.h, x, lo);
            to.store_pieces(g.h + last_plane, nullptr, lo);
          }
#pragma unroll
          for (int i = 0; i < 48; ++i) x[i] = x[16 + i];
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
    __nv_bfloat16* to = m.planes + i * 8;
    *reinterpret_cast<uint4*>(to) = next_plane<true>(f);
    *reinterpret_cast<uint4*>(to + n * 8) = next_plane<false>(f);
    *reinterpret_cast<uint4*>(to + 2 * n * 8) = next_plane<false>(f);
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
