// The gated feed-forward block for 9 to 64 rows (decoding a batch of requests).
//
// Bound by the weights, which are read once: 6 D F bytes in bf16.  They are the M side
// of the MMAs, 128 rows of a weight (of both projections, so that gate and up of a
// hidden unit meet in one thread), and the tokens the N side: the tensor pipe runs no
// rows that are not there, and a stage is nearly all weights.  The large products' tiles
// take 76 us for 37 tokens, 4096 x 12288, in five launches; here are two, the second's
// first weights in flight while the first ends.
//
// Two CTAs share an SM, and the CTAs of a cluster share k where there are fewer tiles
// than that; their sums meet in shared memory in a fixed order, each CTA finishing some
// of the tokens.
//
// Warp roles (192 threads): warp 0 TMA producer, warp 1 TMEM allocation and MMAs (one
// lane each), warps 2..5 epilogue: thread = weight row = TMEM lane, columns = tokens.
#include <cuda_bf16.h>

#include "check.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

constexpr int kThreads = 192;
constexpr int kRows = 128;                       // of a weight in one tile
constexpr int kWeightTile = kRows * kGemmK * 2;  // bytes
constexpr int kMaxTokens = kBatchRows;
constexpr long long kLandLimit = 1LL << 16;   // milliseconds: a load lands within microseconds
constexpr long long kDrainLimit = 1LL << 24;
constexpr int kResident = 2;                     // CTAs an SM holds

template <bool kGlu>
struct Layout {
  static constexpr int kMats = kGlu ? 2 : 1;
  static constexpr int kStages = kGlu ? 2 : 4;
  static constexpr int kStage = kMats * kWeightTile + kMaxTokens * kGemmK * 2;
  static constexpr int kBars = kStages * kStage;
  static constexpr int kSmem = kBars + 256 + 1024;   // slack for alignment
  // the sums take the stages' place in the end
  static_assert(kMats * kMaxTokens * kRows * 4 <= kBars, "shared memory budget");
  static_assert(kResident * (kSmem + 1024) <= 228 * 1024, "shared memory budget");
};

struct Bars {
  uint64_t full[4], empty[4];
  uint64_t acc_full;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void record_timeout(int32_t* status, volatile int* abort, int site) {
  if (atomicCAS(&status[0], 0, 1) == 0) status[1] = site;
  *abort = 1;
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
    ffn_tokens_kernel(const __grid_constant__ FfnTokensArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  using L = Layout<kGlu>;
  constexpr int kStages = L::kStages, kMats = L::kMats;
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shares = (int)gridDim.y, share = (int)blockIdx.y;
  const int n0 = blockIdx.x * kRows;
  const int k_tiles = (a.K + kGemmK - 1) / kGemmK;
  const int k0 = (int)((int64_t)k_tiles * share / shares);
  const int k1 = (int)((int64_t)k_tiles * (share + 1) / shares);
  volatile int* abort = &bars->abort;
  const long long lim = a.wait_limit;
  constexpr uint32_t kCols = kMats * kMaxTokens;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->acc_full, 1);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  if (kGlu) griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      auto load_weights = [&](int k) {
        const int st = (k - k0) % kStages;
        uint8_t* dst = smem + st * L::kStage;
        mbar_expect_tx(&bars->full[st], kMats * kWeightTile + a.tokens * kGemmK * 2);
        if (!CP_IN_RANGE(n0, 0, a.N, a.status, 303)) return;
        for (int m = 0; m < kMats; ++m)
          tma_load_2d(&a.w[m], &bars->full[st], dst + m * kWeightTile, k * kGemmK, n0);
      };
      auto load_tokens = [&](int k) {
        const int st = (k - k0) % kStages;
        tma_load_2d(&a.x, &bars->full[st], smem + st * L::kStage + kMats * kWeightTile, k * kGemmK,
                    0);
      };
      const int early = min(kStages, k1 - k0);
      for (int k = k0; k < k0 + early; ++k) load_weights(k);
      if (!kGlu) griddep_wait();   // the tokens' rows come from the launch before
      for (int k = k0; k < k0 + early; ++k) load_tokens(k);
      int k = k0 + early;
      for (; k < k1 && !*abort; ++k) {
        const int j = k - k0, st = j % kStages;
        if (!mbar_wait(&bars->empty[st], ((j / kStages) - 1) & 1, lim, abort)) {
          record_timeout(a.status, abort, 41);
          break;
        }
        load_weights(k);
        load_tokens(k);
      }
      // every load has landed before the CTA goes on
      int zero = 0;
      for (int x = k - kStages; x < k; ++x)
        if (x >= k0)
          mbar_wait(&bars->full[(x - k0) % kStages], ((x - k0) / kStages) & 1, kLandLimit, &zero);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(kRows, a.tokens, 0, 0);
      bool ok = true;
      for (int k = k0; k < k1; ++k) {
        const int j = k - k0, st = j % kStages;
        if (!mbar_wait(&bars->full[st], (j / kStages) & 1, lim, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t pw = smem_u32(smem + st * L::kStage), px = pw + kMats * kWeightTile;
#pragma unroll
        for (int i = 0; i < kGemmK / 16; ++i)
#pragma unroll
          for (int m = 0; m < kMats; ++m)
            mma_bf16(tmem + m * kMaxTokens, sdesc_sw128(pw + m * kWeightTile + i * 32, 16, 1024),
                     sdesc_sw128(px + i * 32, 16, 1024), idesc, (k > k0 || i > 0) ? 1u : 0u);
        mma_commit(&bars->empty[st]);
      }
      if (ok) {
        mma_commit(&bars->acc_full);
      } else {
        record_timeout(a.status, abort, 42);
        // nothing issued by this thread may still be running at exit
        mma_commit(&bars->drain);
        int zero = 0;
        mbar_wait(&bars->drain, 0, kDrainLimit, &zero);
      }
    }
  }
  // ------------------------------------------------------------ epilogue
  float* red = reinterpret_cast<float*>(smem);   // [matrix][token][row]
  const int quarter = warp & 3, row = quarter * 32 + lane;
  const bool epilogue = warp >= 2;
  bool ok = true;
  auto finish = [&](int token, float v0, float v1) {
    const int n = n0 + row;
    if (n >= a.N) return;
    const int64_t at = (int64_t)token * a.N + n;
    if constexpr (kGlu) {
      float unused;
      static_cast<__nv_bfloat16*>(a.out)[at] =
          __float2bfloat16_rn(activation<false, true>(v0, a.act, unused) * v1);
      if (a.gate != nullptr) {
        const int64_t low = kept_low(a.T, a.N) + token * kept_pitch(a.N) + n;
        const uint32_t g = __float_as_uint(v0), u = __float_as_uint(v1);
        static_cast<uint16_t*>(a.gate)[at] = (uint16_t)(g >> 16);
        static_cast<uint16_t*>(a.up)[at] = (uint16_t)(u >> 16);
        static_cast<uint8_t*>(a.gate)[low] = (uint8_t)(g >> 8);
        static_cast<uint8_t*>(a.up)[low] = (uint8_t)(u >> 8);
      }
    } else {
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v0);
    }
  };
  if (epilogue) {
    if (!kGlu) griddep_wait();   // nothing is written before the launch before is done
    ok = __all_sync(0xffffffffu, mbar_wait(&bars->acc_full, 0, lim, abort));
    if (!ok && lane == 0) record_timeout(a.status, abort, 43);
    tc_fence_after();
    if (ok) {
      const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < a.T; c += 32) {
        uint32_t v[2][32];
#pragma unroll
        for (int m = 0; m < kMats; ++m) tmem_ld32(acc + m * kMaxTokens + c, v[m]);
        tmem_ld_wait();
#pragma unroll
        for (int m = 0; m < kMats; ++m) reg_fence32(v[m]);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (c + i >= a.T) continue;
          if (shares == 1) {
            finish(c + i, __uint_as_float(v[0][i]), __uint_as_float(v[kMats - 1][i]));
          } else {
#pragma unroll
            for (int m = 0; m < kMats; ++m)
              red[(m * kMaxTokens + c + i) * kRows + row] = __uint_as_float(v[m][i]);
          }
        }
        __syncwarp();   // the next load of the accumulator is the whole warp's
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (shares > 1) {
    cluster_sync();
    if (epilogue && ok) {   // the CTAs take tokens in turn
      for (int token = share; token < a.T; token += shares) {
        float p[8][kMats], v[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 8; ++c)   // all on their way before the first is added
#pragma unroll
          for (int m = 0; m < kMats; ++m)
            p[c][m] = c < shares ? peer_load(&red[(m * kMaxTokens + token) * kRows + row], c) : 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
          for (int m = 0; m < kMats; ++m) v[m] += p[c][m];
        finish(token, v[0], v[1]);
      }
    }
    __syncwarp();
    cluster_sync();   // the others have read this CTA's sums
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

template <bool kGlu>
cudaError_t launch(const FfnTokensArgs& a, int sms, cudaStream_t st) {
  using L = Layout<kGlu>;
  auto kernel = ffn_tokens_kernel<kGlu>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       L::kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.N + kRows - 1) / kRows, k_tiles = (a.K + kGemmK - 1) / kGemmK;
  // as many shares of k as run at once, of two k tiles or more
  int shares = kResident * sms / tiles;
  if (shares > k_tiles / 2) shares = k_tiles / 2;
  if (shares > 8) shares = 8;
  if (shares < 1) shares = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)shares);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
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
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_ffn_tokens(const FfnTokensArgs& a, bool glu, int sms, cudaStream_t st) {
  if (a.T < 1 || a.T > a.tokens || a.tokens > kBatchRows || a.tokens % 16 != 0)
    return cudaErrorInvalidValue;
  return glu ? launch<true>(a, sms, st) : launch<false>(a, sms, st);
}

}  // namespace cpattn
