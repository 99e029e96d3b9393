// The gated feed-forward block for 9 to 128 rows (decoding a batch of requests).
//
// Bound by the weights, which are read once: 6 D F bytes in bf16.  They are the M side
// of the MMAs, 128 rows of a weight (of both projections, so that gate and up of a
// hidden unit meet in one thread), and the tokens the N side: the tensor pipe runs no
// rows that are not there, and a stage is nearly all weights.  The large products' tiles
// take 76 us for 37 tokens, 4096 x 12288, in five launches; here are two, the second's
// first weights in flight while the first ends.
//
// Two CTAs share an SM (up to 64 tokens), and the CTAs of a cluster share k where there
// are fewer tiles than that; their sums meet in shared memory in a fixed order, each CTA
// finishing some of the tokens.
//
// Warp roles (320 threads): warp 0 TMA producer, warp 1 TMEM allocation and MMAs (one
// lane each), warps 2..5 sums to shared memory: thread = weight row = TMEM lane, columns =
// tokens; then all, a warp a token (by four warps alone, whose loads from the other CTAs
// take about a microsecond a token, 128 tokens of 4096 x 12288 took 66 us, 62.5 so).
#include <cuda_bf16.h>

#include <atomic>

#include "check.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

constexpr int kWarps = 10, kThreads = kWarps * 32;
constexpr int kRows = 128;                       // of a weight in one tile
constexpr int kWeightTile = kRows * kGemmK * 2;  // bytes

template <bool kGlu, int kTokens>
struct Layout {
  static constexpr int kMats = kGlu ? 2 : 1;
  // CTAs an SM holds, and as many stages as they have
  static constexpr int kResident = kTokens <= 64 ? 2 : 1;
  static constexpr int kStages = kResident == 1 ? (kGlu ? 4 : 6) : !kGlu ? 4 : kTokens <= 32 ? 3 : 2;
  static constexpr int kStage = kMats * kWeightTile + kTokens * kGemmK * 2;
  static constexpr int kBars = kStages * kStage;
  static constexpr int kSmem = kBars + 256 + 1024;   // slack for alignment
  // the sums take the stages' place in the end
  static_assert(kMats * kTokens * kRows * 4 <= kBars, "shared memory budget");
  static_assert(kResident * (kSmem + 1024) <= 228 * 1024, "shared memory budget");
};

struct Bars {
  uint64_t full[6], empty[6];
  uint64_t acc_full;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// 16 bytes of another CTA's shared memory.
__device__ __forceinline__ float4 peer_load4(const float* p, int rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

template <bool kGlu, int kTokens>
__global__ void __launch_bounds__(kThreads, Layout<kGlu, kTokens>::kResident)
    ffn_tokens_kernel(const __grid_constant__ FfnTokensArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  using L = Layout<kGlu, kTokens>;
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
  // a power of two of columns: the second product's begin half way
  constexpr int kMatCols = kTokens <= 32 ? 32 : kTokens <= 64 ? 64 : 128;
  constexpr uint32_t kCols = kMats * kMatCols;

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
        mbar_expect_tx(&bars->full[st], kMats * kWeightTile + kTokens * kGemmK * 2);
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
      constexpr uint32_t idesc = idesc_bf16(kRows, kTokens, 0, 0);
      // its waits are bounded, and the launch before may take longer than the bound
      if (!kGlu) griddep_wait();
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
            mma_bf16(tmem + m * kMatCols, sdesc_sw128(pw + m * kWeightTile + i * 32, 16, 1024),
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
  const int quarter = warp & 3;
  if (warp >= 2 && warp < 6) {
    if (!kGlu) griddep_wait();   // nothing is written before the launch before is done
    const bool ok = __all_sync(0xffffffffu, mbar_wait(&bars->acc_full, 0, lim, abort));
    if (!ok && lane == 0) record_timeout(a.status, abort, 43);
    tc_fence_after();
    if (ok) {
      const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
      for (int c = 0; c < kTokens; c += 32)
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
          uint32_t v[32];
          tmem_ld32(acc + m * kMatCols + c, v);
          tmem_ld_wait();
          reg_fence32(v);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < kTokens)
              red[(m * kTokens + c + i) * kRows + quarter * 32 + lane] = __uint_as_float(v[i]);
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (shares > 1) cluster_sync();
  if (!kGlu) griddep_wait();
  if (!*abort) {
    // a warp has a token, a lane four weight rows; the CTAs of a cluster take turns
    const int row = lane * 4, n = n0 + row;
    for (int token = share + shares * warp; token < a.T; token += shares * kWarps) {
      float4 v[2] = {};
      auto add = [](float4& s, const float4& p) {
        s.x += p.x;
        s.y += p.y;
        s.z += p.z;
        s.w += p.w;
      };
      if (shares == 1) {
#pragma unroll
        for (int m = 0; m < kMats; ++m)
          v[m] = *reinterpret_cast<const float4*>(&red[(m * kTokens + token) * kRows + row]);
      } else {
        float4 p[8][kMats];
#pragma unroll
        for (int c = 0; c < 8; ++c)   // all on their way before the first is added
#pragma unroll
          for (int m = 0; m < kMats; ++m)
            p[c][m] = c < shares ? peer_load4(&red[(m * kTokens + token) * kRows + row], c)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
          for (int m = 0; m < kMats; ++m) add(v[m], p[c][m]);
      }
      if (n >= a.N) continue;   // N is a multiple of 8
      const int64_t at = (int64_t)token * a.N + n;
      float o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
      if constexpr (kGlu) {
        const float u[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
        if (a.gate != nullptr) {
          const int64_t low = kept_low(a.T, a.N) + token * kept_pitch(a.N) + n;
          auto keep = [&](void* p, const float (&f)[4]) {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) =
                make_uint2(upper_halves(f[0], f[1]), upper_halves(f[2], f[3]));
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + low) =
                next_bytes(f[0], f[1], f[2], f[3]);
          };
          keep(a.gate, o);
          keep(a.up, u);
        }
        float unused;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = activation<false, true>(o[i], a.act, unused) * u[i];
      }
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
          make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
  }
  __syncwarp();
  if (shares > 1) cluster_sync();   // the others have read this CTA's sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// How many clusters of `shares` CTAs run at once: a cluster stays within a part of the
// GPU, and fewer fit than there is room for their CTAs.  (Six CTAs for each of 48 tiles on
// 304 places left two clusters for a second round: 20 tokens, 2048 x 6144, 22 us, 20 with
// three; 128 tokens 41 and 26.)  Asked about a kernel that takes the same threads and
// shared memory: of one that allocates tensor memory the answer is one CTA an SM.
__global__ void __launch_bounds__(kThreads) places_kernel(int* p) {
  extern __shared__ int places_smem[];
  if (p != nullptr) *p = places_smem[threadIdx.x];
}
template <bool kGlu, int kTokens>
cudaError_t clusters_at_once(cudaLaunchConfig_t cfg, int shares, int* clusters) {
  static std::atomic<int> known[64][9];   // by device and shares: one more, 0 not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* k = dev < 64 ? &known[dev][shares] : nullptr;
  if (k && k->load() > 0) {
    *clusters = k->load() - 1;
    return cudaSuccess;
  }
  e = cudaFuncSetAttribute(places_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           227 * 1024);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(clusters, places_kernel, &cfg);
  if (e == cudaSuccess && k) k->store(*clusters + 1);
  return e;
}

template <bool kGlu, int kTokens>
cudaError_t launch_t(const FfnTokensArgs& a, int sms, cudaStream_t st) {
  using L = Layout<kGlu, kTokens>;
  auto kernel = ffn_tokens_kernel<kGlu, kTokens>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       L::kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.N + kRows - 1) / kRows, k_tiles = (a.K + kGemmK - 1) / kGemmK;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  auto set_shares = [&](int n) {
    cfg.gridDim = dim3((unsigned)tiles, (unsigned)n);
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = (unsigned)n;
    attr[0].val.clusterDim.z = 1;
  };
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // shares of k, of two k tiles or more, that run at once and leave the busiest SM the least
  int shares = 1, load = (tiles + sms - 1) / sms;   // CTAs of the busiest SM
  for (int n = 2; n <= 8 && n <= k_tiles / 2 && n * tiles <= L::kResident * sms; ++n) {
    const int most = (n * tiles + sms - 1) / sms;
    if (most * shares > load * n) continue;
    set_shares(n);
    cfg.numAttrs = 1;
    int clusters = 0;
    if ((e = clusters_at_once<kGlu, kTokens>(cfg, n, &clusters)) != cudaSuccess) return e;
    if (clusters < tiles) continue;
    shares = n;
    load = most;
  }
  set_shares(shares);
  cfg.numAttrs = kGlu ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool kGlu>
cudaError_t launch(const FfnTokensArgs& a, int sms, cudaStream_t st) {
  switch (a.tokens) {
    case 16: return launch_t<kGlu, 16>(a, sms, st);
    case 32: return launch_t<kGlu, 32>(a, sms, st);
    case 48: return launch_t<kGlu, 48>(a, sms, st);
    case 64: return launch_t<kGlu, 64>(a, sms, st);
    case 96: return launch_t<kGlu, 96>(a, sms, st);
    case 128: return launch_t<kGlu, 128>(a, sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

static_assert(kBatchRows == 128, "the cases above");

cudaError_t launch_ffn_tokens(const FfnTokensArgs& a, bool glu, int sms, cudaStream_t st) {
  if (a.T < 1 || a.T > a.tokens) return cudaErrorInvalidValue;
  return glu ? launch<true>(a, sms, st) : launch<false>(a, sms, st);
}

}  // namespace cpattn
