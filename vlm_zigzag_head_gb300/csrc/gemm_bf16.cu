// Matrix products of the gated feed-forward block on the 5th-generation tensor
// cores (sm_103a), with its activation in their epilogues.
//
//   C[m][n] = sum_k A(m, k) B(n, k),  bf16 operands, fp32 sums in tensor memory
//
// A pair of CTAs shares a tile of 256 x 256 (gate and up: 256 x 128 of each, so that
// both halves of a pair of columns meet in one epilogue), k goes by 64: each CTA
// loads 128 rows of A and of B, and the pair's MMAs read both.  Operands come by TMA
// in the 128-byte swizzle, K-major or MN-major as they lie in memory: no product needs
// a transposed copy.  The kernel is persistent: pairs walk (tile, share of k) units,
// and two accumulators in tensor memory let a tile's epilogue run under the next one's
// products.
//
// Warp roles (384 threads):
//   warp 0       TMA producer (one lane): this CTA's rows of A and B
//   warp 1       TMEM allocation; in the first CTA lane 0 issues every MMA
//   warps 4..11  epilogue: TMEM lane quarter w % 4; the two warps of a quarter have
//                halves of each 64 columns
//
// The epilogue moves boxes of 32 rows x 64 columns through shared memory by TMA, two
// warps to a box: a thread holds one row, and rows read and written straight from it
// (16 bytes in each of 32 lines) took longer than the products.
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
constexpr int kEpiWarps = 8;
constexpr int kRows = kGemmM / 2;                   // of A and B in one CTA
constexpr int kTile = kRows * kGemmK * 2;           // bytes of one operand's part of a stage
constexpr int kBf16Box = 32 * 64 * 2, kByteBox = 32 * 64;
constexpr uint32_t kTmemCols = 512;
constexpr long long kDrainLimit = 1LL << 24;
constexpr long long kLandLimit = 1LL << 16;   // milliseconds: a load lands within microseconds
// Stages, and the boxes of two warps: two of bf16 (or two halves of fp32); h, gate, up
// and the low bytes; gate, up, low bytes in, dgate, dup, h out.
template <int kEpi>
struct Layout {
  static constexpr int kStages = kEpi == GEMM_STORE ? 6 : kEpi == GEMM_GLU ? 5 : 4;
  static constexpr int kPairBytes = kEpi == GEMM_STORE  ? 2 * kBf16Box
                                    : kEpi == GEMM_GLU ? 3 * kBf16Box + 2 * kByteBox
                                                       : 5 * kBf16Box + 2 * kByteBox;
  static constexpr int kBoxes = kStages * 2 * kTile;
  static constexpr int kBars = kBoxes + kEpiWarps / 2 * kPairBytes;
  static constexpr int kSmem = kBars + 256 + 1024;   // slack for alignment
};
static_assert(Layout<GEMM_STORE>::kSmem <= 227 * 1024, "shared memory budget");
static_assert(Layout<GEMM_GLU>::kSmem <= 227 * 1024, "shared memory budget");
static_assert(Layout<GEMM_DGLU>::kSmem <= 227 * 1024, "shared memory budget");

struct Bars {
  uint64_t full[6];        // first CTA: both CTAs' loads of a stage have landed
  uint64_t empty[6];       // both: the stage's MMAs are done
  uint64_t acc_full[2];    // both: a tile's products are done
  uint64_t acc_empty[2];   // first CTA: both CTAs' epilogues have read them
  uint64_t box[4];         // GEMM_DGLU: a quarter's boxes have landed
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// m tiles whose n tiles are walked together: about square patches of tiles run at a
// time, which reads the least of A and B.
constexpr int kGroupM = 8;

struct TilePlace {
  int m, n;
};
__device__ __forceinline__ TilePlace tile_place(const GemmArgs& g, int tile) {
  const unsigned per_group = kGroupM * g.n_tiles;
  const unsigned group = (unsigned)tile / per_group, in = (unsigned)tile % per_group;
  const unsigned first = group * kGroupM;
  const unsigned rows = min(kGroupM, g.m_tiles - (int)first);
  return {(int)(first + in % rows), (int)(in / rows)};
}

// Unit u: a tile, and which of its k tiles.  The issuing thread asks for the k tiles
// alone: between two tiles the tensor core waits for it.
struct Work {
  int tile, slot, k0, k1;   // slot: of the partial sums, -1 for a whole tile
};
__device__ __forceinline__ Work work_at(const GemmArgs& g, int u) {
  if (u < g.whole) return {u, -1, 0, g.k_tiles};
  const unsigned v = u - g.whole, tail = v / g.shares, share = v % g.shares;
  return {(int)(g.whole + tail), (int)v, (int)(g.k_tiles * share / g.shares),
          (int)(g.k_tiles * (share + 1) / g.shares)};
}
struct Unit {
  int tile, m, n, slot, k0, k1;
};
__device__ __forceinline__ Unit unit_at(const GemmArgs& g, int u) {
  const Work w = work_at(g, u);
  const TilePlace t = tile_place(g, w.tile);
  return {w.tile, t.m, t.n, w.slot, w.k0, w.k1};
}

__device__ __forceinline__ void record_timeout(int32_t* status, volatile int* abort, int site) {
  if (atomicCAS(&status[0], 0, 1) == 0) status[1] = site;
  *abort = 1;
}

// 32 columns (pieces 8 c .. 8 c + 7) of tile row `row` into a shared tile's sums.
__device__ __forceinline__ void store_partial(const GemmArgs& g, int slot, int col, int row,
                                              const float (&f)[32]) {
  float4* p = reinterpret_cast<float4*>(g.partial) +
              ((int64_t)slot * (kGemmN / 4) + col / 4) * kGemmM + row;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    p[i * kGemmM] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}

// The same columns of all shares of a tile, added in order.
__device__ __forceinline__ void load_partials(const GemmArgs& g, int tile, int col, int row,
                                              float (&f)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = 0.f;
#pragma unroll 2
  for (int s = 0; s < g.shares; ++s) {
    const float4* p = reinterpret_cast<const float4*>(g.partial) +
                      ((int64_t)((tile - g.whole) * g.shares + s) * (kGemmN / 4) + col / 4) * kGemmM +
                      row;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = __ldcg(p + i * kGemmM);   // written by other CTAs of this launch
      f[4 * i] += v.x;
      f[4 * i + 1] += v.y;
      f[4 * i + 2] += v.z;
      f[4 * i + 3] += v.w;
    }
  }
}

__device__ __forceinline__ void load_acc(uint32_t taddr, float (&f)[32]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_ld_wait();
  reg_fence32(r);
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
}

// 16-byte piece p of a lane's row in a box of 64- or 128-byte rows, as TMA's swizzle
// of that size places it; the eight lanes of a pass meet no bank twice.
template <int kRowBytes>
__device__ __forceinline__ uint4* piece(uint8_t* box, int lane, int p) {
  constexpr int kSwap = kRowBytes / 16 - 1;
  return reinterpret_cast<uint4*>(box + lane * kRowBytes +
                                  ((p ^ (lane * kRowBytes / 128 & kSwap)) << 4));
}

// A lane's 32 columns, the first or second half of a box's (fp32: a box of their own).
__device__ __forceinline__ void put_bf16(uint8_t* box, int lane, int half, const float (&f)[32]) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
    *piece<128>(box, lane, half * 4 + p) =
        make_uint4(pack_bf16x2(f[8 * p], f[8 * p + 1]), pack_bf16x2(f[8 * p + 2], f[8 * p + 3]),
                   pack_bf16x2(f[8 * p + 4], f[8 * p + 5]), pack_bf16x2(f[8 * p + 6], f[8 * p + 7]));
}
__device__ __forceinline__ void put_f32(uint8_t* box, int lane, const float (&f)[32]) {
#pragma unroll
  for (int p = 0; p < 8; ++p)
    *piece<128>(box, lane, p) =
        make_uint4(__float_as_uint(f[4 * p]), __float_as_uint(f[4 * p + 1]),
                   __float_as_uint(f[4 * p + 2]), __float_as_uint(f[4 * p + 3]));
}
__device__ __forceinline__ void put_kept(uint8_t* hi, uint8_t* lo, int lane, int half,
                                         const float (&f)[32]) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t h[8], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* v = f + 16 * p + 4 * i;
      h[2 * i] = upper_halves(v[0], v[1]);
      h[2 * i + 1] = upper_halves(v[2], v[3]);
      l[i] = next_bytes(v[0], v[1], v[2], v[3]);
    }
    *piece<128>(hi, lane, half * 4 + 2 * p) = make_uint4(h[0], h[1], h[2], h[3]);
    *piece<128>(hi, lane, half * 4 + 2 * p + 1) = make_uint4(h[4], h[5], h[6], h[7]);
    *piece<64>(lo, lane, half * 2 + p) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

template <bool kAMN, bool kBMN, int kEpi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ GemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  using L = Layout<kEpi>;
  constexpr int kStages = L::kStages;
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int units = g.whole + (g.m_tiles * g.n_tiles - g.whole) * g.shares;
  griddep_launch_dependents();   // the next product waits for this one where it must
  volatile int* abort = &bars->abort;
  const long long lim = g.wait_limit;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->acc_full[s], 1);
      mbar_init(&bars->acc_empty[s], 2 * kEpiWarps);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&bars->box[q], 1);
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

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      auto load_a = [&](const Unit& t, int k, int st) {
        const bool second = t.m >= g.m_split;
        const int src = k >= g.k_split, kk = (k - (src ? g.k_split : 0)) * kGemmK;
        const int m0 = (t.m - (second ? g.m_split : 0)) * kGemmM + rank * kRows;
        const CUtensorMap* map = &g.a[second || src];
        uint8_t* dst = smem + st * 2 * kTile;
        const uint32_t full = in_first_cta(&bars->full[st]);
        if (!CP_IN_RANGE(m0, 0, g.M + kRows, g.status, 301)) return;
        if constexpr (kAMN) {
          for (int i = 0; i < kRows / 64; ++i)
            tma_load_2d_pair(map, full, dst + i * 64 * kGemmK * 2, m0 + i * 64, kk);
        } else {
          tma_load_2d_pair(map, full, dst, kk, m0);
        }
      };
      auto load_b = [&](const Unit& t, int k, int st) {
        const int src = k >= g.k_split, kk = (k - (src ? g.k_split : 0)) * kGemmK;
        const int n0 = kEpi == GEMM_GLU ? t.n * kRows : t.n * kGemmN + rank * kRows;
        const CUtensorMap* map = &g.b[kEpi == GEMM_GLU ? rank : src];   // gate or up
        uint8_t* dst = smem + st * 2 * kTile + kTile;
        const uint32_t full = in_first_cta(&bars->full[st]);
        if (!CP_IN_RANGE(n0, 0, g.N + kRows, g.status, 302)) return;
        if constexpr (kBMN) {
          for (int i = 0; i < kRows / 64; ++i)
            tma_load_2d_pair(map, full, dst + i * 64 * kGemmK * 2, n0 + i * 64, kk);
        } else {
          tma_load_2d_pair(map, full, dst, kk, n0);
        }
      };
      auto expect = [&](int st) {   // both CTAs' parts
        if (rank == 0) mbar_expect_tx(&bars->full[st], 4 * kTile);
      };
      // the first stages' weights need not wait for the launch before
      int early = 0;
      if (g.follows == FOLLOWS_A) {
        const Unit t = unit_at(g, pair);
        early = min(kStages, t.k1 - t.k0);
        for (int i = 0; i < early; ++i) {
          expect(i);
          load_b(t, t.k0 + i, i);
        }
        griddep_wait();
        for (int i = 0; i < early; ++i) load_a(t, t.k0 + i, i);
      } else if (g.follows == FOLLOWS_BOTH) {
        griddep_wait();
      }
      int j = early;   // k tiles so far, across units
      for (int u = pair; u < units && !*abort; u += pairs) {
        const Unit t = unit_at(g, u);
        for (int k = t.k0 + (u == pair ? early : 0); k < t.k1; ++k, ++j) {
          const int st = j % kStages;
          if (j >= kStages &&
              !mbar_wait_cluster(&bars->empty[st], ((j / kStages) - 1) & 1, lim, abort)) {
            record_timeout(g.status, abort, 31);
            break;
          }
          expect(st);
          load_a(t, k, st);
          load_b(t, k, st);
        }
      }
      // no load may be on its way when the CTA exits (none is once its tiles' epilogues
      // are done; after a wait gave up, nobody may be reading the stages any more)
      int zero = 0;
      for (int x = j - kStages; x < j; ++x)
        if (x >= 0)
          mbar_wait_cluster(&bars->empty[x % kStages], (x / kStages) & 1, kLandLimit, &zero);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16(kGemmM, kGemmN, kAMN, kBMN);
      bool ok = true;
      int j = 0, n = 0;   // k tiles and units so far
      Work t = work_at(g, pair), next = t;
      // its waits are bounded, and the launch before may take longer than the bound
      if (g.follows != FOLLOWS_NONE) griddep_wait();
      for (int u = pair; ok && u < units; u += pairs, ++n, t = next) {
        if (u + pairs < units) next = work_at(g, u + pairs);
        const int s = n & 1;
        if (n >= 2 && !mbar_wait_cluster(&bars->acc_empty[s], ((n >> 1) - 1) & 1, lim, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int k = t.k0; k < t.k1; ++k, ++j) {
          const int st = j % kStages;
          if (!mbar_wait_cluster(&bars->full[st], (j / kStages) & 1, lim, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t pa = smem_u32(smem + st * 2 * kTile), pb = pa + kTile;
#pragma unroll
          for (int i = 0; i < kGemmK / 16; ++i) {
            // 16 k further: 32 bytes along a K-major row, 16 rows of an MN-major box
            const uint64_t da = kAMN ? sdesc_sw128(pa + i * 2048, 64 * kGemmK * 2, 1024)
                                     : sdesc_sw128(pa + i * 32, 16, 1024);
            const uint64_t db = kBMN ? sdesc_sw128(pb + i * 2048, 64 * kGemmK * 2, 1024)
                                     : sdesc_sw128(pb + i * 32, 16, 1024);
            mma_bf16_pair(tmem + s * kGemmN, da, db, idesc, (k > t.k0 || i > 0) ? 1u : 0u);
          }
          mma_commit_pair(&bars->empty[st]);
        }
        if (!ok) break;
        mma_commit_pair(&bars->acc_full[s]);
      }
      if (!ok) {
        record_timeout(g.status, abort, 32);
        // nothing issued by this thread may still be running at exit
        mma_commit_pair(&bars->drain);
        int zero = 0;
        mbar_wait_cluster(&bars->drain, 0, kDrainLimit, &zero);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const bool issues = half == 0 && lane == 0;   // of the two warps' boxes
    const int pair_bar = 1 + quarter;
    auto pair_sync = [&] { named_sync(pair_bar, 64); };
    uint8_t* boxes = smem + L::kBoxes + quarter * L::kPairBytes;
    constexpr int kTileN = kEpi == GEMM_GLU ? kGemmN / 2 : kGemmN;
    constexpr int kChunks = kTileN / 64;
    auto first_row = [&](const Unit& t) {
      return (t.m - (t.m >= g.m_split ? g.m_split : 0)) * kGemmM + rank * kRows + quarter * 32;
    };
    // GEMM_DGLU: the kept gate and up of a chunk, on their way while the one before
    // is worked on
    [[maybe_unused]] auto fetch = [&](const Unit& t, int c) {
      if (!issues) return;
      const int row = first_row(t), col = t.n * kTileN + c * 64;
      uint64_t* bar = &bars->box[quarter];
      mbar_expect_tx(bar, 2 * (kBf16Box + kByteBox));
      tma_load_2d(&g.gate[0], bar, boxes, col, row);
      tma_load_2d(&g.up[0], bar, boxes + kBf16Box, col, row);
      tma_load_2d(&g.gate[1], bar, boxes + 2 * kBf16Box, col, row);
      tma_load_2d(&g.up[1], bar, boxes + 2 * kBf16Box + kByteBox, col, row);
    };
    int n = 0, fetched = 0, got = 0;
    auto fetch_first = [&](int u) {   // the first chunk of unit u, where it is a whole tile
      if constexpr (kEpi == GEMM_DGLU) {
        if (u >= g.whole) return;
        fetch(unit_at(g, u), 0);
        ++fetched;
      }
    };
    if (g.follows != FOLLOWS_NONE) griddep_wait();
    fetch_first(pair);
    bool ok = true;
    for (int u = pair; ok && u < units; u += pairs, ++n) {
      const Unit t = unit_at(g, u);
      const int s = n & 1;
      // both warps of a box go on, or neither
      if (!named_all(pair_bar, 64,
                     mbar_wait_cluster(&bars->acc_full[s], (n >> 1) & 1, lim, abort))) {
        if (lane == 0) record_timeout(g.status, abort, 33);
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + s * kGemmN;
      const int second = t.m >= g.m_split;
      const int row0 = first_row(t), tile_row = rank * kRows + quarter * 32 + lane;
      auto release = [&] {   // the next products may overwrite the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(in_first_cta(&bars->acc_empty[s]));
      };
      const bool shared = t.slot >= 0;
      if (shared) {
        const bool in = row0 + lane < g.M;
#pragma unroll 1
        for (int c = 0; c < kGemmN / 64; ++c) {
          const int col = c * 64 + half * 32;
          float x[32];
          load_acc(acc + col, x);
          if (in) store_partial(g, t.slot, col, tile_row, x);
          __syncwarp();   // the next load of the accumulator is the whole warp's
        }
        release();
        // these two warps' rows of all shares: the last to get here goes on with them
        __threadfence();
        pair_sync();
        bool last = true;
        if (issues) {
          int32_t* ticket = g.tickets + (t.tile - g.whole) * 8 + rank * 4 + quarter;
          last = atomicAdd(ticket, 1) == g.shares - 1;
          if (last) *ticket = 0;
          __threadfence();
        }
        if (!named_all(pair_bar, 64, last)) continue;
      }
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        const int col = c * 64 + half * 32, box_col = t.n * kTileN + c * 64;
        const bool stores = row0 < g.M && box_col < g.N;   // the box is not wholly past the end
        float x[32];
        auto take = [&](int at, float (&f)[32]) {
          if (!shared) {
            load_acc(acc + at, f);
          } else if (row0 + lane < g.M) {
            load_partials(g, t.tile, at, tile_row, f);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = 0.f;
          }
        };
        take(col, x);
        if constexpr (kEpi == GEMM_GLU) {
          float v[32];
          take(kTileN + col, v);
          if (issues) bulk_wait_read<0>();   // the boxes' last stores have read them
          pair_sync();
          if (g.keep) {
            put_kept(boxes + kBf16Box, boxes + 3 * kBf16Box, lane, half, x);
            put_kept(boxes + 2 * kBf16Box, boxes + 3 * kBf16Box + kByteBox, lane, half, v);
          }
          float unused;
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = activation<false, true>(x[i], g.act, unused) * v[i];
          put_bf16(boxes, lane, half, x);
          fence_proxy_async_smem();
          pair_sync();
          if (issues && stores) {
            tma_store_2d(&g.out[0], boxes, box_col, row0);
            if (g.keep) {
              tma_store_2d(&g.gate[0], boxes + kBf16Box, box_col, row0);
              tma_store_2d(&g.up[0], boxes + 2 * kBf16Box, box_col, row0);
              tma_store_2d(&g.gate[1], boxes + 3 * kBf16Box, box_col, row0);
              tma_store_2d(&g.up[1], boxes + 3 * kBf16Box + kByteBox, box_col, row0);
            }
            bulk_commit();
          }
        } else if constexpr (kEpi == GEMM_STORE) {
          uint8_t* box = boxes + (g.out_f32 ? half : c & 1) * kBf16Box;
          if (issues) {
            if (g.out_f32) bulk_wait_read<0>();
            else bulk_wait_read<1>();
          }
          pair_sync();
          if (g.out_f32) put_f32(box, lane, x);
          else put_bf16(box, lane, half, x);
          fence_proxy_async_smem();
          pair_sync();
          if (issues) {
            if (stores) tma_store_2d(&g.out[second], box, box_col, row0);
            if (stores && g.out_f32 && box_col + 32 < g.N)
              tma_store_2d(&g.out[second], box + kBf16Box, box_col + 32, row0);
            bulk_commit();   // one group a chunk, so that the count holds
          }
        } else {
          if (fetched == got) {   // a shared tile's, or the first after one
            fetch(t, c);
            ++fetched;
          }
          if (!named_all(pair_bar, 64, mbar_wait(&bars->box[quarter], got & 1, lim, abort))) {
            if (lane == 0) record_timeout(g.status, abort, 34);
            ok = false;
            break;
          }
          ++got;
          uint4 kg[4], ku[4], lg[2], lu[2];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            kg[p] = *piece<128>(boxes, lane, half * 4 + p);
            ku[p] = *piece<128>(boxes + kBf16Box, lane, half * 4 + p);
          }
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            lg[p] = *piece<64>(boxes + 2 * kBf16Box, lane, half * 2 + p);
            lu[p] = *piece<64>(boxes + 2 * kBf16Box + kByteBox, lane, half * 2 + p);
          }
          if (issues) bulk_wait_read<0>();   // the last stores have read their boxes
          pair_sync();   // all have read: the next chunk may land
          if (c + 1 < kChunks) {
            fetch(t, c + 1);
            ++fetched;
          } else {
            fetch_first(u + pairs);
          }
          uint8_t* out = boxes + 2 * (kBf16Box + kByteBox);
          const uint32_t* wg = reinterpret_cast<const uint32_t*>(kg);
          const uint32_t* wu = reinterpret_cast<const uint32_t*>(ku);
          const uint32_t* bg = reinterpret_cast<const uint32_t*>(lg);
          const uint32_t* bu = reinterpret_cast<const uint32_t*>(lu);
#pragma unroll
          for (int p = 0; p < 4; ++p) {   // eight columns at a time
            float gate[8], up[8], h[8];
            rejoin8(wg + 4 * p, bg + 2 * p, gate);
            rejoin8(wu + 4 * p, bu + 2 * p, up);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float da;
              const float a = activation<true, true>(gate[e], g.act, da), dh = x[8 * p + e];
              h[e] = a * up[e];
              gate[e] = dh * up[e] * da;
              up[e] = dh * a;
            }
            auto put = [&](int which, const float (&f)[8]) {
              *piece<128>(out + which * kBf16Box, lane, half * 4 + p) =
                  make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                             pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
            };
            put(0, gate);
            put(1, up);
            put(2, h);
          }
          fence_proxy_async_smem();
          pair_sync();
          if (issues && stores) {
            tma_store_2d(&g.dgate, out, box_col, row0);
            tma_store_2d(&g.dup, out + kBf16Box, box_col, row0);
            tma_store_2d(&g.out[0], out + 2 * kBf16Box, box_col, row0);
            bulk_commit();
          }
        }
      }
      if (!ok) break;
      if (!shared) release();
    }
    if (issues) {
      int zero = 0;   // a load that nobody waited for (after a wait gave up)
      for (; got < fetched; ++got) mbar_wait(&bars->box[quarter], got & 1, kDrainLimit, &zero);
      bulk_wait_all();
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

template <bool kAMN, bool kBMN, int kEpi>
cudaError_t launch_t(const GemmArgs& g, int sms, cudaStream_t st) {
  auto kernel = gemm_kernel<kAMN, kBMN, kEpi>;
  constexpr int smem = Layout<kEpi>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t units = g.whole + ((int64_t)g.m_tiles * g.n_tiles - g.whole) * g.shares;
  if (units < 1 || units > 0x3fffffff) return cudaErrorInvalidConfiguration;
  const int64_t pairs = units < sms / 2 ? units : sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.follows != FOLLOWS_NONE ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, g);
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
