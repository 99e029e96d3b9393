// Matrix products of the gated feed-forward block on the 5th-generation tensor
// cores (sm_103a), with its activation in their epilogues.
//
//   C[m][n] = sum_k A(m, k) B(n, k),  bf16 operands, fp32 sums in tensor memory
//
// A pair of CTAs shares a tile of 256 x 256 (gate and up: 256 x 128 of each, so that
// both halves of a pair of columns meet in one epilogue), or half as wide where that
// fills the GPU better; k goes by 64: each CTA loads 128 rows of A and half the tile's
// rows of B, and the pair's MMAs read both.  Operands come by TMA in the 128-byte
// swizzle, K-major or MN-major as they lie in memory: no product needs a transposed copy.
// The kernel is persistent: pairs walk (product, tile, share of k) units, and two
// accumulators in tensor memory let a tile's epilogue run under the next one's products.
//
// Warp roles (576 threads):
//   warp 0       TMA producer (one lane): this CTA's rows of A and B
//   warp 1       TMEM allocation; in the first CTA lane 0 issues every MMA
//   warps 2..17  epilogue: TMEM lane quarter w % 4; the four warps of a quarter have
//                16 of each 64 columns each (by eight warps 2048 x 2048 x 6144 forward
//                103 us, so 99)
//
// The epilogue moves boxes of 32 rows x 64 columns through shared memory by TMA, four
// warps to a box: a thread holds one row, and rows read and written straight from it
// (16 bytes in each of 32 lines) took longer than the products.
//
// Rows and columns past the matrices' ends are zeros by TMA's fill and are not
// stored.
#include <cuda_bf16.h>

#include "check.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "gemm_units.cuh"
#include "ptx.cuh"

namespace cpattn {

namespace {

using namespace ptx;

constexpr int kEpiWarps = 16;
constexpr int kThreads = 64 + kEpiWarps * 32;
constexpr int kParts = kEpiWarps / 4;   // warps that share a box
constexpr int kCols = 64 / kParts;      // of a box in one of them
constexpr int kBoxThreads = 32 * kParts;
constexpr int kRows = kGemmM / 2;                   // of A in one CTA
constexpr int kTileA = kRows * kGemmK * 2;          // bytes of a CTA's part of a stage
constexpr int kBf16Box = 32 * 64 * 2, kByteBox = 32 * 64;
// Stages, and the boxes of a quarter's warps: two of bf16 (or two halves of fp32); h, gate, up
// and the low bytes; gate, up, low bytes in, dgate, dup, h out.
template <int kEpi, int kN>
struct Layout {
  static constexpr int kBoxBytes = kEpi == GEMM_STORE  ? 2 * kBf16Box
                                    : kEpi == GEMM_GLU ? 3 * kBf16Box + 2 * kByteBox
                                                       : 5 * kBf16Box + 2 * kByteBox;
  static constexpr int kTileB = kN / 2 * kGemmK * 2;
  static constexpr int kStage = kTileA + kTileB;
  static constexpr int kEpiBytes = 4 * kBoxBytes;
  static constexpr int kStages = (224 * 1024 - kEpiBytes) / kStage;   // 4 to 8
  static constexpr int kBoxes = kStages * kStage;
  static constexpr int kBars = kBoxes + kEpiBytes;
  static constexpr int kSmem = kBars + 256 + 1024;   // slack for alignment
  static_assert(kStages <= 8 && kSmem <= 227 * 1024, "shared memory budget");
};

struct Bars {
  uint64_t full[8];        // first CTA: both CTAs' loads of a stage have landed
  uint64_t empty[8];       // both: the stage's MMAs are done
  uint64_t acc_full[2];    // both: a tile's products are done
  uint64_t acc_empty[2];   // first CTA: both CTAs' epilogues have read them
  uint64_t box[4];         // GEMM_DGLU: a quarter's boxes have landed
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// 16-byte piece p of a lane's row in a box of 64- or 128-byte rows, as TMA's swizzle
// of that size places it; the eight lanes of a pass meet no bank twice.
template <int kRowBytes>
__device__ __forceinline__ uint4* piece(uint8_t* box, int lane, int p) {
  constexpr int kSwap = kRowBytes / 16 - 1;
  return reinterpret_cast<uint4*>(box + lane * kRowBytes +
                                  ((p ^ (lane * kRowBytes / 128 & kSwap)) << 4));
}

// A lane's kCols columns, part `part` of a box's (fp32: of two boxes of 32).
__device__ __forceinline__ void put_bf16(uint8_t* box, int lane, int part,
                                         const float (&f)[kCols]) {
#pragma unroll
  for (int p = 0; p < kCols / 8; ++p)
    *piece<128>(box, lane, part * (kCols / 8) + p) =
        make_uint4(pack_bf16x2(f[8 * p], f[8 * p + 1]), pack_bf16x2(f[8 * p + 2], f[8 * p + 3]),
                   pack_bf16x2(f[8 * p + 4], f[8 * p + 5]), pack_bf16x2(f[8 * p + 6], f[8 * p + 7]));
}
__device__ __forceinline__ void put_f32(uint8_t* boxes, int lane, int part,
                                        const float (&f)[kCols]) {
#pragma unroll
  for (int p = 0; p < kCols / 4; ++p) {
    const int at = part * (kCols / 4) + p;
    *piece<128>(boxes + at / 8 * kBf16Box, lane, at % 8) =
        make_uint4(__float_as_uint(f[4 * p]), __float_as_uint(f[4 * p + 1]),
                   __float_as_uint(f[4 * p + 2]), __float_as_uint(f[4 * p + 3]));
  }
}
__device__ __forceinline__ void put_kept(uint8_t* hi, uint8_t* lo, int lane, int part,
                                         const float (&f)[kCols]) {
#pragma unroll
  for (int p = 0; p < kCols / 16; ++p) {
    uint32_t h[8], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* v = f + 16 * p + 4 * i;
      h[2 * i] = upper_halves(v[0], v[1]);
      h[2 * i + 1] = upper_halves(v[2], v[3]);
      l[i] = next_bytes(v[0], v[1], v[2], v[3]);
    }
    const int at = part * (kCols / 16) + p;
    *piece<128>(hi, lane, 2 * at) = make_uint4(h[0], h[1], h[2], h[3]);
    *piece<128>(hi, lane, 2 * at + 1) = make_uint4(h[4], h[5], h[6], h[7]);
    *piece<64>(lo, lane, at) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

template <int kEpi, int kN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ GemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  using L = Layout<kEpi, kN>;
  constexpr int kStages = L::kStages, kRowsB = kN / 2;
  constexpr uint32_t kTmemCols = 2 * kN;   // two accumulators
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int units = g.units;
  // the units are dealt out to and fro: the longest come first
  auto unit_of = [&](int r) { return r * pairs + (r & 1 ? pairs - 1 - pair : pair); };
  griddep_launch_dependents();   // the next product waits for this one where it must
  volatile int* abort = &bars->abort;
  const long long lim = g.wait_limit;

  if (blockIdx.x == 0)   // long before any wait may give up
    for (int i = threadIdx.x; i < g.clear; i += kThreads) g.status[i] = 0;
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
      // Where a unit's operands come from; this thread's time is near the products'
      // where both operands take two loads a stage, so all that is the same for each
      // stage stays in registers.
      struct Source {
        const CUtensorMap *a, *a_next, *b, *b_next;   // the latter from k_split on
        int m0, n0, k_split;
        bool a_mn, b_mn;
      };
      auto source = [&](const Unit& t) {
        const GemmProblem& p = g.p[t.p];
        const bool second = t.m >= p.m_split;
        Source f;
        f.a = &p.a[second];
        f.a_next = &p.a[1];
        f.b = &p.b[kEpi == GEMM_GLU ? rank : 0];   // gate or up
        f.b_next = &p.b[1];
        f.m0 = (t.m - (second ? p.m_split : 0)) * kGemmM + rank * kRows;
        f.n0 = kEpi == GEMM_GLU ? t.n * kRowsB : t.n * kN + rank * kRowsB;
        f.k_split = p.k_split;
        f.a_mn = p.a_mn;
        f.b_mn = p.b_mn;
        if (!CP_IN_RANGE(f.m0, 0, p.M + kRows, g.status, 301)) f.m0 = 0;
        if (!CP_IN_RANGE(f.n0, 0, p.N + kRows, g.status, 302)) f.n0 = 0;
        return f;
      };
      auto load_a = [&](const Source& f, int k, int st) {
        const bool next = k >= f.k_split;
        const int kk = (k - (next ? f.k_split : 0)) * kGemmK;
        const CUtensorMap* map = next ? f.a_next : f.a;
        uint8_t* dst = smem + st * L::kStage;
        const uint32_t full = in_first_cta(&bars->full[st]);
        if (f.a_mn) {
#pragma unroll
          for (int i = 0; i < kRows / 64; ++i)
            tma_load_2d_pair(map, full, dst + i * 64 * kGemmK * 2, f.m0 + i * 64, kk);
        } else {
          tma_load_2d_pair(map, full, dst, kk, f.m0);
        }
      };
      auto load_b = [&](const Source& f, int k, int st) {
        const bool next = k >= f.k_split;
        const int kk = (k - (next ? f.k_split : 0)) * kGemmK;
        const CUtensorMap* map = next ? f.b_next : f.b;
        uint8_t* dst = smem + st * L::kStage + kTileA;
        const uint32_t full = in_first_cta(&bars->full[st]);
        if (f.b_mn) {
#pragma unroll
          for (int i = 0; i < kRowsB / 64; ++i)
            tma_load_2d_pair(map, full, dst + i * 64 * kGemmK * 2, f.n0 + i * 64, kk);
        } else {
          tma_load_2d_pair(map, full, dst, kk, f.n0);
        }
      };
      auto expect = [&](int st) {   // both CTAs' parts
        if (rank == 0) mbar_expect_tx(&bars->full[st], 2 * L::kStage);
      };
      // the first stages' weights need not wait for the launch before
      int early = 0;
      if (g.follows == FOLLOWS_A) {
        const Unit t = unit_at(g, pair);
        const Source f = source(t);
        early = min(kStages, t.k1 - t.k0);
        for (int i = 0; i < early; ++i) {
          expect(i);
          load_b(f, t.k0 + i, i);
        }
        griddep_wait();
        for (int i = 0; i < early; ++i) load_a(f, t.k0 + i, i);
      } else if (g.follows == FOLLOWS_BOTH) {
        griddep_wait();
      }
      int j = early;   // k tiles so far, across units
      for (int r = 0; unit_of(r) < units && !*abort; ++r) {
        const Unit t = unit_at(g, unit_of(r));
        const Source f = source(t);
        for (int k = t.k0 + (r == 0 ? early : 0); k < t.k1; ++k, ++j) {
          const int st = j % kStages;
          if (j >= kStages &&
              !mbar_wait_cluster(&bars->empty[st], ((j / kStages) - 1) & 1, lim, abort)) {
            record_timeout(g.status, abort, 31);
            break;
          }
          expect(st);
          load_a(f, k, st);
          load_b(f, k, st);
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
      bool ok = true;
      int j = 0, n = 0;   // k tiles and units so far
      Work t = work_at(g, pair), next = t;
      // its waits are bounded, and the launch before may take longer than the bound
      if (g.follows != FOLLOWS_NONE) griddep_wait();
      for (; ok && unit_of(n) < units; ++n, t = next) {
        if (unit_of(n + 1) < units) next = work_at(g, unit_of(n + 1));
        const int s = n & 1;
        const int a_mn = g.p[t.p].a_mn, b_mn = g.p[t.p].b_mn;
        const uint32_t idesc = idesc_bf16(kGemmM, kN, a_mn, b_mn);
        // 16 k further: 32 bytes along a K-major row, 16 rows of an MN-major box
        const uint32_t a_step = a_mn ? 2048 : 32, b_step = b_mn ? 2048 : 32;
        const uint32_t a_lbo = a_mn ? 64 * kGemmK * 2 : 16, b_lbo = b_mn ? 64 * kGemmK * 2 : 16;
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
          const uint32_t pa = smem_u32(smem + st * L::kStage), pb = pa + kTileA;
#pragma unroll
          for (int i = 0; i < kGemmK / 16; ++i)
            mma_bf16_pair(tmem + s * kN, sdesc_sw128(pa + i * a_step, a_lbo, 1024),
                          sdesc_sw128(pb + i * b_step, b_lbo, 1024), idesc,
                          (k > t.k0 || i > 0) ? 1u : 0u);
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
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const bool issues = part == 0 && lane == 0;   // of the quarter's boxes
    const int box_bar = 1 + quarter;
    auto box_sync = [&] { named_sync(box_bar, kBoxThreads); };
    uint8_t* boxes = smem + L::kBoxes + quarter * L::kBoxBytes;
    constexpr int kTileN = kEpi == GEMM_GLU ? kN / 2 : kN;
    constexpr int kChunks = kTileN / 64;
    auto first_row = [&](const Unit& t) {
      const int split = g.p[t.p].m_split;
      return (t.m - (t.m >= split ? split : 0)) * kGemmM + rank * kRows + quarter * 32;
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
        if (u >= g.p[0].whole) return;
        fetch(unit_at(g, u), 0);
        ++fetched;
      }
    };
    if (g.follows != FOLLOWS_NONE) griddep_wait();
    fetch_first(pair);
    bool ok = true;
    for (; ok && unit_of(n) < units; ++n) {
      const Unit t = unit_at(g, unit_of(n));
      const int s = n & 1;
      // all warps of a box go on, or none
      if (!named_all(box_bar, kBoxThreads,
                     mbar_wait_cluster(&bars->acc_full[s], (n >> 1) & 1, lim, abort))) {
        if (lane == 0) record_timeout(g.status, abort, 33);
        break;
      }
      tc_fence_after();
      const GemmProblem& p = g.p[t.p];
      const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + s * kN;
      const int second = t.m >= p.m_split;
      const int row0 = first_row(t), tile_row = rank * kRows + quarter * 32 + lane;
      auto release = [&] {   // the next products may overwrite the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(in_first_cta(&bars->acc_empty[s]));
      };
      const bool shared = t.slot >= 0;
      if (shared) {
        const bool in = row0 + lane < p.M;
#pragma unroll 1
        for (int c = 0; c < kN / 64; ++c) {
          const int col = c * 64 + part * kCols;
          float x[kCols];
          load_acc(acc + col, x);
          if (in) store_partial<kN>(g.partial, t.slot, col, tile_row, x);
          __syncwarp();   // the next load of the accumulator is the whole warp's
        }
        release();
        // these warps' rows of all shares: the last to get here goes on with them
        __threadfence();
        box_sync();
        bool last = true;
        if (issues) {
          int32_t* ticket = g.tickets + t.ticket * kTickets + rank * 4 + quarter;
          last = atomicAdd(ticket, 1) == p.shares - 1;
          if (last) *ticket = 0;
          __threadfence();
        }
        if (!named_all(box_bar, kBoxThreads, last)) continue;
      }
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        const int col = c * 64 + part * kCols, box_col = t.n * kTileN + c * 64;
        const bool stores = row0 < p.M && box_col < p.N;   // the box is not wholly past the end
        float x[kCols];
        auto take = [&](int at, float (&f)[kCols]) {
          if (!shared) {
            load_acc(acc + at, f);
          } else if (row0 + lane < p.M) {
            load_partials<kN>(g.partial, t.slot - t.share, p.shares, at, tile_row, f);
          } else {
#pragma unroll
            for (int i = 0; i < kCols; ++i) f[i] = 0.f;
          }
        };
        take(col, x);
        if constexpr (kEpi == GEMM_GLU) {
          float v[kCols];
          take(kTileN + col, v);
          if (issues) bulk_wait_read<0>();   // the boxes' last stores have read them
          box_sync();
          if (g.keep) {
            put_kept(boxes + kBf16Box, boxes + 3 * kBf16Box, lane, part, x);
            put_kept(boxes + 2 * kBf16Box, boxes + 3 * kBf16Box + kByteBox, lane, part, v);
          }
          with_activation(g.act, [&](auto act) {
            float unused;
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              x[i] = activation<false, true>(x[i], act.value, unused) * v[i];
          });
          put_bf16(boxes, lane, part, x);
          fence_proxy_async_smem();
          box_sync();
          if (issues && stores) {
            tma_store_2d(&p.out[0], boxes, box_col, row0);
            if (g.keep) {
              tma_store_2d(&g.gate[0], boxes + kBf16Box, box_col, row0);
              tma_store_2d(&g.up[0], boxes + 2 * kBf16Box, box_col, row0);
              tma_store_2d(&g.gate[1], boxes + 3 * kBf16Box, box_col, row0);
              tma_store_2d(&g.up[1], boxes + 3 * kBf16Box + kByteBox, box_col, row0);
            }
            bulk_commit();
          }
        } else if constexpr (kEpi == GEMM_STORE) {
          uint8_t* box = boxes + (p.out_f32 ? 0 : c & 1) * kBf16Box;
          if (issues) {
            if (p.out_f32 || c == 0) bulk_wait_read<0>();   // the last tile's may be fp32
            else bulk_wait_read<1>();
          }
          box_sync();
          if (p.out_f32) put_f32(box, lane, part, x);
          else put_bf16(box, lane, part, x);
          fence_proxy_async_smem();
          box_sync();
          if (issues) {
            if (stores) tma_store_2d(&p.out[second], box, box_col, row0);
            if (stores && p.out_f32 && box_col + 32 < p.N)
              tma_store_2d(&p.out[second], box + kBf16Box, box_col + 32, row0);
            bulk_commit();   // one group a chunk, so that the count holds
          }
        } else {
          if (fetched == got) {   // a shared tile's, or the first after one
            fetch(t, c);
            ++fetched;
          }
          if (!named_all(box_bar, kBoxThreads, mbar_wait(&bars->box[quarter], got & 1, lim, abort))) {
            if (lane == 0) record_timeout(g.status, abort, 34);
            ok = false;
            break;
          }
          ++got;
          uint4 kg[kCols / 8], ku[kCols / 8], lg[kCols / 16], lu[kCols / 16];
#pragma unroll
          for (int q = 0; q < kCols / 8; ++q) {
            kg[q] = *piece<128>(boxes, lane, part * (kCols / 8) + q);
            ku[q] = *piece<128>(boxes + kBf16Box, lane, part * (kCols / 8) + q);
          }
#pragma unroll
          for (int q = 0; q < kCols / 16; ++q) {
            lg[q] = *piece<64>(boxes + 2 * kBf16Box, lane, part * (kCols / 16) + q);
            lu[q] = *piece<64>(boxes + 2 * kBf16Box + kByteBox, lane, part * (kCols / 16) + q);
          }
          if (issues) bulk_wait_read<0>();   // the last stores have read their boxes
          box_sync();   // all have read: the next chunk may land
          if (c + 1 < kChunks) {
            fetch(t, c + 1);
            ++fetched;
          } else {
            fetch_first(unit_of(n + 1));
          }
          uint8_t* out = boxes + 2 * (kBf16Box + kByteBox);
          const uint32_t* wg = reinterpret_cast<const uint32_t*>(kg);
          const uint32_t* wu = reinterpret_cast<const uint32_t*>(ku);
          const uint32_t* bg = reinterpret_cast<const uint32_t*>(lg);
          const uint32_t* bu = reinterpret_cast<const uint32_t*>(lu);
#pragma unroll
          for (int q = 0; q < kCols / 8; ++q) {   // eight columns at a time
            float gate[8], up[8], h[8];
            rejoin8(wg + 4 * q, bg + 2 * q, gate);
            rejoin8(wu + 4 * q, bu + 2 * q, up);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float da;
              const float a = activation<true, true>(gate[e], g.act, da), dh = x[8 * q + e];
              h[e] = a * up[e];
              gate[e] = dh * up[e] * da;
              up[e] = dh * a;
            }
            auto put = [&](int which, const float (&f)[8]) {
              *piece<128>(out + which * kBf16Box, lane, part * (kCols / 8) + q) =
                  make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                             pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
            };
            put(0, gate);
            put(1, up);
            put(2, h);
          }
          fence_proxy_async_smem();
          box_sync();
          if (issues && stores) {
            tma_store_2d(&g.dgate, out, box_col, row0);
            tma_store_2d(&g.dup, out + kBf16Box, box_col, row0);
            tma_store_2d(&p.out[0], out + 2 * kBf16Box, box_col, row0);
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
      bulk_wait_read<0>();   // the boxes may go; the kernel's end waits for the writes
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

template <int kEpi, int kN>
cudaError_t launch_t(const GemmArgs& g, int sms, cudaStream_t st) {
  auto kernel = gemm_kernel<kEpi, kN>;
  constexpr int smem = Layout<kEpi, kN>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int pairs = g.units < sms / 2 ? g.units : sms / 2;
  if (pairs < 1) return cudaErrorInvalidConfiguration;
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

cudaError_t launch_gemm_bf16(const GemmArgs& g, int epilogue, int tile_n, int sms,
                             cudaStream_t st) {
  if (tile_n != 256 && tile_n != 128) return cudaErrorInvalidValue;
  const bool wide = tile_n == 256;
  if (epilogue == GEMM_GLU)
    return wide ? launch_t<GEMM_GLU, 256>(g, sms, st) : launch_t<GEMM_GLU, 128>(g, sms, st);
  if (epilogue == GEMM_DGLU)
    return wide ? launch_t<GEMM_DGLU, 256>(g, sms, st) : launch_t<GEMM_DGLU, 128>(g, sms, st);
  return wide ? launch_t<GEMM_STORE, 256>(g, sms, st) : launch_t<GEMM_STORE, 128>(g, sms, st);
}

}  // namespace cpattn
