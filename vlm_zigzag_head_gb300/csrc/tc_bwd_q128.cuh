// Attention backward over all ring steps in one launch, on 5th-generation
// tensor cores (sm_103a), with 128-query tiles so that every product is a
// 128 x 128 (x D) MMA.
//
// One CTA owns one key tile (128 keys of one KV head) and walks, in ring-step
// order, the query runs that meet those keys over all ring steps, for every
// query head that reads this KV head (page "context-parallel-multimodal"
// §4.2: each rank differentiates its queries against the KV it saw; the KV
// owner receives dK/dV, here summed on chip over the steps and written once;
// the replicated prefix gets one gradient per rank: one item per slot when
// the per-rank terms are kept, else one item that walks every rank's queries
// and writes their sum).  Per 128-row query tile i, with the final lse:
//
//   S^T  = K Q^T          dP^T = V dO^T                          (TMEM)
//   P^T  = exp2(S^T * scale*log2e - lse2),  dS^T = P^T (dP^T - D)  (registers)
//   dV  += P^T dO   (P^T read from TMEM)   dK += dS^T Q            (TMEM, whole item)
//   dQ   = dS K     -> staged per warp in swizzled shared memory, added
//                      into fp32 dQ (scaled) by bulk tensor reduce-adds
//
// Tensor memory (512 columns):
//   D = 128: S^T [0,128) (P^T overwrites its columns [0,32) and [64,96)),
//            dP^T [128,256) (dQ overwrites it once read), dK [256,384),
//            dV [384,512);
//   D = 64:  S^T [0,128), dP^T [128,256), dK [256,320), dV [320,384),
//            dQ [384,448).
// Issue order per tile: dP_i, dV_i, S_{i+1}, dQ_i, dK_i.  The P part of the
// softmax work of tile i runs while dQ_{i-1}, dK_{i-1} and dP_i compute; the
// dS part while dV_i and S_{i+1} do; the dQ drain while dK_i does.  With
// D = 128, dP_{i+1} waits for the drain to have read dQ_i out of the dP^T
// columns.
//
// For softmax scales above kF16OperandScale the dQ values are large enough
// that one bf16 rounding of dS would dominate their error.  S^T, dQ and dK
// then run on f16 operands: the host-made copies Q * 2^-eQ and K * 2^-eK, and
// dS^T * 2^-eS rounded to f16 (three more mantissa bits than bf16); the
// factors are undone in fp32 (OpScales).  dP^T and dV keep bf16 V, dO and P^T.
// Modified scores choose the types item by item, from the range of the item's sample
// (OPS_ITEM, operand_range.cuh): one power of two for all of a call's dS would take the
// bits of samples and tokens with small gradients.
//
// Warp roles (512 threads; TMEM lane quarter of warp w is w % 4):
//   warp 0       TMA producer: K, V once; Q and the lse2 / D rows per tile
//   warp 1       TMEM allocation; lane 0 issues every tcgen05.mma
//   warp 2       TMA producer: dO per tile
//   warp 3       clears rows of another sample in the tiles that hold some (isolate)
//   warps 4..11  P / dS (two warpgroups, 64 query columns each; thread = key
//                row), then the dK / dV epilogue
//   warps 12..15 dQ drain; thread = query row (TMEM lane of dQ)
// Registers: warpgroup 0 drops to 64 (the least that leaves its MMA and
// producer code without spills), the P / dS warpgroups rise to 136 and the
// drain warpgroup to 168 (128 * 64 + 256 * 136 + 128 * 168 <= 512 * 128), so a
// drain thread can hold its whole dQ row and free the TMEM at once.  Modified
// scores need more: 144 and 152 (the same sum; 18688 tokens, 8 heads, capped: 1688
// us against 1819; plain scores are better off with the first split, 1491 to 1527);
// a table 152 and 144, the launch's total (1633 -> 1605, 12 288 tokens x 8 of 64
// 595 -> 577; a cap without one 1642 -> 1654).
//
// With kCap or kBias (score.cuh) the P / dS warps recompute the modified scores
// from S^T; under a cap dS also takes the factor 1 - tanh^2.  A table bias's
// gradient is the sum of dS over the pairs of a distance (bias_grad below).
#pragma once
#include <cuda_bf16.h>

#include <type_traits>

#include "check.cuh"
#include "kernels.h"
#include "operand_range.cuh"
#include "ptx.cuh"
#include "score.cuh"
#include "tc.h"

namespace cpattn {

namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kBK = kBwdTileK;     // 128 keys
constexpr int kBQ = 128;           // queries per inner tile
constexpr int kQStages = 2;
constexpr int kLdRows = kBQ + 4;   // lse2 / D box: 128 rows plus alignment slack
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColDP = 128;

template <int D>
struct Cols {
  static constexpr uint32_t kDK = 256;
  static constexpr uint32_t kDV = kDK + D;
  static constexpr uint32_t kDQ = D == 128 ? kColDP : kDV + D;   // D = 128: aliases dP^T
  static constexpr bool kAliased = D == 128;
};

template <int D>
struct Lay {
  static constexpr int kBox = 128 * 128;        // 128 rows x 128 bytes
  static constexpr int kTile = D / 64 * kBox;   // 128 rows x D bf16
  // dO is read only by dP_i and dV_i (adjacent products): with D = 128 one
  // buffer suffices and leaves room for the dQ staging
  static constexpr int kDOStages = D == 128 ? 1 : 2;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kTile;
  static constexpr int kQ = kV + kTile;                     // [stage]
  static constexpr int kDO = kQ + kQStages * kTile;         // [stage]
  static constexpr int kDS = kDO + kDOStages * kTile;       // dS^T: 2 boxes [128 keys][64 q]
  static constexpr int kStg = kDS + 2 * kBox;
  static constexpr int kStgWarp = 32 * 128;                 // [32 rows][32 fp32], 128-byte swizzle
  static constexpr int kLd = kStg + 4 * kStgWarp;           // [stage] {lse2[132], D[132]}
  static constexpr int kLdBytes = 2 * kLdRows * 4;
  static constexpr int kLdStride = (kLdBytes + 127) / 128 * 128;
  static constexpr int kItem = kLd + kQStages * kLdStride;
  static constexpr int kInfo = kItem + 128;                 // [stage] TileInfo of the Q tile
  static constexpr int kBars = kInfo + kQStages * 32;
  static constexpr int kBytes = kBars + 256;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kStg % 1024 == 0, "swizzled staging must be 1024-byte aligned");
  static_assert(kLd % 16 == 0 && (kLdRows * 4) % 16 == 0, "16-byte lse2 / D loads");
};
static_assert(Lay<128>::kAlloc <= 227 * 1024, "shared memory budget");
static_assert(Lay<64>::kAlloc <= 227 * 1024, "shared memory budget");

// What the P / dS warps need of a query tile, written by the Q producer
// beside the tile (published by the same barrier as the Q load).
struct TileInfo {
  int32_t tile_row;   // natural row of the tile's first query
  int32_t row_in;     // the same query's position inside its run
  int32_t causal, delta, len;   // the run's visibility rule and length
  int32_t rel;        // distance between the run's first query and the item's first key
  int32_t pad[2];
};
static_assert(sizeof(TileInfo) == 32, "TileInfo layout");

struct Bars {
  uint64_t kv_full;
  uint64_t kv_raw, q_raw[kQStages], do_raw[2];   // tiles cleared before their *_full (isolate)
  uint64_t q_full[kQStages], q_empty[kQStages];
  uint64_t do_full[2], do_empty[2];
  uint64_t s_full, p_full, dp_full, ds_full;
  uint64_t dq_full, dq_free;
  uint64_t dkv_done;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  Operands ops;   // OPS_ITEM
};
static_assert(sizeof(Bars) <= 256, "barrier block");

__device__ __forceinline__ int run_qtiles(const Seg& s) {
  const int start = s.causal && s.delta < 0 ? -s.delta : 0;
  const int n = s.len - start;
  return n > 0 ? (n + kBQ - 1) / kBQ : 0;
}
__device__ __forceinline__ int run_qstart(const Seg& s) {
  return s.causal && s.delta < 0 ? -s.delta : 0;
}

// Each role walks the item's query tiles in order: g advances by one, or
// wraps to 0 for the next query head.  The walk keeps its current run and
// the number of tiles before it, so finding the g-th tile (its run, the run's
// first query and the tile index inside the run) costs one run read.
struct TileWalk {
  int s = 0, base = 0;
};
__device__ __forceinline__ void tile_of(const Seg* runs, int nseg, int g, TileWalk& w, Seg& sg,
                                        int& q0, int& t) {
  if (g < w.base) {
    w.s = 0;
    w.base = 0;
  }
  sg = runs[w.s];
  int nt = run_qtiles(sg);
  while (g >= w.base + nt && w.s + 1 < nseg) {
    w.base += nt;
    sg = runs[++w.s];
    nt = run_qtiles(sg);
  }
  q0 = run_qstart(sg);
  t = g - w.base;
}

// The barriers of a producer's loads over N stages: a stage's own one, or its raw
// one for a tile that warp 3 clears first.  Bit st of each word belongs to stage st.
template <int N>
struct Loads {
  uint32_t used = 0, raw = 0;                  // the stage has a load; it is on the raw barrier
  uint32_t full_phase = 0, raw_phase = 0;      // phases of the next load
  uint32_t last = 0;                           // phase of the last load
  __device__ __forceinline__ uint64_t* next(int st, bool on_raw, uint64_t* full, uint64_t* rawb) {
    const uint32_t bit = 1u << st;
    // a stage's own barrier completes once per tile, whoever publishes it
    last = (last & ~bit) | ((on_raw ? raw_phase : full_phase) & bit);
    used |= bit;
    raw = on_raw ? raw | bit : raw & ~bit;
    if (on_raw) raw_phase ^= bit;
    full_phase ^= bit;
    return on_raw ? rawb + st : full + st;
  }
  // every load must have landed before the CTA exits (normally the consumers
  // already waited for them and these waits return at once)
  __device__ __forceinline__ void drain(uint64_t* full, uint64_t* rawb) const {
    int zero = 0;
    for (int st = 0; st < N; ++st)
      if (used >> st & 1)
        mbar_wait(raw >> st & 1 ? rawb + st : full + st, last >> st & 1, kDrainLimit, &zero);
  }
};

// Four neighbouring per-query values (minus lse2 or minus D); vec: 16-byte aligned.
__device__ __forceinline__ void load_row4(const float* p, bool vec, float (&v)[4]) {
  if (vec) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else {
#pragma unroll
    for (int y = 0; y < 4; ++y) v[y] = p[y];
  }
}

// With a cap and a table P is kept as f16 for the bias's gradient.  P is a probability,
// about 1 at most, and far keys of a long row have 2^-17 and less: f16 holds P 2^14 to
// 2^-11 of its value from P = 2^-28 on, P itself from 2^-14 (2048 tokens, far buckets held
// down to P of 2^-26: dbias off by 28 % and 5e-6).  The factor is a term of the exponent,
// so it costs nothing; bf16 and fp32 round alike at any power of two, and it is taken out
// where dQ, dK, dV and the sums of dS leave.
template <bool kCap, int kBias>
constexpr int kPLog2 = kCap && kBias == SCORE_TABLE ? 14 : 0;
template <bool kCap, int kBias>
constexpr float kPUnit = 1.f / (1 << kPLog2<kCap, kBias>);   // 1 / 2^kPLog2

// P^T of 32 queries from their products (rs), with modified scores: the
// probabilities as bf16 pairs in pk (the dV operand); in place over the products
// what dS multiplies: P, or under a cap -P (1 - tanh^2), whose sign the factors of
// dQ and dK undo.  kFast: every pair is
// visible, the cap's polynomial holds and the bias is linear along the queries.
// With a cap and a table, ph: P alone as f16 pairs, for the bias's gradient (registers
// for fp32 are lacking; bf16 pairs would show in it).  All of these are then P times
// 2^kPLog2.
// mul: scale or cap in log2 units, inv its inverse.  x0: the half's first query in
// the 64; ld: its lse2.
template <bool kCap, int kBias, bool kFast>
__device__ __forceinline__ void score_columns(uint32_t (&rs)[32], uint32_t (&pk)[16],
                                              uint32_t* ph, int x0, float mul,
                                              float inv, const score::BwdCap<kCap>& cap,
                                              const score::TileBias& tb, bool poly,
                                              const float* ld, bool vec, int first_vis,
                                              int end_vis) {
  float base = tb.base;
  if constexpr (kPLog2<kCap, kBias> != 0) base += kPLog2<kCap, kBias>;
  const uint64_t mul_2 = pack2(mul, mul), base2 = pack2(base, base);
  const float step = tb.step * inv;   // slopes, before `mul`
  const bool column = kBias != SCORE_PLAIN && (tb.both || tb.tab != nullptr);
#pragma unroll
  for (int x = 0; x < 32; x += 4) {
    float l[4];
    load_row4(ld + x, vec, l);
#pragma unroll
    for (int y = x; y < x + 4; y += 2) {
      uint64_t s = pack2(__uint_as_float(rs[y]), __uint_as_float(rs[y + 1])), w = 0;
      float s0, s1;
      if constexpr (kCap) {
        if (kFast || poly) {
          s = cap.poly(s);
        } else {
          unpack2(s, s0, s1);
          s = pack2(cap.any(s0), cap.any(s1));
        }
        w = cap.minus_slope(s);
      }
      if constexpr (kBias == SCORE_SLOPES) {
        unpack2(s, s0, s1);
        s = pack2(fmaf((float)y, step, s0), fmaf((float)(y + 1), step, s1));
      }
      uint64_t add = pack2(l[y - x], l[y - x + 1]);   // minus lse2
      if constexpr (kBias != SCORE_PLAIN) add = add2(add, base2);
      if (!kFast && column)
        add = add2(add, pack2(score::column_bias<kBias, 1>(tb, x0 + y),
                              score::column_bias<kBias, 1>(tb, x0 + y + 1)));
      float p0, p1;
      unpack2(fma2(s, mul_2, add), p0, p1);
      p0 = ex2(p0);
      p1 = ex2(p1);
      if constexpr (!kFast) {
        if (x0 + y < first_vis || x0 + y >= end_vis) p0 = 0.f;
        if (x0 + y + 1 < first_vis || x0 + y + 1 >= end_vis) p1 = 0.f;
      }
      pk[y / 2] = pack_bf16x2(p0, p1);
      if constexpr (kCap && kBias == SCORE_TABLE) ph[y / 2] = pack_f16x2(p0, p1);
      if constexpr (kCap) unpack2(mul2(pack2(p0, p1), w), p0, p1);   // -P (1 - tanh^2)
      rs[y] = __float_as_uint(p0);
      rs[y + 1] = __float_as_uint(p1);
    }
  }
}

// Whether a warp's 64 products per lane all lie in the polynomial's range.
template <bool kCap>
__device__ __forceinline__ bool in_poly_range(const uint32_t (&rs)[2][32],
                                              const score::BwdCap<kCap>& cap) {
  if constexpr (!kCap) return true;
  float big[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int x = 0; x < 64; x += 2)
    big[(x >> 1) & 3] = fmaxf(fmaxf(big[(x >> 1) & 3], fabsf(__uint_as_float(rs[x >> 5][x & 31]))),
                              fabsf(__uint_as_float(rs[x >> 5][(x & 31) + 1])));
  return cap.in_range(fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3])));
}

// Gradient of a table bias: dS summed over the pairs of each |distance|.
//
// In a tile near the diagonal lane u of a warp holds distance base + x - u at
// query x of a block of 32.  Query x's values are turned by x lanes, lane L
// taking u = (x - L) mod 32: it then always adds distance base + L (x >= L) or
// base + L - 32 (x < L).  The shuffles do not wait on one another, and a warp
// hands over 96 sums per 64 queries, one per lane in three coalesced atomics,
// where an atomic per element would be 21 times as many.  Tiles at or past the
// table's last distance sum into one register.
struct Diagonals {
  float all = 0.f, up = 0.f;   // both kinds of a block's sums; those with x >= L
};
__device__ __forceinline__ void bias_grad(Diagonals& g, int x, float v, int lane) {
  const float w = __shfl_sync(0xffffffffu, v, (x - lane) & 31);
  g.all += w;
  if (x >= lane) g.up += w;
}
// mul: kPUnit (the far sums keep the factor to the end).
__device__ __forceinline__ void add_distance(const ScoreArgs& s, int h, int dist, float v,
                                             float mul, float& far_sum) {
  const int d = dist < 0 ? -dist : dist;
  if (d >= s.n_dist - 1) far_sum += v;
  else atomicAdd(s.dtable + (long long)h * s.n_dist + d, v * mul);
}
__device__ __forceinline__ void flush_far(const ScoreArgs& s, int h, int lane, float mul,
                                          float& far_sum) {
  float v = far_sum;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) atomicAdd(s.dtable + (long long)h * s.n_dist + s.n_dist - 1, v * mul);
  far_sum = 0.f;
}

template <int D, int kOps, bool kShared, bool kCap, int kBias>
__global__ void __launch_bounds__(kThreads, 1)
    tc_bwd_q128_kernel(const __grid_constant__ TcBwdArgs a) {
  using L = Lay<D>;
  using C = Cols<D>;
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte aligned base, derived from the shared array itself so that the
  // compiler keeps shared-space (not generic) loads and stores
  uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_item = a.item_major ? (kShared ? a.Hkv * a.kv_split : a.Hkv) : 1;
  const int item_idx = a.item_major ? blockIdx.x / per_item : blockIdx.x % a.n_items;
  const int slot = a.item_major ? blockIdx.x % per_item : blockIdx.x / a.n_items;
  // KV head hk; its query heads are hk*G .. hk*G+G-1.  Shared groups
  // (kv_split > 1): kv_split CTAs take Gs = G / kv_split consecutive query
  // heads each, and their partial dK / dV meet in global memory by
  // reduce-adds.
  const int hk = kShared ? slot / a.kv_split : slot;
  const int G = a.H / a.Hkv;
  const int Gs = kShared ? G / a.kv_split : G;   // query heads of this CTA
  const int hq0 = hk * G + (kShared ? slot % a.kv_split * Gs : 0);
  BwdItem& it = *reinterpret_cast<BwdItem*>(smem + L::kItem);
  if (warp == 0)  // the work item, copied once into shared memory (128 bytes)
    reinterpret_cast<uint32_t*>(&it)[lane] =
        reinterpret_cast<const uint32_t*>(a.items + item_idx)[lane];
  volatile int* abort = &bars->abort;
  const long long lim = a.wait_limit;

  if (threadIdx.x == 0) {
    mbar_init(&bars->kv_full, 1);
    mbar_init(&bars->kv_raw, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->q_raw[s], 1);
      mbar_init(&bars->do_raw[s], 1);
    }
    for (int s = 0; s < kQStages; ++s) {
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->do_full[s], 1);
      mbar_init(&bars->do_empty[s], 1);
    }
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->p_full, 8);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->ds_full, 8);
    mbar_init(&bars->dq_full, 1);
    mbar_init(&bars->dq_free, 4);
    mbar_init(&bars->dkv_done, 1);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    if constexpr (kOps == OPS_ITEM) {
      const int sample = a.items[item_idx].slot;
      bars->ops = choose_operands(CP_IN_RANGE(sample, 0, a.n_samples, a.status, 213) &&
                                          CP_IN_RANGE(hk, 0, a.Hkv, a.status, 214)
                                      ? a.ranges[(long long)sample * a.Hkv + hk]
                                      : OperandRange{});
    }
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
  // S, dQ and dK of this item on f16 operands
  const bool f16 = kOps == OPS_F16 || (kOps == OPS_ITEM && bars->ops.f16 != 0);

  // the item's query runs, in ring-step order, from the plan's run list
  const int nseg = it.nseg;
  const Seg* runs = a.runs + it.run0;
  int n_qt = 0;   // query tiles of one query head
  for (int s = 0; s < nseg; ++s) n_qt += run_qtiles(runs[s]);
  // Every role walks the same Gs * n_qt query tiles in the same order: query
  // head hq0 + j / n_qt, tile j % n_qt.  dK / dV of the KV head accumulate
  // over all of them, across every ring step, and are written once.
  // Concurrent CTAs are neighbouring key tiles that meet the same queries in
  // the same order, so the Q / dO tiles they load are shared through L2.
  const int n_all = Gs * n_qt;
  // isolate: K / V rows past the item's keys and Q / dO rows (and lse2, D) past a
  // run's end are another sample's and may be NaN.  Their P and dS are 0; so that 0
  // meets 0, the loads of such a tile complete on a raw barrier, and warp 3 clears
  // the foreign rows before it publishes the tile.
  const bool clear_kv = a.isolate && it.k_len < kBK && n_all > 0;

  if (warp < 4) {
    setmaxnreg_dec<64>();
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer: K, V, Q, lse2 / D
      if (lane == 0) {
        Loads<kQStages> loads;
        bool kv_issued = false;
        if (n_all > 0 && !(CP_IN_RANGE(it.k_row0, 0, a.T, a.status, 201) &&
                           CP_IN_RANGE(hk, 0, a.Hkv, a.status, 202))) {
          *abort = 1;
        } else if (n_all > 0) {
          uint64_t* landed = clear_kv ? &bars->kv_raw : &bars->kv_full;
          mbar_expect_tx(landed, 2 * L::kTile);
          const CUtensorMap* mk = kOps == OPS_ITEM && f16 ? &a.tm_k16 : &a.tm_k;
          for (int b = 0; b < D / 64; ++b) {
            tma_load_3d(mk, landed, smem + L::kK + b * L::kBox, b * 64, hk, it.k_row0);
            tma_load_3d(&a.tm_v, landed, smem + L::kV + b * L::kBox, b * 64, hk, it.k_row0);
          }
          kv_issued = true;
        }
        const CUtensorMap* mq = kOps == OPS_ITEM && f16 ? &a.tm_q16 : &a.tm_q;
        TileWalk walk;
        int jt = 0, hq = hq0;
        for (int j = 0; j < n_all; ++j, jt = jt + 1 == n_qt ? 0 : jt + 1, hq += jt == 0) {
          const int st = j % kQStages;
          if (*abort || (j >= kQStages &&
                         !mbar_wait(&bars->q_empty[st], ((j / kQStages) - 1) & 1, lim, abort))) {
            record_timeout(a.status, abort, 21);
            break;
          }
          Seg sg;
          int q0, t;
          tile_of(runs, nseg, jt, walk, sg, q0, t);
          const int grow = sg.row0 + q0 + t * kBQ;   // natural row of the tile's first query
          if (!CP_IN_RANGE(grow, 0, a.T, a.status, 203) || !CP_IN_RANGE(hq, 0, a.H, a.status, 204)) {
            *abort = 1;
            break;
          }
          TileInfo* info = reinterpret_cast<TileInfo*>(smem + L::kInfo) + st;
          info->tile_row = grow;
          info->row_in = q0 + t * kBQ;
          info->causal = sg.causal;
          info->delta = sg.delta;
          info->len = sg.len;
          info->rel = sg.rel;
          uint64_t* landed = loads.next(st, a.isolate && sg.len - q0 - t * kBQ < kBQ, bars->q_full,
                                        bars->q_raw);
          mbar_expect_tx(landed, L::kTile + L::kLdBytes);
          for (int b = 0; b < D / 64; ++b)
            tma_load_3d(mq, landed, smem + L::kQ + st * L::kTile + b * L::kBox, b * 64, hq,
                        grow);
          // the lse2 / D box starts at the row rounded down to 4 (16-byte TMA alignment)
          tma_load_3d(&a.tm_ld, landed, smem + L::kLd + st * L::kLdStride, grow & ~3, hq, 0);
        }
        // every load issued here must land before the CTA exits (normally the
        // consumers already waited for them and these waits return at once)
        int zero = 0;
        if (kv_issued) mbar_wait(clear_kv ? &bars->kv_raw : &bars->kv_full, 0, kDrainLimit, &zero);
        loads.drain(bars->q_full, bars->q_raw);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- TMA producer: dO
      if (lane == 0) {
        constexpr int S = L::kDOStages;
        Loads<S> loads;
        TileWalk walk;
        int jt = 0, hq = hq0;
        for (int j = 0; j < n_all; ++j, jt = jt + 1 == n_qt ? 0 : jt + 1, hq += jt == 0) {
          const int st = j % S;
          if (*abort || (j >= S && !mbar_wait(&bars->do_empty[st], ((j / S) - 1) & 1, lim, abort))) {
            record_timeout(a.status, abort, 22);
            break;
          }
          Seg sg;
          int q0, t;
          tile_of(runs, nseg, jt, walk, sg, q0, t);
          const int grow = sg.row0 + q0 + t * kBQ;
          if (!CP_IN_RANGE(grow, 0, a.T, a.status, 205) || !CP_IN_RANGE(hq, 0, a.H, a.status, 206)) {
            *abort = 1;
            break;
          }
          uint64_t* landed = loads.next(st, a.isolate && sg.len - q0 - t * kBQ < kBQ, bars->do_full,
                                        bars->do_raw);
          mbar_expect_tx(landed, L::kTile);
          for (int b = 0; b < D / 64; ++b)
            tma_load_3d(&a.tm_do, landed, smem + L::kDO + st * L::kTile + b * L::kBox, b * 64, hq,
                        grow);
        }
        loads.drain(bars->do_full, bars->do_raw);
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------- rows of another sample
      // Clears them in the tiles that landed on a raw barrier, then publishes the
      // tile; in the order in which the MMA issuer takes the tiles.
      if (clear_kv) {
        if (__all_sync(0xffffffffu, mbar_wait(&bars->kv_raw, 0, lim, abort))) {
          clear_rows<D, 32>(smem + L::kK, it.k_len, lane);
          clear_rows<D, 32>(smem + L::kV, it.k_len, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->kv_full);
        }
      }
      TileWalk walk;
      uint32_t q_phase = 0, do_phase = 0;   // bit st: phase of the stage's raw barrier
      int jt = 0;
      for (int j = 0; a.isolate && j < n_all; ++j, jt = jt + 1 == n_qt ? 0 : jt + 1) {
        Seg sg;
        int q0, t;
        tile_of(runs, nseg, jt, walk, sg, q0, t);
        const int tail = sg.len - q0 - t * kBQ;
        if (tail >= kBQ) continue;
        const int st = j % kQStages, so = j % L::kDOStages;
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&bars->q_raw[st], q_phase >> st & 1, lim, abort)))
          break;
        q_phase ^= 1u << st;
        clear_rows<D, 32>(smem + L::kQ + st * L::kTile, tail, lane);
        float* ld = reinterpret_cast<float*>(smem + L::kLd + st * L::kLdStride) +
                    ((sg.row0 + q0 + t * kBQ) & 3);
        for (int x = tail + lane; x < kBQ; x += 32) ld[x] = ld[kLdRows + x] = 0.f;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full[st]);
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&bars->do_raw[so], do_phase >> so & 1, lim, abort)))
          break;
        do_phase ^= 1u << so;
        clear_rows<D, 32>(smem + L::kDO + so * L::kTile, tail, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->do_full[so]);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0) {
        // K-major A and B; B (Q, dO) MN-major; A (dS), B (K) MN-major.  S^T, dQ
        // and dK take f16 operands when f16 (K, Q copies and dS^T all f16);
        // dP^T and dV always bf16 (V, dO, P^T)
        const uint32_t idesc_s = f16 ? idesc_f16(kBK, kBQ, 0, 0) : idesc_bf16(kBK, kBQ, 0, 0);
        constexpr uint32_t idesc_dp = idesc_bf16(kBK, kBQ, 0, 0);
        constexpr uint32_t idesc_dv = idesc_bf16(kBK, D, 0, 1);
        const uint32_t idesc_dk = f16 ? idesc_f16(kBK, D, 0, 1) : idesc_bf16(kBK, D, 0, 1);
        const uint32_t idesc_dq = f16 ? idesc_f16(kBQ, D, 1, 1) : idesc_bf16(kBQ, D, 1, 1);
        const uint32_t k_addr = smem_u32(smem + L::kK), v_addr = smem_u32(smem + L::kV);
        const uint32_t ds_addr = smem_u32(smem + L::kDS);
        // S^T (into the S columns) from K and Q stage st
        auto issue_s = [&](int st) {
          const uint32_t q_addr = smem_u32(smem + L::kQ + st * L::kTile);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {      // over head dim
            const uint32_t o = (kk / 4) * L::kBox + (kk % 4) * 32;
            mma_bf16(tmem + kColS, sdesc_sw128(k_addr + o, 16, 1024),
                     sdesc_sw128(q_addr + o, 16, 1024), idesc_s, kk > 0 ? 1u : 0u);
          }
          mma_commit(&bars->s_full);
        };
        bool ok = true;
        if (n_all > 0) {
          ok = mbar_wait(&bars->kv_full, 0, lim, abort) &&
               mbar_wait(&bars->q_full[0], 0, lim, abort);
          if (ok) {
            tc_fence_after();
            issue_s(0);
          }
        }
        for (int i = 0; ok && i < n_all; ++i) {
          const int st = i % kQStages, so = i % L::kDOStages;
          // ---- dP^T_i = V dO_i^T
          if (!mbar_wait(&bars->do_full[so], (i / L::kDOStages) & 1, lim, abort) ||
              (C::kAliased && i >= 1 && !mbar_wait(&bars->dq_free, (i - 1) & 1, lim, abort))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t do_addr = smem_u32(smem + L::kDO + so * L::kTile);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk / 4) * L::kBox + (kk % 4) * 32;
            mma_bf16(tmem + kColDP, sdesc_sw128(v_addr + o, 16, 1024),
                     sdesc_sw128(do_addr + o, 16, 1024), idesc_dp, kk > 0 ? 1u : 0u);
          }
          mma_commit(&bars->dp_full);
          // ---- dV += P^T_i dO_i, P^T from the S columns (query pairs per column)
          if (!mbar_wait(&bars->p_full, i & 1, lim, abort)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kBQ / 16; ++kk) {    // over queries
            const uint32_t pa = tmem + kColS + (kk / 4) * 64 + (kk % 4) * 8;
            mma_bf16_ts(tmem + C::kDV, pa, sdesc_sw128(do_addr + kk * 16 * 128, L::kBox, 1024),
                        idesc_dv, (i > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(&bars->do_empty[so]);
          // ---- S^T_{i+1} (overwrites P^T_i: issued after dV_i)
          if (i + 1 < n_all) {
            const int st1 = (i + 1) % kQStages;
            if (!mbar_wait(&bars->q_full[st1], ((i + 1) / kQStages) & 1, lim, abort)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_s(st1);
          }
          // ---- dQ_i = dS_i K, then dK += dS^T_i Q_i
          if (!mbar_wait(&bars->ds_full, i & 1, lim, abort) ||
              (!C::kAliased && i >= 1 && !mbar_wait(&bars->dq_free, (i - 1) & 1, lim, abort))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {    // over keys
            const uint64_t kb = sdesc_sw128(k_addr + kk * 16 * 128, L::kBox, 1024);
            mma_bf16(tmem + C::kDQ, sdesc_sw128(ds_addr + kk * 16 * 128, L::kBox, 1024), kb,
                     idesc_dq, kk > 0 ? 1u : 0u);
          }
          mma_commit(&bars->dq_full);
          const uint32_t q_addr = smem_u32(smem + L::kQ + st * L::kTile);
#pragma unroll
          for (int kk = 0; kk < kBQ / 16; ++kk) {    // over queries
            mma_bf16(tmem + C::kDK,
                     sdesc_sw128(ds_addr + (kk / 4) * L::kBox + (kk % 4) * 32, 16, 1024),
                     sdesc_sw128(q_addr + kk * 16 * 128, L::kBox, 1024), idesc_dk,
                     (i > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(&bars->q_empty[st]);
        }
        if (ok && n_all > 0) mma_commit(&bars->dkv_done);
        if (!ok) {
          record_timeout(a.status, abort, 23);
          // nothing issued by this thread may still be running at exit
          mma_commit(&bars->drain);
          int zero = 0;
          mbar_wait(&bars->drain, 0, kDrainLimit, &zero);
        }
      }
    }
  } else if (warp >= 12) {
    setmaxnreg_inc<kBias == SCORE_TABLE ? 144 : kCap || kBias != SCORE_PLAIN ? 152 : 168>();
    // ------------------------------------------------------------ dQ drain
    // thread = query row wq * 32 + lane of the tile (TMEM lane of dQ).  The
    // whole row comes out of TMEM first (its columns are free again for the
    // next product at once); then the warp stages it 32 columns at a time in
    // its own swizzled buffer, and lane 0 adds each staged [32 rows][32
    // columns] block into dQ by a bulk tensor reduce-add (the reduction runs
    // in L2; rows past the run carry exact zeros, rows past T are clipped by
    // the tensor map).
    const int wq = warp & 3;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    // dQ = scale * (dS K); with f16 operands also undo the dS and K factors
    // dS comes negated under a cap, and times 2^kPLog2 (in f16: taken out before it is
    // rounded)
    const float dq_scale = (kCap ? -a.scale : a.scale) * (f16 ? 1.f : kPUnit<kCap, kBias>);
    const float dq_mul = kOps == OPS_F16    ? dq_scale * a.op_scales->dq_mul
                         : kOps == OPS_ITEM ? dq_scale * bars->ops.dq_mul
                                            : dq_scale;
    uint8_t* stg = smem + L::kStg + wq * L::kStgWarp;
    uint8_t* my_row = stg + lane * 128;
    const int sw = lane & 7;
    bool ok = true;
    bool pending = false;
    TileWalk walk;
    int jt = 0, hq = hq0;
    for (int j = 0; ok && j < n_all; ++j, jt = jt + 1 == n_qt ? 0 : jt + 1, hq += jt == 0) {
      Seg sg;
      int q0, t;
      tile_of(runs, nseg, jt, walk, sg, q0, t);
      const int grow = sg.row0 + q0 + t * kBQ + wq * 32;   // natural row of this warp's first query
      if (!mbar_wait(&bars->dq_full, j & 1, lim, abort)) { ok = false; break; }
      tc_fence_after();
      uint32_t r[D / 32][32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) tmem_ld32(tmem + lane_off + C::kDQ + c * 32, r[c]);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < D / 32; ++c) reg_fence32(r[c]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->dq_free);
      // rows past the run's end are another sample's: what this sample's keys (NaN,
      // it may be) give them is replaced by zero
      const bool foreign = a.isolate && lane >= sg.len - q0 - t * kBQ - wq * 32;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        // the previous reduce of this warp must have read the buffer
        if (pending && lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float4 v = make_float4(__uint_as_float(r[c][4 * x]) * dq_mul,
                                       __uint_as_float(r[c][4 * x + 1]) * dq_mul,
                                       __uint_as_float(r[c][4 * x + 2]) * dq_mul,
                                       __uint_as_float(r[c][4 * x + 3]) * dq_mul);
          *reinterpret_cast<float4*>(my_row + ((x ^ sw) << 4)) = v;
        }
        if (foreign) {
#pragma unroll 1
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<float4*>(my_row + x * 16) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && CP_IN_RANGE(grow - wq * 32, 0, a.T, a.status, 207) &&
            CP_IN_RANGE(hq, 0, a.H, a.status, 208)) {
          tma_reduce_add_3d(&a.tm_dq, stg, c * 32, hq, grow);
          bulk_commit();
        }
        pending = true;
      }
    }
    if (lane == 0) bulk_wait_all();   // every reduce-add finished before exit
    if (!ok) record_timeout(a.status, abort, 24);
  } else {
    setmaxnreg_inc<kBias == SCORE_TABLE ? 152 : kCap || kBias != SCORE_PLAIN ? 144 : 136>();
    // ------------------------------------------------------------ P / dS
    // Two warpgroups share every query tile: warpgroup g (warps 4+4g .. 7+4g)
    // computes P^T / dS^T for query columns [64g, 64g + 64) of its key rows.
    const int g = (warp - 4) >> 2;
    const int u = (warp & 3) * 32 + lane;        // key row == TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    // S^T = (K16 Q16^T) * qk_mul and dS16 = dS * ds_inv with f16 operands
    const float sl2 = kOps == OPS_F16    ? a.scale_log2 * a.op_scales->qk_mul
                      : kOps == OPS_ITEM ? a.scale_log2 * bars->ops.qk_mul
                                         : a.scale_log2;
    const float ds_inv = kOps == OPS_F16    ? a.op_scales->ds_inv
                         : kOps == OPS_ITEM ? bars->ops.ds_inv * kPUnit<kCap, kBias>
                                            : 1.f;
    const bool key_ok = u < it.k_len;
    const int sw = u & 7;
    bool ok = true;
    constexpr bool kScored = kCap || kBias != SCORE_PLAIN;
    const score::BwdCap<kCap> cap(a.score, sl2);
    const float s_mul = kCap ? cap.mul : sl2, s_inv = kScored ? 1.f / s_mul : 0.f;
    int jt = 0, hq = hq0;       // tile and query head, as the producers walk them
    float far_sum = 0.f;        // this thread's dS beyond the table (kBias: table),
    uint64_t far2 = 0;          // and the same by even and odd queries
    [[maybe_unused]] constexpr float bias_mul = kPUnit<kCap, kBias>;
    for (int i = 0; ok && i < n_all; ++i) {
      const int st = i % kQStages;
      if (!mbar_wait(&bars->q_full[st], (i / kQStages) & 1, lim, abort)) {
        ok = false;
        break;
      }
      // Everything that follows from the tile's place is worked out before its
      // products are ready.  The slot is rewritten only after this tile's dK
      // product, which waits for this warpgroup's dS.
      const TileInfo ti = reinterpret_cast<const TileInfo*>(smem + L::kInfo)[st];
      const int tile_row = ti.tile_row;                     // natural row of the tile's first query
      const int row0 = ti.row_in + g * 64;                  // first query of this half (inside the run)
      const float* ld = reinterpret_cast<const float*>(smem + L::kLd + st * L::kLdStride) +
                        (tile_row & 3) + g * 64;
      // key u is visible to query row0 + x iff x < len - row0 and, for a causal
      // run, u <= row0 + x + delta
      const int first_vis = ti.causal ? u - ti.delta - row0 : 0;
      const int end_vis = key_ok ? ti.len - row0 : 0;
      const bool whole = __all_sync(0xffffffffu, first_vis <= 0 && end_vis >= 64);
      const bool vec = (tile_row & 3) == 0;
      // distances rise along the queries; the half tile's span over its 128 keys
      const int first = ti.rel + row0;
      score::TileBias tb;
      if constexpr (kBias != SCORE_PLAIN) {
        const float slope2 = kBias == SCORE_SLOPES ? a.score.slopes[hq] * score::kLog2e : 0.f;
        tb = score::tile_bias<kBias, 1>(a.score, hq, slope2, first - u, first - (kBK - 1),
                                        first + 63, ti.causal != 0);
      }
      if (!mbar_wait(&bars->s_full, i & 1, lim, abort)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t rs[2][32];
      tmem_ld32(tmem + lane_off + kColS + g * 64, rs[0]);
      tmem_ld32(tmem + lane_off + kColS + g * 64 + 32, rs[1]);
      tmem_ld_wait();
      reg_fence32(rs[0]);
      reg_fence32(rs[1]);
      // ---- P^T: probabilities of the 64 queries, computed in place over S and
      // kept in fp32 for dS; bf16 pairs into the first 32 of this warpgroup's
      // S columns, in halves
      uint32_t ph[2][16];   // P^T as f16 pairs (cap and table), 32 queries each
      const bool poly = in_poly_range<kCap>(rs, cap);
      auto p_tile = [&](auto fast) {
        constexpr bool kFast = decltype(fast)::value;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          score::TileBias th = tb;
          th.base += 32 * h * tb.step;
          uint32_t pk[16];   // P^T as bf16 pairs
          score_columns<kCap, kBias, kFast>(rs[h], pk, ph[h], 32 * h, s_mul, s_inv, cap, th, poly,
                                            ld + 32 * h, vec, first_vis, end_vis);
          tmem_st16(tmem + lane_off + kColS + g * 64 + 16 * h, pk);
        }
      };
      if (whole && poly && !tb.both && tb.tab == nullptr) p_tile(std::true_type{});
      else p_tile(std::false_type{});
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_full);
      // ---- dS^T = P^T (dP^T - D), bf16 into shared memory (row u of box g,
      // 128-byte swizzle), 32 queries at a time
      if (!mbar_wait(&bars->dp_full, i & 1, lim, abort)) { ok = false; break; }
      tc_fence_after();
      uint8_t* srow = smem + L::kDS + g * L::kBox + u * 128;
      Diagonals diag[2];   // of the two blocks of 32 queries (kBias: table)
      auto ds_half = [&](int h, auto near_tile, auto in_f16) {
        [[maybe_unused]] constexpr bool kNear = decltype(near_tile)::value;
        constexpr bool kF16 = decltype(in_f16)::value;
        uint32_t rd[32];
        tmem_ld32(tmem + lane_off + kColDP + g * 64 + h * 32, rd);
        tmem_ld_wait();
        reg_fence32(rd);
        uint32_t hk[16];
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          float dd[4];
          load_row4(ld + kLdRows + h * 32 + x, vec, dd);
#pragma unroll
          for (int y = 0; y < 4; y += 2) {
            float d0, d1;
            const uint64_t diff = add2(pack2(dd[y], dd[y + 1]),   // minus D
                                       pack2(__uint_as_float(rd[x + y]),
                                             __uint_as_float(rd[x + y + 1])));
            const uint64_t ds = mul2(pack2(__uint_as_float(rs[h][x + y]),
                                           __uint_as_float(rs[h][x + y + 1])), diff);
            if constexpr (kBias == SCORE_TABLE) {
              uint64_t b = ds;
              if constexpr (kCap) {   // the bias is added behind the cap: P alone
                float p0, p1;
                unpack_f16x2(ph[h][(x + y) / 2], p0, p1);
                b = mul2(pack2(p0, p1), diff);
              }
              if constexpr (kNear) {
                float b0, b1;
                unpack2(b, b0, b1);
                bias_grad(diag[h], x + y, b0, lane);
                bias_grad(diag[h], x + y + 1, b1, lane);
              } else {
                far2 = add2(far2, b);
              }
            }
            unpack2(ds, d0, d1);
            if constexpr (kF16)
              hk[(x + y) / 2] = pack_f16x2(d0 * ds_inv, d1 * ds_inv);
            else
              hk[(x + y) / 2] = pack_bf16x2(d0, d1);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int off = ((h * 4 + c) ^ sw) << 4;
          *reinterpret_cast<uint4*>(srow + off) =
              make_uint4(hk[c * 4], hk[c * 4 + 1], hk[c * 4 + 2], hk[c * 4 + 3]);
        }
      };
      auto ds_tile = [&](auto in_f16) {
        if (kBias == SCORE_TABLE && tb.tab != nullptr) {
          ds_half(0, std::true_type{}, in_f16);
          ds_half(1, std::true_type{}, in_f16);
        } else {
          ds_half(0, std::false_type{}, in_f16);
          ds_half(1, std::false_type{}, in_f16);
        }
      };
      if constexpr (kOps == OPS_ITEM) {
        if (f16) ds_tile(std::true_type{});
        else ds_tile(std::false_type{});
      } else {
        ds_tile(std::bool_constant<kOps == OPS_F16>{});
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ds_full);
      if constexpr (kBias == SCORE_TABLE) {
        if (tb.tab != nullptr) {
          // distances base + L - 32, base + L and base + L + 32 of this warp's keys
          const int base = ti.rel + row0 - (warp & 3) * 32 + lane;
          add_distance(a.score, hq, base - 32, diag[0].all - diag[0].up, bias_mul, far_sum);
          add_distance(a.score, hq, base, diag[0].up + (diag[1].all - diag[1].up), bias_mul,
                       far_sum);
          add_distance(a.score, hq, base + 32, diag[1].up, bias_mul, far_sum);
        }
      }
      if (++jt == n_qt) {
        if constexpr (kBias == SCORE_TABLE) {
          float f0, f1;
          unpack2(far2, f0, f1);
          far_sum += f0 + f1;
          flush_far(a.score, hq, lane, bias_mul, far_sum);
          far2 = 0;
        }
        jt = 0;
        ++hq;
      }
    }
    // ------------------------------------------------------------ dK / dV epilogue
    if (ok && n_all > 0 && !mbar_wait(&bars->dkv_done, 0, lim, abort)) ok = false;
    if (!ok) {
      record_timeout(a.status, abort, 25);
    } else {
      tc_fence_after();
      // warpgroup 0 writes dK (scaled), warpgroup 1 writes dV
      float* dst;
      bool row_ok = key_ok && CP_IN_RANGE(hk, 0, a.Hkv, a.status, 209);
      if (it.dk_mode == DK_TEXT) {
        row_ok = row_ok && CP_IN_RANGE(it.k_row0 + u, 0, a.T, a.status, 210);
        dst = (g == 0 ? a.dk : a.dv) + ((long long)(it.k_row0 + u) * a.Hkv + hk) * D;
      } else {
        row_ok = row_ok && CP_IN_RANGE(it.slot, 0, a.n_slots, a.status, 211) &&
                 CP_IN_RANGE(it.dk_row0 + u, 0, a.pre_rows, a.status, 212);
        const long long row = (long long)it.slot * a.pre_rows + it.dk_row0 + u;
        dst = (g == 0 ? a.pre_k : a.pre_v) + (row * a.Hkv + hk) * D;
      }
      __nv_bfloat16* dst16 =
          reinterpret_cast<__nv_bfloat16*>(g == 0 ? a.dk : a.dv) +
          ((long long)(it.k_row0 + u) * a.Hkv + hk) * D;   // dkv_bf16: DK_TEXT items only
      const bool first = (it.flags & F_FIRST) != 0;
      constexpr float p_unit = kPUnit<kCap, kBias>;
      float dk_mul = (kCap ? -a.scale : a.scale) * (f16 ? 1.f : p_unit);
      if constexpr (kOps == OPS_F16) dk_mul *= a.op_scales->dk_mul;
      if constexpr (kOps == OPS_ITEM) dk_mul *= bars->ops.dk_mul;
      const float mul = g == 0 ? dk_mul : p_unit;
      const uint32_t col = g == 0 ? C::kDK : C::kDV;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        if (n_all > 0) {
          tmem_ld32(tmem + lane_off + col + c * 32, r);
          tmem_ld_wait();
          reg_fence32(r);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) r[x] = 0u;
        }
        if (!row_ok) continue;
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          float4 v = make_float4(__uint_as_float(r[x]) * mul, __uint_as_float(r[x + 1]) * mul,
                                 __uint_as_float(r[x + 2]) * mul, __uint_as_float(r[x + 3]) * mul);
          if (a.dkv_bf16) {
            *reinterpret_cast<uint2*>(dst16 + c * 32 + x) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
            continue;
          }
          float4* d4 = reinterpret_cast<float4*>(dst + c * 32 + x);
          if (kShared && (!kScored || a.add_dkdv)) {   // CTAs of one key tile meet (zeroed)
            red_add_v4(d4, v);
            continue;
          }
          if (!first) {
            const float4 o = *d4;
            v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
          }
          *d4 = v;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int kOps, bool kShared, bool kCap, int kBias>
cudaError_t launch_q128(const TcBwdArgs& a, cudaStream_t st) {
  constexpr int smem = Lay<D>::kAlloc;
  cudaError_t e = cudaFuncSetAttribute(tc_bwd_q128_kernel<D, kOps, kShared, kCap, kBias>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long blocks = (long long)a.n_items * a.Hkv * a.kv_split;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  tc_bwd_q128_kernel<D, kOps, kShared, kCap, kBias><<<(unsigned)blocks, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

}  // namespace cpattn
