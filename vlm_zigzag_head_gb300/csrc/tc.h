// Tensor-core (tcgen05 / TMEM / TMA) attention kernels for sm_103a.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "plan.h"

namespace cpattn {

// Softmax scales above this make dQ = scale * dS K large enough that one bf16
// rounding of a probability-sized operand (P in the forward's PV product, dS
// in the backward's dQ and dK products) shows in dQ.  Those products then run
// on f16 operands (three more mantissa bits): P and dS are rounded to f16, and
// the other operand is a per-call f16 copy of V (forward) or of Q and K
// (backward), scaled by a power of two so that its largest magnitude lies in
// [2^14, 2^15).  The scaling is exact; the factors are undone in fp32.
constexpr float kF16OperandScale = 0.25f;
inline bool uses_f16_operands(float scale) { return scale > kF16OperandScale; }

// 3-D tensor map over a 16-bit [rows][H][d] tensor (bf16, or f16 when f16 is
// set), box {64, 1, rows_per_box}, 128-byte swizzle.  Returns false (and a
// message) if encoding fails.
bool make_tmap_thd(CUtensorMap* map, const void* base, int64_t rows, int H, int d,
                   int rows_per_box, const char** err, bool f16 = false);
// 3-D tensor map over an fp32 [rows][H][d] tensor, box {32, 1, box_rows} with
// the 128-byte swizzle (the dQ reduce-add target of the 128-query backward).
bool make_tmap_f32_sw128(CUtensorMap* map, void* base, int64_t rows, int H, int d, int box_rows,
                         const char** err);
// 3-D tensor map over the fp32 planes [2][H][pitch] (lse2, D) of the backward
// preprocess, box {box_rows, 1, 2}; pitch must be a multiple of 4.
bool make_tmap_ld(CUtensorMap* map, const void* base, int64_t pitch, int H, int box_rows,
                  const char** err);

// Scores modified before the softmax (score.cuh).  kBias of the kernels:
enum : int { SCORE_PLAIN = 0, SCORE_SLOPES = 1, SCORE_TABLE = 2 };
struct ScoreArgs {
  float cap_log2, inv_cap_log2;   // softcap * log2(e) and its inverse (kCap)
  // the forward's cap: scores are s (k0 + k1 s^2 + .. + k4 s^8) for |s| <= cap_reach
  float cap_k[5];
  float cap_reach;
  const float* slopes;            // SCORE_SLOPES: [H], natural units
  // SCORE_TABLE: [H][table_pitch] bias * log2(e) by signed distance: entry
  // table_mid + distance, |distance| <= table_mid; constant from n_dist - 1 on
  const float* table;
  int n_dist, table_pitch, table_mid;
  float* dtable;                  // backward: [H][n_dist], sums of dS by |distance|
};
// tanh(z) = z (1 + c1 z^2 + .. + c4 z^8) for |z| <= 0.75, minimax (off by at most
// 6e-7 of the value)
constexpr float kCapPolyRange = 0.75f;
constexpr float kCapPoly[4] = {-0.33329880795843986f, 0.13270406554292946f,
                               -0.050340821426050376f, 0.013161359006389609f};
// Fills cap_k and cap_reach from the caps and the scale.  A coefficient that is no
// normal number is left out, and the reach ends where its term passes 3e-7.
void fill_cap_polynomial(ScoreArgs* s, float scale_log2);
// Entries of the table past +-n_dist: a 128 x 128 tile that holds a distance
// below n_dist spans 254 more, so it reads the table without bounds checks.
constexpr int kTableSlack = 256;

struct TcFwdArgs {
  CUtensorMap tm_q_text, tm_k_text, tm_v_text;  // rank-local (gathered) text rows
  CUtensorMap tm_q_nat, tm_k_nat, tm_v_nat;     // natural order (prefix rows)
  const FwdItem* items;
  const Seg* runs;            // non-null: all ring steps in one launch; item key runs are
                              // runs[run_row0 .. run_row0 + nseg) (no running result)
  const int32_t* units;       // nullable: CTA b walks units[cta_off[b] .. cta_off[b + 1]),
  const int32_t* cta_off;     // entries item + n_items * head (a permutation of all units)
  int n_ctas;                 // grid size when units != null (cta_off has n_ctas + 1 entries);
                              // null units: CTA b walks b, b + grid, ...  (grid chosen here)
  int n_items, H, d;
  int Hkv;                    // KV heads; query head h reads KV head h / (H / Hkv)
  float scale_log2;           // softmax scale * log2(e)
  int f16_pv;                 // PV on f16 operands: P and the scaled copy of V behind
                              // tm_v_*; O is multiplied by op_scales->v_mul
  const OpScales* op_scales;  // device; read when f16_pv
  int pdl;                    // launched as a programmatic dependent of the previous ring step
  float* o_run; float* lse_run; int64_t run_rows;
  void* out; float* lse; int64_t T;
  void* out_lo;               // nullable: bf16 remainder o - bf16(o)
  int32_t* status;            // DevStatus of the workspace
  long long wait_limit;
  int64_t text_rows;          // rows of the rank-local (gathered) tensors (index checks)
  int isolate;                // nonzero: rows past a run's end are cleared before a product
                              // reads them (0 * NaN of a neighbouring sample is NaN)
  ScoreArgs score;            // read by the scored kernels only
};
cudaError_t launch_tc_fwd(const TcFwdArgs& a, cudaStream_t st);

// Largest magnitudes of one sample's rows for one KV head and its query heads (bit
// patterns, which order as integers; all 0 at first).
struct OperandRange {
  uint32_t q, k;        // max |x| over the finite elements
  uint32_t v2, g2;      // largest sum of squares of a row of V and dO
  uint32_t g2_least;    // complement of the least one of a row of dO that is not zero
  uint32_t pad[3];
};
static_assert(sizeof(OperandRange) == 32, "OperandRange layout");

// Operand types of S, dQ and dK (dP and dV: bf16).
enum : int {
  OPS_BF16 = 0,
  OPS_F16 = 1,    // f16 with the factors of op_scales
  OPS_ITEM = 2,   // each item's own choice (operand_range.cuh) from `ranges`
};

struct TcBwdArgs {
  CUtensorMap tm_q, tm_k, tm_v, tm_do;  // natural order (Q, K: the f16 copies when f16)
  CUtensorMap tm_q16, tm_k16;            // f16 copies of the samples that take them (ranges)
  CUtensorMap tm_ld;                     // [2][H][pitch] fp32: lse2, D
  CUtensorMap tm_dq;                     // dq fp32 [T][H][d], box {32, 1, 32}, 128-byte swizzle:
                                         // reduce-add target
  const BwdItem* items;
  const Seg* runs;            // run list of the all-steps plan: item i's query runs are
                              // runs[items[i].run0 .. + nseg)
  int f16;                    // S, dQ and dK on f16 operands (scaled Q, K copies; dS in f16)
  const OpScales* op_scales;  // device; read when f16
  const OperandRange* ranges; // scored kernels, nullable: [n_samples][Hkv], each item's choice
                              // of operand types (item.slot: its sample)
  int n_samples;
  int n_items, H, d;
  int Hkv;                    // KV heads; one CTA per (key tile, KV head) walks its H / Hkv query heads
  float scale, scale_log2;
  int64_t T;
  float* dq; float* dk; float* dv;
  int dkv_bf16;               // dk, dv point to bf16 (scored plans, not add_dkdv)
  float* pre_k; float* pre_v; int64_t pre_rows;
  int32_t* status;
  long long wait_limit;
  int kv_split;               // CTAs sharing one KV head's query heads (divides H / Hkv)
  int add_dkdv;               // several CTAs share a key tile (kv_split > 1, or cut query runs):
                              // dK / dV / prefix slots are reduce-added into zeroed memory
  int isolate;                // as TcFwdArgs::isolate, for query and key rows
  int item_major;             // nonzero: blocks go item by item (all heads of the heaviest
                              // item first), else head by head
  int n_slots;                // prefix-gradient slots (P + 1) behind pre_k / pre_v (index checks)
  ScoreArgs score;            // read by the scored kernels only
};
// The backward (tc_bwd_q128.cuh): one launch over the all-steps plan, every
// item a key tile with the query runs of all ring steps, in 128-query tiles.
cudaError_t launch_tc_bwd_q128(const TcBwdArgs& a, cudaStream_t st);

// With grouped KV heads one CTA walks all G = H / Hkv query heads of its KV
// head.  When that leaves too few CTAs to fill the GPU (under ~4 per SM), the
// group is shared by this many CTAs (a power of two dividing G).
inline int bwd_kv_split(int64_t n_items, int H, int Hkv, int sms) {
  const int G = H / Hkv;
  int split = 1;
  while (G % (2 * split) == 0 && (double)n_items * Hkv * split < 4.0 * sms) split *= 2;
  return split;
}
// The same kernels with modified scores: items carry the distance of their
// first query and key in Seg::rel.  score.cap_log2 > 0: capped.
cudaError_t launch_tc_fwd_scored(const TcFwdArgs& a, int bias, cudaStream_t st);
cudaError_t launch_tc_bwd_scored(const TcBwdArgs& a, int bias, cudaStream_t st);

}  // namespace cpattn
