// Launchers of attention with modified scores that are not tensor-core kernels:
// the distance tables and the fp32 path.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "scored_plan.h"
#include "tc.h"

namespace cpattn {

// ---- learned bias by bucket <-> table by distance (scored_aux.cu) --------------
// table[h][mid + s] = mul * bias[h][bucket[min(|s|, n_dist - 1)]] for |s| <= mid;
// entries at or below -1e37 become -inf (the key is hidden).
cudaError_t launch_expand_bias(const void* bias, bool bf16, int64_t stride_h, int64_t stride_b,
                               const int32_t* buckets, int n_dist, int H, float mul, float* table,
                               int mid, int pitch, cudaStream_t st);
// dbias[h][b] = sum of dtable[h][t] over the distances of bucket b, in order.
cudaError_t launch_reduce_dbias(const float* dtable, const int32_t* buckets, int n_dist,
                                int n_buckets, int H, void* dbias, bool bf16, cudaStream_t st);
// dst[i] = bf16(src[i]) for three tensors of n[i] elements (multiples of 4).
cudaError_t launch_cast_bf16(const float* const (&src)[3], void* const (&dst)[3],
                             const int64_t (&n)[3], int sms, cudaStream_t st);
// out, lse (and out_lo, nullable) of the rows of cut tiles from their partial
// results po [H][run_rows][d], pl [H][run_rows].
cudaError_t launch_join_parts(const Join* joins, int n_joins, const float* po, const float* pl,
                              int64_t run_rows, int H, int d, int64_t T, void* out, void* out_lo,
                              float* lse, cudaStream_t st);

// ---- f16 operands of short samples' backward (scored_aux.cu, operand_range.cuh) ----
// One block per 64-row tile and KV head; tiles of samples of more than kF16Tokens
// tokens are passed over.  ranges [n_samples][Hkv], zeroed before.
cudaError_t launch_operand_ranges(const Tile32* tiles, int n_tiles, const void* q, const void* k,
                                  const void* v, const void* dout, int H, int Hkv, int d,
                                  OperandRange* ranges, cudaStream_t st);
// Scaled f16 copies of the rows of Q and K whose sample and KV head take f16.
cudaError_t launch_f16_operands(const Tile32* tiles, int n_tiles, const void* q, const void* k,
                                int H, int Hkv, int d, const OperandRange* ranges, void* q16,
                                void* k16, cudaStream_t st);

// ---- fp32 inputs: CUDA cores (attn_f32.cu) ---------------------------------------
struct F32Args {
  const float *q, *k, *v, *dout;       // [T][H or Hkv][d]
  const Tile32* tiles;
  int n_tiles, H, Hkv;
  int64_t T;
  float scale, softcap, inv_cap;       // softcap 0: none
  const float* slopes;                 // nullable [H]
  const float* table;                  // nullable [H][pitch], natural units
  int table_pitch, table_mid, n_dist;
  int splits;                          // blocks that share the tiles one block would walk
  float* out; float* lse;              // forward; splits > 1: partial results [splits][T][H][d],
                                       // [splits][H][T] for the log-sum-exp merge
  const float* lse_in; const float* D; // backward; D [H][pitch_d]
  int64_t pitch_d;
  float *dq, *dk, *dv;
  float* dtable;                       // nullable [H][n_dist]
  bool add_dq, add_dkdv;               // add into zeroed dq / dk and dv instead of storing
};
// Blocks along a walk of up to `walk` tiles: as many as keep the launch within four
// blocks per SM, down to a tile each.  (Forward / backward us with one block per
// walk, two blocks per SM and two tiles each, and this: 768 tokens, 8 heads over 2,
// d = 128: 168 / 1201, 94 / 237, 79 / 191; 273 + 146 tokens, 4 over 2, d = 64: 29 / 70
// and 21 / 46.  Six per SM: 88 / 203 for the former.)
inline int f32_splits(int64_t blocks, int walk, int sms) {
  int64_t s = 4LL * sms / (blocks > 0 ? blocks : 1);
  if (s > walk) s = walk;
  return s < 1 ? 1 : (int)s;
}
cudaError_t launch_f32_fwd(const F32Args& a, int d, cudaStream_t st);
cudaError_t launch_f32_bwd(const F32Args& a, int d, cudaStream_t st);

}  // namespace cpattn
