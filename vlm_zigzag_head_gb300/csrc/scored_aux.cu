// The small kernels around attention with modified scores: the learned bias laid
// out by distance and its gradient summed back (a few KB a head: bound by the
// launch), the join of partial results, the gradients' rounding to bf16, and the
// ranges and f16 copies of short samples (one pass each, bound by memory).
#include <cuda_bf16.h>

#include "operand_range.cuh"
#include "ptx.cuh"
#include "scored.h"

namespace cpattn {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    expand_bias_kernel(const void* bias, int bf16, int64_t sh, int64_t sb, const int32_t* buckets,
                       int n_dist, float mul, float* table, int mid, int pitch) {
  const int h = blockIdx.y;
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < pitch; i += gridDim.x * kThreads) {
    const int s = i - mid;
    const int64_t at = h * sh + buckets[min(s < 0 ? -s : s, n_dist - 1)] * sb;
    const float b = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(bias)[at])
                         : static_cast<const float*>(bias)[at];
    table[(int64_t)h * pitch + i] = b <= -1e37f ? -INFINITY : b * mul;
  }
}

// One block per head, one warp per bucket at a time; lanes take the distances
// 32 apart and meet in a fixed order.
constexpr int kReduceThreads = 1024;
__global__ void __launch_bounds__(kReduceThreads)
    reduce_dbias_kernel(const float* dtable, const int32_t* buckets, int n_dist, int n_buckets,
                        void* dbias, int bf16) {
  const int h = blockIdx.x, lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < n_buckets; b += kReduceThreads / 32) {
    float v = 0.f;
    for (int t = lane; t < n_dist; t += 32)
      if (buckets[t] == b) v += dtable[(int64_t)h * n_dist + t];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane != 0) continue;
    const int64_t at = (int64_t)h * n_buckets + b;
    if (bf16) static_cast<__nv_bfloat16*>(dbias)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(dbias)[at] = v;
  }
}

struct Cast3 {
  const float4* src[3];
  uint2* dst[3];
  int64_t n[3];   // groups of four elements
};

// Block row blockIdx.y: tensor; four elements per thread and step.
__global__ void __launch_bounds__(kThreads) cast_bf16_kernel(const Cast3 c) {
  const int t = blockIdx.y;
  const float4* src = t == 0 ? c.src[0] : t == 1 ? c.src[1] : c.src[2];
  uint2* dst = t == 0 ? c.dst[0] : t == 1 ? c.dst[1] : c.dst[2];
  const int64_t n = t == 0 ? c.n[0] : t == 1 ? c.n[1] : c.n[2];
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreads) {
    const float4 v = src[i];
    dst[i] = make_uint2(ptx::pack_bf16x2(v.x, v.y), ptx::pack_bf16x2(v.z, v.w));
  }
}

// Softmax parts: out = sum_p e^(lse_p - m) out_p / sum_p e^(lse_p - m), m the largest
// lse_p (NaN if one is).  Block (join, piece of its rows, head); D / 4 lanes per row.
constexpr int kJoinRows = 32;
template <int D>
__global__ void __launch_bounds__(kThreads)
    join_parts_kernel(const Join* joins, const float* po, const float* pl, int64_t run_rows, int H,
                      int64_t T, __nv_bfloat16* out, __nv_bfloat16* out_lo, float* lse) {
  constexpr int kLanes = D / 4, kPass = kThreads / kLanes;
  const Join jn = joins[blockIdx.x];
  const int h = blockIdx.z, lane = threadIdx.x % kLanes;
  const int end = min(jn.len, ((int)blockIdx.y + 1) * kJoinRows);
  for (int t = blockIdx.y * kJoinRows + threadIdx.x / kLanes; t < end; t += kPass) {
    const int64_t row0 = h * run_rows + jn.run_row0 + t;
    float m = -INFINITY;
    for (int p = 0; p < jn.parts; ++p) m = ptx::max_nan(m, pl[row0 + (int64_t)p * jn.len]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    if (m != -INFINITY) {
#pragma unroll 4
      for (int p = 0; p < jn.parts; ++p) {
        const int64_t row = row0 + (int64_t)p * jn.len;
        const float w = expf(pl[row] - m);
        const float4 v = *reinterpret_cast<const float4*>(po + row * D + lane * 4);
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
        sum += w;
      }
      const float inv = 1.f / sum;
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    const uint2 hi = make_uint2(ptx::pack_bf16x2(acc.x, acc.y), ptx::pack_bf16x2(acc.z, acc.w));
    const int64_t at = ((jn.out_row0 + t) * (int64_t)H + h) * D + lane * 4;
    *reinterpret_cast<uint2*>(out + at) = hi;
    if (out_lo != nullptr)   // the remainder, itself rounded to bf16
      *reinterpret_cast<uint2*>(out_lo + at) = make_uint2(
          ptx::pack_bf16x2(acc.x - __uint_as_float(hi.x << 16),
                           acc.y - __uint_as_float(hi.x & 0xffff0000u)),
          ptx::pack_bf16x2(acc.z - __uint_as_float(hi.y << 16),
                           acc.w - __uint_as_float(hi.y & 0xffff0000u)));
    if (lane == 0)
      lse[h * T + jn.out_row0 + t] = m == -INFINITY ? -INFINITY : m + logf(sum);
  }
}

// Eight bf16 of one row's piece.
struct Piece {
  uint32_t w[4];
  __device__ __forceinline__ explicit Piece(const __nv_bfloat16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  // bit pattern of the largest finite magnitude, as fp32
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = (w[i] & 0x7fffu) << 16, hi = w[i] & 0x7fff0000u;
      m = max(m, lo < 0x7f800000u ? lo : 0u);
      m = max(m, hi < 0x7f800000u ? hi : 0u);
    }
    return m;
  }
  __device__ __forceinline__ bool any() const {
    return ((w[0] | w[1] | w[2] | w[3]) & 0x7fff7fffu) != 0;
  }
  __device__ __forceinline__ float squares() const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
      s = fmaf(lo, lo, fmaf(hi, hi, s));
    }
    return s;
  }
};

// D / 8 lanes per row; block: a tile's rows for one KV head.
template <int D>
__global__ void __launch_bounds__(kThreads)
    operand_range_kernel(const Tile32* tiles, const __nv_bfloat16* q, const __nv_bfloat16* k,
                         const __nv_bfloat16* v, const __nv_bfloat16* dout, int H, int Hkv,
                         OperandRange* ranges) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  const Tile32 tl = tiles[blockIdx.x];
  if (tl.seq_len > kF16Tokens) return;
  const int hk = blockIdx.y, G = H / Hkv;
  const int e = threadIdx.x % kLanes * 8, r0 = threadIdx.x / kLanes;
  // the row's sum of squares in all its lanes; rows that are not there count as zero
  auto row_squares = [&](const Piece& p, bool there, bool& any) {
    float s = there ? p.squares() : 0.f;
    int a = there && p.any();
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      a |= __shfl_xor_sync(0xffffffffu, a, o);
    }
    any = a != 0;
    return s;
  };
  uint32_t m[5] = {0, 0, 0, 0, 0};   // q, k, v2, g2, g2_least
  bool any;
  for (int base = 0; base < tl.len; base += kRows) {
    const bool there = base + r0 < tl.len;
    const int64_t at = ((int64_t)(tl.row0 + min(base + r0, tl.len - 1)) * Hkv + hk) * D + e;
    if (there) m[1] = max(m[1], Piece(k + at).largest());
    m[2] = max(m[2], __float_as_uint(row_squares(Piece(v + at), there, any)));
  }
  const int rows = tl.len * G;   // (token, query head) pairs
  for (int base = 0; base < rows; base += kRows) {
    const int x = min(base + r0, rows - 1);
    const bool there = base + r0 < rows;
    const int64_t at = ((int64_t)(tl.row0 + x / G) * H + hk * G + x % G) * D + e;
    if (there) m[0] = max(m[0], Piece(q + at).largest());
    const float s = row_squares(Piece(dout + at), there, any);
    m[3] = max(m[3], __float_as_uint(s));
    // a row whose squares underflow is not zero: it counts as the smallest number
    if (any) m[4] = max(m[4], ~__float_as_uint(fmaxf(s, 1e-38f)));
  }
  __shared__ uint32_t part[kThreads / 32][5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    m[i] = __reduce_max_sync(0xffffffffu, m[i]);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][i] = m[i];
  }
  __syncthreads();
  if (threadIdx.x >= 5) return;
  uint32_t top = 0;
  for (int w = 0; w < kThreads / 32; ++w) top = max(top, part[w][threadIdx.x]);
  // the fields q, k, v2, g2, g2_least lie in this order
  uint32_t* dst = &ranges[(int64_t)tl.sample * Hkv + hk].q + threadIdx.x;
  if (top != 0) atomicMax(dst, top);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    f16_operands_kernel(const Tile32* tiles, const __nv_bfloat16* q, const __nv_bfloat16* k, int H,
                        int Hkv, const OperandRange* ranges, uint4* q16, uint4* k16) {
  constexpr int kPieces = D / 8;
  const Tile32 tl = tiles[blockIdx.x];
  if (tl.seq_len > kF16Tokens) return;
  const int hk = blockIdx.y, G = H / Hkv;
  const Operands ops = choose_operands(ranges[(int64_t)tl.sample * Hkv + hk]);
  if (!ops.f16) return;
  auto copy = [](const __nv_bfloat16* src, uint4* dst, int64_t piece, float f) {
    const Piece p(src + piece * 8);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = ptx::pack_f16x2(__uint_as_float(p.w[i] << 16) * f,
                             __uint_as_float(p.w[i] & 0xffff0000u) * f);
    dst[piece] = make_uint4(o[0], o[1], o[2], o[3]);
  };
  const float fq = range_pow2(-ops.eq), fk = range_pow2(-ops.ek);
  for (int i = threadIdx.x; i < tl.len * G * kPieces; i += kThreads) {
    const int x = i / kPieces;
    copy(q, q16, ((int64_t)(tl.row0 + x / G) * H + hk * G + x % G) * kPieces + i % kPieces, fq);
  }
  for (int i = threadIdx.x; i < tl.len * kPieces; i += kThreads)
    copy(k, k16, ((int64_t)(tl.row0 + i / kPieces) * Hkv + hk) * kPieces + i % kPieces, fk);
}

}  // namespace

cudaError_t launch_operand_ranges(const Tile32* tiles, int n_tiles, const void* q, const void* k,
                                  const void* v, const void* dout, int H, int Hkv, int d,
                                  OperandRange* ranges, cudaStream_t st) {
  const auto* qb = static_cast<const __nv_bfloat16*>(q);
  const auto* kb = static_cast<const __nv_bfloat16*>(k);
  const auto* vb = static_cast<const __nv_bfloat16*>(v);
  const auto* gb = static_cast<const __nv_bfloat16*>(dout);
  const dim3 grid(n_tiles, Hkv);
  if (d == 64)
    operand_range_kernel<64><<<grid, kThreads, 0, st>>>(tiles, qb, kb, vb, gb, H, Hkv, ranges);
  else
    operand_range_kernel<128><<<grid, kThreads, 0, st>>>(tiles, qb, kb, vb, gb, H, Hkv, ranges);
  return cudaGetLastError();
}

cudaError_t launch_f16_operands(const Tile32* tiles, int n_tiles, const void* q, const void* k,
                                int H, int Hkv, int d, const OperandRange* ranges, void* q16,
                                void* k16, cudaStream_t st) {
  const auto* qb = static_cast<const __nv_bfloat16*>(q);
  const auto* kb = static_cast<const __nv_bfloat16*>(k);
  auto* qo = static_cast<uint4*>(q16);
  auto* ko = static_cast<uint4*>(k16);
  const dim3 grid(n_tiles, Hkv);
  if (d == 64)
    f16_operands_kernel<64><<<grid, kThreads, 0, st>>>(tiles, qb, kb, H, Hkv, ranges, qo, ko);
  else
    f16_operands_kernel<128><<<grid, kThreads, 0, st>>>(tiles, qb, kb, H, Hkv, ranges, qo, ko);
  return cudaGetLastError();
}

cudaError_t launch_join_parts(const Join* joins, int n_joins, const float* po, const float* pl,
                              int64_t run_rows, int H, int d, int64_t T, void* out, void* out_lo,
                              float* lse, cudaStream_t st) {
  const dim3 grid(n_joins, kFwdPairQ / kJoinRows, H);
  auto* o = static_cast<__nv_bfloat16*>(out);
  auto* lo = static_cast<__nv_bfloat16*>(out_lo);
  if (d == 64)
    join_parts_kernel<64><<<grid, kThreads, 0, st>>>(joins, po, pl, run_rows, H, T, o, lo, lse);
  else
    join_parts_kernel<128><<<grid, kThreads, 0, st>>>(joins, po, pl, run_rows, H, T, o, lo, lse);
  return cudaGetLastError();
}

cudaError_t launch_cast_bf16(const float* const (&src)[3], void* const (&dst)[3],
                             const int64_t (&n)[3], int sms, cudaStream_t st) {
  Cast3 c;
  int64_t most = 0;
  for (int i = 0; i < 3; ++i) {
    c.src[i] = reinterpret_cast<const float4*>(src[i]);
    c.dst[i] = static_cast<uint2*>(dst[i]);
    c.n[i] = n[i] / 4;
    most = c.n[i] > most ? c.n[i] : most;
  }
  const int64_t want = (most + 4 * kThreads - 1) / (4 * kThreads), cap = 8LL * sms;
  const unsigned blocks = (unsigned)(want < 1 ? 1 : want < cap ? want : cap);
  cast_bf16_kernel<<<dim3(blocks, n[1] > 0 || n[2] > 0 ? 3 : 1), kThreads, 0, st>>>(c);
  return cudaGetLastError();
}

cudaError_t launch_expand_bias(const void* bias, bool bf16, int64_t stride_h, int64_t stride_b,
                               const int32_t* buckets, int n_dist, int H, float mul, float* table,
                               int mid, int pitch, cudaStream_t st) {
  expand_bias_kernel<<<dim3((pitch + kThreads - 1) / kThreads, H), kThreads, 0, st>>>(
      bias, bf16 ? 1 : 0, stride_h, stride_b, buckets, n_dist, mul, table, mid, pitch);
  return cudaGetLastError();
}

cudaError_t launch_reduce_dbias(const float* dtable, const int32_t* buckets, int n_dist,
                                int n_buckets, int H, void* dbias, bool bf16, cudaStream_t st) {
  reduce_dbias_kernel<<<H, kReduceThreads, 0, st>>>(dtable, buckets, n_dist, n_buckets, dbias,
                                              bf16 ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace cpattn
