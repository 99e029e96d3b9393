// Gated feed-forward block: its matrix products (tensor cores for bf16, CUDA cores
// for fp32) and the passes between them (kernel launchers).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace cpattn {

enum : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// 2-D tensor map over a bf16 [rows][cols] matrix with a row stride in elements (a
// multiple of 8), box {64, box_rows}, 128-byte swizzle.
bool make_tmap_matrix(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                      int64_t stride, int box_rows, const char** err);

constexpr int kGemmM = 128, kGemmN = 256, kGemmK = 64;   // tile

// What becomes of a tile of products.
enum : int {
  GEMM_STORE = 0,   // out = A B^T
  GEMM_GLU = 1,     // two products, gate and up: out = act(gate) up (and both kept)
  GEMM_DGLU = 2,    // dh = A B^T: dgate, dup and h from the kept gate and up
};

// C[M][N] = sum over k of A(m, k) B(n, k).  A tile of either operand is loaded from
// memory where k runs along a row (K-major) or where m (n) does (MN-major).
struct GemmArgs {
  CUtensorMap a[2], b[2];
  int M, N;            // of one output
  int m_tiles, n_tiles;
  int m_split;         // m tiles from here on: a[1], out[1] (m_tiles: none)
  int k_tiles;         // all k tiles
  int k_split;         // k tiles from here on: a[1], b[1] (k_tiles: none)
  int splits;          // > 1: that many units share a tile's k; sums go to `partial`
  float* partial;      // [splits][M][N], once for each output (GEMM_GLU: gate, up)
  void* out[2];        // row stride N
  int out_f32;
  int act;
  void* gate;          // [M][N]; GEMM_GLU: written (nullable), GEMM_DGLU: read
  void* up;
  void* dgate;         // GEMM_DGLU: written; h goes to out[0]
  void* dup;
  int32_t* status;
  long long wait_limit;
};
// a_mn, b_mn: the operand is MN-major (GEMM_GLU: neither; GEMM_DGLU: B alone).
cudaError_t launch_gemm_bf16(const GemmArgs& g, int epilogue, bool a_mn, bool b_mn, int sms,
                             cudaStream_t st);

// The sums of the shares of a product, and what its epilogue would have done.
struct JoinArgs {
  const float* partial;   // [splits][n]; gate and up: [2][splits][n]
  int splits;
  int64_t n;              // elements of the output
  void* out;              // sum; act(gate) up; h
  int act;
  void* gate;             // as GemmArgs
  void* up;
  void* dgate;
  void* dup;
};
// bf16: out, gate, up, dgate, dup are bf16 (else fp32).
cudaError_t launch_ffn_join(const JoinArgs& j, int epilogue, bool bf16, cudaStream_t st);

// fp32 products on CUDA cores: partial[split][m][n] = sum over the split's k of
// A(m, k) B(n, k), an element of A at m * sam + k * sak (one of the strides is 1).
struct GemmF32Args {
  const float *a, *b;
  int64_t sam, sak, sbn, sbk;
  int M, N, K;
  int splits;
  int accumulate;      // add to what is there (splits == 1)
  float* out;          // [splits][M][N]
};
cudaError_t launch_gemm_f32(const GemmF32Args& g, cudaStream_t st);

}  // namespace cpattn
