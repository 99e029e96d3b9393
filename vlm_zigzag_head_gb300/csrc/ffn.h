// Gated feed-forward block: its matrix products (on tensor cores; fp32 ones of up to
// kSimtRows rows on CUDA cores) and the passes between them (kernel launchers).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace cpattn {

enum : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// 2-D tensor map over an [rows][cols] matrix of elements of 1, 2 (bf16) or 4 (fp32)
// bytes with a row stride in elements (whole 16-byte pieces), box rows of 64 or 128
// bytes in the swizzle of that size.
bool make_tmap_matrix(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                      int64_t stride, int elem, int box_cols, int box_rows, const char** err);
bool make_tmap_planes(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                      int box_rows, const char** err);

// The projections kept for a bf16 backward are the upper 24 bits of their fp32 values:
// a plane [M][N] of upper halves (bf16, cut off), then a plane of the bytes below them,
// row pitch kept_pitch(N).  With bf16 alone their rounding passes into every gradient
// (dw_down off by 3.5e-3 in relative L2; 2.4e-3 so, 1.7e-3 its own rounding).
inline __host__ __device__ int64_t kept_pitch(int64_t N) { return (N + 15) / 16 * 16; }
inline __host__ __device__ int64_t kept_low(int64_t M, int64_t N) { return M * N * 2; }  // bytes
inline int64_t kept_bytes(int64_t M, int64_t N) { return kept_low(M, N) + M * kept_pitch(N); }

// Tile of a CTA pair (kGemmM x tile_n, 256 or 128) and k step; an epilogue moves boxes of
// 32 rows and 64 columns (fp32: 32).
constexpr int kGemmM = 256, kGemmK = 64;

// What becomes of a tile of products.
enum : int {
  GEMM_STORE = 0,   // out = A B^T
  GEMM_GLU = 1,     // two products, gate and up, tile_n / 2 columns of each: out = act(gate)
                    // up (and both kept)
  GEMM_DGLU = 2,    // dh = A B^T: dgate, dup and h from the kept gate and up
};

enum : int { FOLLOWS_NONE = 0, FOLLOWS_A = 1, FOLLOWS_BOTH = 2 };

// C[M][N] = sum over k of A(m, k) B(n, k).  A tile of either operand is loaded from
// memory where k runs along a row (K-major) or where m (n) does (MN-major).
struct GemmTiles {
  int a_mn, b_mn;      // MN-major (GEMM_GLU: neither; GEMM_DGLU: B alone)
  int M, N;            // of one output
  int m_tiles, n_tiles;
  int m_split;         // m tiles from here on: a[1], out[1] (m_tiles: none)
  int k_tiles;         // all k tiles
  int k_split;         // k tiles from here on: a[1], b[1] (k_tiles: none)
  int first;           // number of its first unit in the launch
  int whole;           // tiles of one unit; each tile after them is `shares` units,
  int shares;          // which share its k and leave their sums in `partial`; the last
                       // to finish adds them in order and goes on with the epilogue
  int first_slot, first_ticket;   // of its shared tiles
};
struct GemmProblem : GemmTiles {
  CUtensorMap a[2], b[2];      // box {64, 128} (b: {64, tile_n / 2}) K-major, {64, 64} MN-major
  CUtensorMap out[2];          // box {64, 32} bf16, {32, 32} fp32
  int out_f32;
};
constexpr int kGemmProblems = 3;
constexpr int kTickets = 16;   // of a tile (bf16 products: 8 of them)
struct GemmArgs {
  GemmProblem p[kGemmProblems];   // GEMM_STORE: one to three, their units one after another
  int problems;
  int units;           // of all problems, below 2^30
  CUtensorMap gate[2], up[2];  // the kept planes, box {64, 32}
  CUtensorMap dgate, dup;      // GEMM_DGLU: written; h goes to out[0]
  float* partial;      // [slot][tile_n / 4][256][4]: columns 4 c .. 4 c + 3
  int32_t* tickets;    // [shared tile][kTickets]: shares finished; zero before and after
  int follows;         // the launch before is of the same call: this one may start while
                       // it ends (FOLLOWS_A: its weights, B, do not come from there)
  int clear;           // words from `status` on, cleared at the start (no shared tiles)
  int act;
  int keep;            // GEMM_GLU: write gate and up
  int32_t* status;
  long long wait_limit;
};
cudaError_t launch_gemm_bf16(const GemmArgs& g, int epilogue, int tile_n, int sms,
                             cudaStream_t st);

// The same for fp32 operands, each as three bf16 planes that add up to it (24 bits):
// hi, mid, lo, one behind another, rows contiguous.  Tiles of kGemmM x kSplitN.
constexpr int kSplitN = 128;
struct SplitProblem : GemmTiles {
  CUtensorMap a[2], b[2];      // {cols, rows, plane}, boxes as above (tile_n = kSplitN), one plane
  float* out[2];               // GEMM_STORE
};
struct SplitArgs {
  SplitProblem p[kGemmProblems];
  int problems, units;
  float *gate, *up;            // [M][N]: written (GEMM_GLU, nullable), read (GEMM_DGLU)
  __nv_bfloat16 *h, *dgate, *dup;   // planes [3][M][N]
  float* partial;              // as above
  int32_t* tickets;
  int act;
  int32_t* status;
  long long wait_limit;
};
constexpr int kSimtRows = 64;   // of calls that stay on CUDA cores
// Follows the launch before it on the stream, which must be of the same call.
cudaError_t launch_gemm_split(const SplitArgs& g, int epilogue, int sms, cudaStream_t st);

// Planes of up to five fp32 matrices; clears `clear` words from `status` on.
struct SplitPass {
  struct {
    const float* src;
    __nv_bfloat16* planes;
    int64_t rows, stride;
    int cols;                  // a multiple of 8
  } m[5];
  int n;
  int32_t* status;
  int clear;
};
cudaError_t launch_split(const SplitPass& s, cudaStream_t st);

// How a launch's products are cut into units: the last tiles, too few for all pairs of
// CTAs at once, along k where that saves time.
struct GemmCut {
  int64_t tiles;
  int k_tiles;
  int64_t whole;
  int shares;
};
// About the microseconds that a pair takes for a k tile and for the last tile's epilogue,
// and the fewest k tiles of a share.
struct GemmCost {
  int tile_n;
  double step, epilogue;
  int least_k;
};
GemmCost gemm_cost(int epilogue, int tile_n);
GemmCost split_cost(int epilogue);
// Sets whole and shares, the products in the order of the launch; returns about the
// microseconds that the launch takes.
double cut_products(GemmCut* p, int n, int pairs, const GemmCost& cost);
inline size_t partial_bytes(const GemmCut& p, int tile_n) {
  return p.shares < 2 ? 0
                      : (size_t)(p.tiles - p.whole) * p.shares * kGemmM * tile_n * sizeof(float);
}

// More rows than that (T <= kBatchRows): the same two forms, with tensor maps of the
// operands, box {64, 128} of the weights (one in the second form), {64, tokens} of x.
constexpr int kBatchRows = 128;
struct FfnTokensArgs {
  CUtensorMap w[2], x;
  void* out;
  void* gate;                // kept planes (nullable)
  void* up;
  int T, N, K;
  int tokens;                // T, rounded up to 16, 32, 48, 64, 96 or 128
  int act;
  int32_t* status;
  long long wait_limit;
};
cudaError_t launch_ffn_tokens(const FfnTokensArgs& a, bool glu, int sms, cudaStream_t st);

// fp32: the sums of the shares of a product (partial [splits][M][N]; gate and up:
// [2][splits][M][N]) and what its epilogue does.  All arrays [M][N] fp32.
struct F32JoinArgs {
  const float* partial;
  int splits;
  int64_t n;           // M N
  float* out;          // sum; act(gate) up; h
  int act;
  float* gate;         // GEMM_GLU: written (nullable), GEMM_DGLU: read
  float* up;
  float* dgate;
  float* dup;
};
cudaError_t launch_f32_join(const F32JoinArgs& j, int epilogue, cudaStream_t st);

// Few rows (T <= kFewRows): out [T][N] = act(x w0^T) (x w1^T), or x w0^T with the two
// halves of each 32 rows of one weight as w0 and w1.  The second form may start while
// the launch before it, which writes x, still runs.
constexpr int kFewRows = 8;
struct FfnRowsArgs {
  const void* x;             // [T][K] bf16
  int64_t x_stride;
  const void* w[2];          // [N][K] bf16
  int64_t w_stride[2];
  void* out;
  void* gate;                // kept planes (nullable)
  void* up;
  int T, N, K;
  int act;
  int32_t* status;           // cleared by the first form
};
cudaError_t launch_ffn_rows(const FfnRowsArgs& a, bool glu, int sms, cudaStream_t st);
// The same in fp32 (x, weights, out, gate and up), T <= kFewRowsF32; no second weight in
// the second form.
constexpr int kFewRowsF32 = 24;
cudaError_t launch_ffn_rows_f32(const FfnRowsArgs& a, bool glu, int sms, cudaStream_t st);

// fp32 products on CUDA cores: out[o][share][m][n] = sum over the share's k of
// A(m, k) B(n, k), an element of A at m * sam + k * sak (one of the strides is 1, the
// other a multiple of 4, pointers 16-byte aligned).  Two outputs have operands of their
// own; with two phases k runs through a[0], b[0] and then a[1], b[1].
struct GemmF32Args {
  const float *a[2], *b[2];
  int64_t sam, sak;
  int64_t sbn[2], sbk[2];   // of b[0], b[1]
  int M, N, K;
  int outputs, phases;   // 1 or 2; not both 2
  int splits;
  float* out[2];         // [splits][M][N]
};
cudaError_t launch_gemm_f32(const GemmF32Args& g, cudaStream_t st);
// Shares of k that fill the GPU.
int share_f32(int64_t M, int64_t N, int64_t K, int outputs, int phases, int sms);

}  // namespace cpattn
