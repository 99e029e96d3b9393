// C ABI of the gated feed-forward block: argument checks, work split and the launch
// sequence.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "../../include/cpattn.h"
#include "entry.h"
#include "ffn.h"

using namespace cpattn;

namespace {

constexpr int kMaxWidth = 1 << 20;

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
inline int tiles(int64_t n, int tile) { return (int)((n + tile - 1) / tile); }

cp_status_t check_desc(const cp_gated_ffn_t* p) {
  if (!p) return entry_fail(CP_ERR_INVALID_ARG, "desc is NULL");
  if (p->dtype != CP_F32 && p->dtype != CP_BF16)
    return entry_fail(CP_ERR_DTYPE, "dtype must be CP_F32 or CP_BF16");
  if (p->grad_dtype != CP_F32 && !(p->grad_dtype == CP_BF16 && p->dtype == CP_BF16))
    return entry_fail(CP_ERR_DTYPE, "grad_dtype must be CP_F32, or CP_BF16 with bf16 inputs");
  if (p->activation < CP_ACT_SILU || p->activation > CP_ACT_GELU_TANH)
    return entry_fail(CP_ERR_INVALID_ARG, "unknown activation");
  if (p->T < 0) return entry_fail(CP_ERR_INVALID_ARG, "T >= 0");
  for (int n : {p->D, p->F, p->D_out})
    if (n < 8 || n > kMaxWidth || n % 8 != 0)
      return entry_fail(CP_ERR_SHAPE, "D, F and D_out must be multiples of 8 in [8, 2^20]");
  const int per16 = p->dtype == CP_BF16 ? 8 : 4;
  const struct { int64_t stride, rows, width; } m[5] = {
      {p->x_stride, p->T, p->D},         {p->w_gate_stride, p->F, p->D},
      {p->w_up_stride, p->F, p->D},      {p->w_down_stride, p->D_out, p->F},
      {p->dy_stride, p->T, p->D_out}};
  for (int i = 0; i < 5; ++i) {
    if (m[i].rows <= 1) continue;   // never used
    if (m[i].stride < m[i].width)
      return entry_fail(CP_ERR_SHAPE, "rows must not overlap");
    if (m[i].stride % per16 != 0)
      return entry_fail(CP_ERR_ALIGNMENT, "row strides must be whole 16-byte pieces");
    if (m[i].stride >= (int64_t)1 << 36)
      return entry_fail(CP_ERR_SHAPE, "a row stride is too large");
  }
  return CP_OK;
}

// 16-byte aligned and not NULL.
cp_status_t check_ptr(const void* p, const char* name) {
  if (!p) return entry_fail(CP_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (!aligned_to(p, 16))
    return entry_fail(CP_ERR_ALIGNMENT, std::string(name) + " must be 16-byte aligned");
  return CP_OK;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Forward calls that the kernels for few rows take, and for a batch of them.
bool few_rows(const cp_gated_ffn_t* p) { return p->dtype == CP_BF16 && p->T <= kFewRows; }
bool batch_rows(const cp_gated_ffn_t* p) {
  return p->dtype == CP_BF16 && p->T > kFewRows && p->T <= kBatchRows;
}

// How the bf16 products' last tiles and the fp32 products' k are shared, and what of
// the workspace that takes.
struct Share {
  int whole, shares;   // fp32: the tile, and the shares
};
struct Plan {
  int sms = 0;
  Share gate_up, down, dh, d_down, d_in, d_both, dx;   // d_in: one weight, d_both: both
  size_t fwd_partial = 0, bwd_partial = 0;   // bytes
};

Plan make_plan(const cp_gated_ffn_t* p, int sms) {
  Plan r;
  r.sms = sms;
  if (sms < 2) return r;
  const int64_t T = p->T, D = p->D, F = p->F, O = p->D_out;
  if (p->dtype == CP_BF16) {
    auto share = [&](int64_t M, int64_t N, int tile_n, int k_tiles, int outputs, size_t* most) {
      const int64_t n = (int64_t)outputs * tiles(M, kGemmM) * tiles(N, tile_n);
      Share s;
      share_tail(n, k_tiles, sms / 2, &s.whole, &s.shares);
      *most = std::max(*most, s.shares > 1 ? partial_bytes(n, s.whole, s.shares) : 0);
      return s;
    };
    r.gate_up = share(T, F, kGemmN / 2, tiles(D, kGemmK), 1, &r.fwd_partial);
    r.down = share(T, O, kGemmN, tiles(F, kGemmK), 1, &r.fwd_partial);
    r.dh = share(T, F, kGemmN, tiles(O, kGemmK), 1, &r.bwd_partial);
    r.dx = share(T, D, kGemmN, 2 * tiles(F, kGemmK), 1, &r.bwd_partial);
    r.d_down = share(O, F, kGemmN, tiles(T, kGemmK), 1, &r.bwd_partial);
    r.d_in = share(F, D, kGemmN, tiles(T, kGemmK), 1, &r.bwd_partial);
    r.d_both = share(F, D, kGemmN, tiles(T, kGemmK), 2, &r.bwd_partial);
    return r;
  }
  // gate and up always go through the workspace, and so does dh
  auto share = [&](int64_t M, int64_t N, int64_t K, int outputs, int phases, bool always,
                   size_t* most) {
    Share s;
    share_f32(M, N, K, outputs, phases, sms, &s.whole, &s.shares);
    if (always || s.shares > 1) *most = std::max(*most, (size_t)outputs * s.shares * M * N * 4);
    return s;
  };
  r.gate_up = share(T, F, D, 2, 1, true, &r.fwd_partial);
  r.down = share(T, O, F, 1, 1, false, &r.fwd_partial);
  r.dh = share(T, F, O, 1, 1, true, &r.bwd_partial);
  r.dx = share(T, D, F, 1, 2, false, &r.bwd_partial);
  r.d_down = share(O, F, T, 1, 1, false, &r.bwd_partial);
  r.d_in = share(F, D, T, 1, 1, false, &r.bwd_partial);
  r.d_both = share(F, D, T, 2, 1, false, &r.bwd_partial);
  return r;
}

// At the start of a workspace, cleared by every call: the status word, and the tickets
// of shared tiles (fewer than there are pairs of CTAs, eight each).
constexpr size_t kTicketsAt = 256;
size_t header_bytes(const Plan& plan) { return kTicketsAt + up256((size_t)plan.sms / 2 * 8 * 4); }

size_t hidden_bytes(const cp_gated_ffn_t* p) {
  return up256((size_t)p->T * p->F * (p->dtype == CP_BF16 ? 2 : 4));
}

size_t fwd_bytes(const cp_gated_ffn_t* p, const Plan& plan) {
  return header_bytes(plan) + hidden_bytes(p) + up256(plan.fwd_partial);
}
size_t bwd_bytes(const cp_gated_ffn_t* p, const Plan& plan) {
  return header_bytes(plan) + 3 * hidden_bytes(p) + up256(plan.bwd_partial);
}

cp_status_t check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws) return entry_fail(CP_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned_to(ws, 256))
    return entry_fail(CP_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  if (have < need)
    return entry_fail(CP_ERR_WORKSPACE, "workspace smaller than cp_gated_ffn_*_workspace_size()");
  return CP_OK;
}

// One operand of a bf16 product: an [rows][cols] matrix in memory.
struct Matrix {
  const void* p;
  int64_t rows, cols, stride;
};

bool make_map(CUtensorMap* m, const Matrix& x, int elem, int cols, int rows, const char** err) {
  // a single row's stride is never used, but has to be whole 16-byte pieces
  const int64_t stride = x.rows > 1 ? x.stride : (x.cols + 15) / 16 * 16;
  return make_tmap_matrix(m, x.p, x.rows, x.cols, stride, elem, cols, rows, err);
}

// A product under construction; failures stick.
struct Product {
  GemmArgs g = {};
  int epilogue;
  bool a_mn, b_mn;
  const char* err = nullptr;

  Product(int epi, bool amn, bool bmn, int M, int N, Share s, int follows, uint8_t* ws,
          void* partial)
      : epilogue(epi), a_mn(amn), b_mn(bmn) {
    g.M = M;
    g.N = N;
    g.m_tiles = g.m_split = tiles(M, kGemmM);
    g.n_tiles = tiles(N, epi == GEMM_GLU ? kGemmN / 2 : kGemmN);
    g.whole = s.whole;
    g.shares = s.shares;
    g.partial = static_cast<float*>(partial);
    g.follows = follows;
    g.status = reinterpret_cast<int32_t*>(ws);
    g.tickets = reinterpret_cast<int32_t*>(ws + kTicketsAt);
    g.wait_limit = device_wait_limit();
  }
  void map(CUtensorMap* m, const Matrix& x, int elem, int cols, int rows) {
    const char* e = nullptr;
    if (!make_map(m, x, elem, cols, rows, &e) && !err) err = e;
  }
  void a(int i, const Matrix& m) { map(&g.a[i], m, 2, kGemmK, a_mn ? 64 : kGemmM / 2); }
  void b(int i, const Matrix& m) { map(&g.b[i], m, 2, kGemmK, b_mn ? 64 : kGemmN / 2); }
  void k(int64_t K, int phases = 1) {
    g.k_split = tiles(K, kGemmK);
    g.k_tiles = phases * g.k_split;
  }
  void box(CUtensorMap* m, void* p, int elem, int64_t stride) {   // what an epilogue moves
    map(m, {p, g.M, g.N, stride}, elem, elem == 4 ? 32 : 64, 32);
  }
  void out(int i, void* p, bool f32 = false) {
    g.out_f32 = f32;
    box(&g.out[i], p, f32 ? 4 : 2, g.N);
  }
  void kept(void* gate, void* up) {
    g.keep = gate != nullptr;
    if (!gate) return;
    for (int i = 0; i < 2; ++i) {
      uint8_t* p = static_cast<uint8_t*>(i ? up : gate);
      CUtensorMap* m = i ? g.up : g.gate;
      box(&m[0], p, 2, g.N);
      map(&m[1], {p + kept_low(g.M, g.N), g.M, g.N, kept_pitch(g.N)}, 1, 64, 32);
    }
  }
  void gradients(void* dgate, void* dup) {
    box(&g.dgate, dgate, 2, g.N);
    box(&g.dup, dup, 2, g.N);
  }

  cp_status_t run(const Plan& plan, cudaStream_t st, const char* what) {
    if (err) return entry_fail(CP_ERR_CUDA, std::string(what) + ": " + err);
    ENTRY_CUDA(launch_gemm_bf16(g, epilogue, a_mn, b_mn, plan.sms, st), what);
    return CP_OK;
  }
};

cp_status_t fwd_rows(const cp_gated_ffn_t* p, const Plan& plan, const void* x, const void* wg,
                     const void* wu, const void* wd, void* y, void* gate, void* up, uint8_t* ws,
                     cudaStream_t st) {
  FfnRowsArgs a = {};
  a.x = x;
  a.x_stride = p->x_stride;
  a.w[0] = wg;
  a.w[1] = wu;
  a.w_stride[0] = p->w_gate_stride;
  a.w_stride[1] = p->w_up_stride;
  a.out = ws + header_bytes(plan);
  a.gate = gate;
  a.up = up;
  a.T = p->T;
  a.N = p->F;
  a.K = p->D;
  a.act = p->activation;
  a.status = reinterpret_cast<int32_t*>(ws);
  ENTRY_CUDA(launch_ffn_rows(a, true, plan.sms, st), "gate and up projections");
  a.x = a.out;
  a.x_stride = p->F;
  a.w[0] = a.w[1] = wd;
  a.w_stride[0] = a.w_stride[1] = p->w_down_stride;
  a.out = y;
  a.N = p->D_out;
  a.K = p->F;
  ENTRY_CUDA(launch_ffn_rows(a, false, plan.sms, st), "down projection");
  return CP_OK;
}

cp_status_t fwd_tokens(const cp_gated_ffn_t* p, const Plan& plan, const void* x, const void* wg,
                       const void* wu, const void* wd, void* y, void* gate, void* up, uint8_t* ws,
                       cudaStream_t st) {
  const int T = p->T, D = p->D, F = p->F, O = p->D_out;
  FfnTokensArgs a = {};
  a.gate = gate;
  a.up = up;
  a.T = T;
  a.tokens = T <= 64 ? (T + 15) / 16 * 16 : (T + 31) / 32 * 32;
  a.act = p->activation;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.wait_limit = device_wait_limit();
  void* h = ws + header_bytes(plan);
  const char* err = nullptr;
  if (!make_map(&a.w[0], {wg, F, D, p->w_gate_stride}, 2, kGemmK, 128, &err) ||
      !make_map(&a.w[1], {wu, F, D, p->w_up_stride}, 2, kGemmK, 128, &err) ||
      !make_map(&a.x, {x, T, D, p->x_stride}, 2, kGemmK, a.tokens, &err))
    return entry_fail(CP_ERR_CUDA, std::string("gate and up projections: ") + err);
  a.out = h;
  a.N = F;
  a.K = D;
  ENTRY_CUDA(launch_ffn_tokens(a, true, plan.sms, st), "gate and up projections");
  if (!make_map(&a.w[0], {wd, O, F, p->w_down_stride}, 2, kGemmK, 128, &err) ||
      !make_map(&a.x, {h, T, F, F}, 2, kGemmK, a.tokens, &err))
    return entry_fail(CP_ERR_CUDA, std::string("down projection: ") + err);
  a.out = y;
  a.N = O;
  a.K = F;
  ENTRY_CUDA(launch_ffn_tokens(a, false, plan.sms, st), "down projection");
  return CP_OK;
}

cp_status_t fwd_bf16(const cp_gated_ffn_t* p, const Plan& plan, const void* x, const void* wg,
                     const void* wu, const void* wd, void* y, void* gate, void* up, uint8_t* ws,
                     cudaStream_t st) {
  void* h = ws + header_bytes(plan);
  void* partial = ws + header_bytes(plan) + hidden_bytes(p);
  const int T = p->T, D = p->D, F = p->F, O = p->D_out;
  cp_status_t e;
  Product gu(GEMM_GLU, false, false, T, F, plan.gate_up, FOLLOWS_NONE, ws, partial);
  gu.a(0, {x, T, D, p->x_stride});
  gu.b(0, {wg, F, D, p->w_gate_stride});
  gu.b(1, {wu, F, D, p->w_up_stride});
  gu.k(D);
  gu.out(0, h);
  gu.g.act = p->activation;
  gu.kept(gate, up);
  if ((e = gu.run(plan, st, "gate and up projections")) != CP_OK) return e;
  Product down(GEMM_STORE, false, false, T, O, plan.down, FOLLOWS_A, ws, partial);
  down.a(0, {h, T, F, F});
  down.b(0, {wd, O, F, p->w_down_stride});
  down.k(F);
  down.out(0, y);
  return down.run(plan, st, "down projection");
}

cp_status_t bwd_bf16(const cp_gated_ffn_t* p, const Plan& plan, const void* x, const void* wg,
                     const void* wu, const void* wd, const void* gate, const void* up,
                     const void* dy, void* dx, void* dwg, void* dwu, void* dwd, uint8_t* ws,
                     cudaStream_t st) {
  uint8_t* at = ws + header_bytes(plan);
  void *dg = at, *du = at + hidden_bytes(p), *h = at + 2 * hidden_bytes(p);
  void* partial = at + 3 * hidden_bytes(p);
  const int T = p->T, D = p->D, F = p->F, O = p->D_out;
  const bool wide = p->grad_dtype == CP_F32;
  cp_status_t e;
  Product dh(GEMM_DGLU, false, true, T, F, plan.dh, FOLLOWS_NONE, ws, partial);
  dh.a(0, {dy, T, O, p->dy_stride});
  dh.b(0, {wd, O, F, p->w_down_stride});
  dh.k(O);
  dh.out(0, h);
  dh.g.act = p->activation;
  dh.kept(const_cast<void*>(gate), const_cast<void*>(up));
  dh.gradients(dg, du);
  if ((e = dh.run(plan, st, "hidden gradients")) != CP_OK) return e;
  if (dx) {   // dg Wg + du Wu as one product, k running through both
    Product q(GEMM_STORE, false, true, T, D, plan.dx, FOLLOWS_A, ws, partial);
    q.a(0, {dg, T, F, F});
    q.a(1, {du, T, F, F});
    q.b(0, {wg, F, D, p->w_gate_stride});
    q.b(1, {wu, F, D, p->w_up_stride});
    q.k(F, 2);
    q.out(0, dx);
    if ((e = q.run(plan, st, "input gradient")) != CP_OK) return e;
  }
  if (dwd) {
    Product q(GEMM_STORE, true, true, O, F, plan.d_down, FOLLOWS_BOTH, ws, partial);
    q.a(0, {dy, T, O, p->dy_stride});
    q.b(0, {h, T, F, F});
    q.k(T);
    q.out(0, dwd, wide);
    if ((e = q.run(plan, st, "down weight's gradient")) != CP_OK) return e;
  }
  if (dwg || dwu) {   // both as one product, m running through both
    const bool both = dwg && dwu;
    Product q(GEMM_STORE, true, true, F, D, both ? plan.d_both : plan.d_in, FOLLOWS_BOTH, ws,
              partial);
    q.a(0, {dwg ? dg : du, T, F, F});
    q.out(0, dwg ? dwg : dwu, wide);
    if (both) {
      q.a(1, {du, T, F, F});
      q.out(1, dwu, wide);
      q.g.m_tiles *= 2;
    }
    q.b(0, {x, T, D, p->x_stride});
    q.k(T);
    if ((e = q.run(plan, st, "gate and up weights' gradients")) != CP_OK) return e;
  }
  return CP_OK;
}

// fp32 products, their shares joined where there are several.
struct F32 {
  float* partial;
  cudaStream_t st;

  // The operands' order in memory: A and B row by row along k, or across it.
  static GemmF32Args args(int M, int N, int K, int64_t a_stride, bool a_mn, int64_t b_stride,
                          bool b_mn, const Share& s) {
    GemmF32Args g = {};
    g.M = M;
    g.N = N;
    g.K = K;
    g.sam = a_mn ? 1 : a_stride;
    g.sak = a_mn ? a_stride : 1;
    for (int i = 0; i < 2; ++i) {
      g.sbn[i] = b_mn ? 1 : b_stride;
      g.sbk[i] = b_mn ? b_stride : 1;
    }
    g.outputs = g.phases = 1;
    g.tile = s.whole;
    g.splits = s.shares;
    return g;
  }
  static const float* in(const void* p) { return static_cast<const float*>(p); }
  // to the workspace, as [outputs][splits][M][N]
  cp_status_t shares(GemmF32Args& g, const char* what) const {
    g.out[0] = partial;
    g.out[1] = partial + (int64_t)g.splits * g.M * g.N;
    ENTRY_CUDA(launch_gemm_f32(g, st), what);
    return CP_OK;
  }
  cp_status_t run(GemmF32Args& g, void* out0, void* out1, const char* what) const {
    void* out[2] = {out0, out1};
    if (g.splits == 1) {
      for (int i = 0; i < 2; ++i) g.out[i] = static_cast<float*>(out[i]);
      ENTRY_CUDA(launch_gemm_f32(g, st), what);
      return CP_OK;
    }
    cp_status_t e = shares(g, what);
    for (int i = 0; i < g.outputs && e == CP_OK; ++i) {
      F32JoinArgs j = {};
      j.partial = g.out[i];
      j.splits = g.splits;
      j.n = (int64_t)g.M * g.N;
      j.out = static_cast<float*>(out[i]);
      ENTRY_CUDA(launch_f32_join(j, GEMM_STORE, st), what);
    }
    return e;
  }
};

cp_status_t fwd_f32(const cp_gated_ffn_t* p, const Plan& plan, const void* x, const void* wg,
                    const void* wu, const void* wd, void* y, void* gate, void* up, uint8_t* ws,
                    cudaStream_t st) {
  float* h = reinterpret_cast<float*>(ws + header_bytes(plan));
  const F32 f{reinterpret_cast<float*>(ws + header_bytes(plan) + hidden_bytes(p)), st};
  const int T = p->T, D = p->D, F = p->F, O = p->D_out;
  cp_status_t e;
  GemmF32Args g = F32::args(T, F, D, p->x_stride, false, p->w_gate_stride, false, plan.gate_up);
  for (int i = 0; i < 2; ++i) {
    g.a[i] = F32::in(x);
    g.b[i] = F32::in(i ? wu : wg);
  }
  g.sbn[1] = p->w_up_stride;
  g.outputs = 2;
  if ((e = f.shares(g, "gate and up projections")) != CP_OK) return e;
  F32JoinArgs j = {};
  j.partial = f.partial;
  j.splits = g.splits;
  j.n = (int64_t)T * F;
  j.out = h;
  j.act = p->activation;
  j.gate = static_cast<float*>(gate);
  j.up = static_cast<float*>(up);
  ENTRY_CUDA(launch_f32_join(j, GEMM_GLU, st), "activation");
  g = F32::args(T, O, F, F, false, p->w_down_stride, false, plan.down);
  g.a[0] = h;
  g.b[0] = F32::in(wd);
  return f.run(g, y, nullptr, "down projection");
}

cp_status_t bwd_f32(const cp_gated_ffn_t* p, const Plan& plan, const void* x, const void* wg,
                    const void* wu, const void* wd, const void* gate, const void* up,
                    const void* dy, void* dx, void* dwg, void* dwu, void* dwd, uint8_t* ws,
                    cudaStream_t st) {
  uint8_t* at = ws + header_bytes(plan);
  float* dg = reinterpret_cast<float*>(at);
  float* du = reinterpret_cast<float*>(at + hidden_bytes(p));
  float* h = reinterpret_cast<float*>(at + 2 * hidden_bytes(p));
  const F32 f{reinterpret_cast<float*>(at + 3 * hidden_bytes(p)), st};
  const int T = p->T, D = p->D, F = p->F, O = p->D_out;
  cp_status_t e;
  GemmF32Args g = F32::args(T, F, O, p->dy_stride, false, p->w_down_stride, true, plan.dh);
  g.a[0] = F32::in(dy);
  g.b[0] = F32::in(wd);
  if ((e = f.shares(g, "hidden gradients")) != CP_OK) return e;
  F32JoinArgs j = {};
  j.partial = f.partial;
  j.splits = g.splits;
  j.n = (int64_t)T * F;
  j.out = h;
  j.act = p->activation;
  j.gate = static_cast<float*>(const_cast<void*>(gate));
  j.up = static_cast<float*>(const_cast<void*>(up));
  j.dgate = dg;
  j.dup = du;
  ENTRY_CUDA(launch_f32_join(j, GEMM_DGLU, st), "activation's gradient");
  if (dx) {   // dg Wg + du Wu as one product, k running through both
    g = F32::args(T, D, F, F, false, p->w_gate_stride, true, plan.dx);
    g.a[0] = dg;
    g.a[1] = du;
    g.b[0] = F32::in(wg);
    g.b[1] = F32::in(wu);
    g.sbk[1] = p->w_up_stride;
    g.phases = 2;
    if ((e = f.run(g, dx, nullptr, "input gradient")) != CP_OK) return e;
  }
  if (dwd) {
    g = F32::args(O, F, T, p->dy_stride, true, F, true, plan.d_down);
    g.a[0] = F32::in(dy);
    g.b[0] = h;
    if ((e = f.run(g, dwd, nullptr, "down weight's gradient")) != CP_OK) return e;
  }
  if (dwg || dwu) {
    const bool both = dwg && dwu;
    g = F32::args(F, D, T, F, true, p->x_stride, true, both ? plan.d_both : plan.d_in);
    g.a[0] = dwg ? dg : du;
    g.a[1] = du;
    g.b[0] = g.b[1] = F32::in(x);
    g.outputs = both ? 2 : 1;
    if ((e = f.run(g, dwg ? dwg : dwu, dwu, "gate and up weights' gradients")) != CP_OK) return e;
  }
  return CP_OK;
}

}  // namespace

extern "C" {

size_t cp_gated_ffn_kept_size(const cp_gated_ffn_t* desc) {
  if (check_desc(desc) != CP_OK) return 0;
  return desc->dtype == CP_BF16 ? (size_t)kept_bytes(desc->T, desc->F)
                                : (size_t)desc->T * desc->F * 4;
}

size_t cp_gated_ffn_fwd_workspace_size(const cp_gated_ffn_t* desc) {
  const int sms = check_desc(desc) == CP_OK ? sm_count() : 0;
  return sms > 0 ? fwd_bytes(desc, make_plan(desc, sms)) : 0;
}

size_t cp_gated_ffn_bwd_workspace_size(const cp_gated_ffn_t* desc) {
  const int sms = check_desc(desc) == CP_OK ? sm_count() : 0;
  return sms > 0 ? bwd_bytes(desc, make_plan(desc, sms)) : 0;
}

cp_status_t cp_gated_ffn_fwd(const cp_gated_ffn_t* desc, const void* x, const void* w_gate,
                             const void* w_up, const void* w_down, void* y, void* gate, void* up,
                             void* workspace, size_t ws_bytes, void* stream) {
  ENTRY_TRY
  cp_status_t e = check_desc(desc);
  if (e != CP_OK) return e;
  if (desc->T == 0) return CP_OK;
  if ((e = check_ptr(x, "x")) != CP_OK || (e = check_ptr(w_gate, "w_gate")) != CP_OK ||
      (e = check_ptr(w_up, "w_up")) != CP_OK || (e = check_ptr(w_down, "w_down")) != CP_OK ||
      (e = check_ptr(y, "y")) != CP_OK)
    return e;
  if ((gate == nullptr) != (up == nullptr))
    return entry_fail(CP_ERR_INVALID_ARG, "gate and up are kept together or not at all");
  if (!aligned_to(gate, 16) || !aligned_to(up, 16))
    return entry_fail(CP_ERR_ALIGNMENT, "gate and up must be 16-byte aligned");
  if (!workspace) return entry_fail(CP_ERR_WORKSPACE, "workspace is NULL");
  const Plan plan = make_plan(desc, sm_count());
  if (plan.sms < 2) return entry_fail(CP_ERR_CUDA, "no CUDA device");
  if ((e = check_workspace(workspace, ws_bytes, fwd_bytes(desc, plan))) != CP_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (few_rows(desc))
    return fwd_rows(desc, plan, x, w_gate, w_up, w_down, y, gate, up, ws, st);
  ENTRY_CUDA(cudaMemsetAsync(ws, 0, header_bytes(plan), st), "clear the status word");
  if (batch_rows(desc)) return fwd_tokens(desc, plan, x, w_gate, w_up, w_down, y, gate, up, ws, st);
  return desc->dtype == CP_BF16 ? fwd_bf16(desc, plan, x, w_gate, w_up, w_down, y, gate, up, ws, st)
                                : fwd_f32(desc, plan, x, w_gate, w_up, w_down, y, gate, up, ws, st);
  ENTRY_CATCH
}

cp_status_t cp_gated_ffn_bwd(const cp_gated_ffn_t* desc, const void* x, const void* w_gate,
                             const void* w_up, const void* w_down, const void* gate,
                             const void* up, const void* dy, void* dx, void* dw_gate, void* dw_up,
                             void* dw_down, void* workspace, size_t ws_bytes, void* stream) {
  ENTRY_TRY
  cp_status_t e = check_desc(desc);
  if (e != CP_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (const void* p : {(const void*)dx, (const void*)dw_gate, (const void*)dw_up,
                        (const void*)dw_down})
    if (!aligned_to(p, 16)) return entry_fail(CP_ERR_ALIGNMENT, "gradients must be 16-byte aligned");
  if (desc->T == 0) {   // no rows: the weights' gradients are zero
    const size_t elem = desc->grad_dtype == CP_BF16 ? 2 : 4;
    const size_t in = (size_t)desc->F * desc->D * elem, out = (size_t)desc->F * desc->D_out * elem;
    if (dw_gate) ENTRY_CUDA(cudaMemsetAsync(dw_gate, 0, in, st), "clear gradients");
    if (dw_up) ENTRY_CUDA(cudaMemsetAsync(dw_up, 0, in, st), "clear gradients");
    if (dw_down) ENTRY_CUDA(cudaMemsetAsync(dw_down, 0, out, st), "clear gradients");
    return CP_OK;
  }
  if ((e = check_ptr(x, "x")) != CP_OK || (e = check_ptr(w_gate, "w_gate")) != CP_OK ||
      (e = check_ptr(w_up, "w_up")) != CP_OK || (e = check_ptr(w_down, "w_down")) != CP_OK ||
      (e = check_ptr(gate, "gate")) != CP_OK || (e = check_ptr(up, "up")) != CP_OK ||
      (e = check_ptr(dy, "dy")) != CP_OK)
    return e;
  if (!dx && !dw_gate && !dw_up && !dw_down) return CP_OK;   // nothing is wanted
  if (!workspace) return entry_fail(CP_ERR_WORKSPACE, "workspace is NULL");
  const Plan plan = make_plan(desc, sm_count());
  if (plan.sms < 2) return entry_fail(CP_ERR_CUDA, "no CUDA device");
  if ((e = check_workspace(workspace, ws_bytes, bwd_bytes(desc, plan))) != CP_OK) return e;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ENTRY_CUDA(cudaMemsetAsync(ws, 0, header_bytes(plan), st), "clear the status word");
  return desc->dtype == CP_BF16
             ? bwd_bf16(desc, plan, x, w_gate, w_up, w_down, gate, up, dy, dx, dw_gate, dw_up,
                        dw_down, ws, st)
             : bwd_f32(desc, plan, x, w_gate, w_up, w_down, gate, up, dy, dx, dw_gate, dw_up,
                       dw_down, ws, st);
  ENTRY_CATCH
}

}  // extern "C"
