// C ABI of the gated feed-forward block: argument checks, work split and the launch
// sequence.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>
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

// A checked descriptor as the launches take it.  The stride of a single row is not checked and may
// be anything, 1 among them, which would read as another order of the operand in memory: a
// contiguous row's instead.
cp_gated_ffn_t with_strides(const cp_gated_ffn_t* p) {
  cp_gated_ffn_t d = *p;
  if (d.T <= 1) {
    d.x_stride = d.D;
    d.dy_stride = d.D_out;
  }
  return d;
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
  // a thread that has not used the device yet (autograd's, say) has no context until it is
  // set, and tensor maps cannot be made without one
  if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Forward calls that the kernels for few rows take, and for a batch of them.
bool few_rows(const cp_gated_ffn_t* p) {
  return p->T <= (p->dtype == CP_BF16 ? kFewRows : kFewRowsF32);
}
bool batch_rows(const cp_gated_ffn_t* p) {
  return p->dtype == CP_BF16 && p->T > kFewRows && p->T <= kBatchRows;
}

// fp32 calls of more rows go through the tensor cores.
bool split_rows(const cp_gated_ffn_t* p) { return p->dtype == CP_F32 && p->T > kSimtRows; }

// A launch of products: the width of its tiles and how it is cut into units.  bf16: wide
// tiles are quicker per product (backward of 4096 rows, 2048 -> 5504, 375 and 594 us),
// narrow ones where wide ones are too few for the GPU (700 rows, 320 -> 1664, 31 and 23).
struct Launch {
  int n = 0, tile_n = 256;
  GemmCut cut[kGemmProblems] = {};
  size_t partial = 0;   // bytes
  bool shared() const { return partial > 0; }
};
struct Shape {
  int64_t M, N;
  int k_tiles, outputs;
};
Launch plan_launch(std::initializer_list<Shape> products, int epilogue, int pairs, bool split) {
  Launch best;
  double least = 0;
  for (int tile_n : {256, 128}) {
    if (split && tile_n != kSplitN) continue;
    const GemmCost cost = split ? split_cost(epilogue) : gemm_cost(epilogue, tile_n);
    Launch l;
    l.tile_n = tile_n;
    for (const Shape& p : products) {
      if (p.outputs == 0) continue;
      l.cut[l.n].tiles = (int64_t)p.outputs * tiles(p.M, kGemmM) *
                         tiles(p.N, epilogue == GEMM_GLU ? tile_n / 2 : tile_n);
      l.cut[l.n++].k_tiles = p.k_tiles;
    }
    const double t = cut_products(l.cut, l.n, pairs, cost);
    for (int i = 0; i < l.n; ++i) l.partial += partial_bytes(l.cut[i], tile_n);
    if (least == 0 || t < least) {
      best = l;
      least = t;
    }
  }
  return best;
}

// The products of a backward pass behind the hidden gradients, those with the longest k
// first: dx [T][D], k through both weights; `in` weights' gradients [F][D]; that of the
// down weight [D_out][F].  One launch: alone, each leaves most pairs of CTAs idle in its
// last round of tiles (the whole pass, 2000 rows, 512 -> 1360, 55 -> 35 us; 2000 rows,
// 1024 -> 2816, 95 -> 79; 18688 rows, 2048 -> 8192, 2345 -> 2285).
bool dx_first(const cp_gated_ffn_t* p) { return 2 * tiles(p->F, kGemmK) >= tiles(p->T, kGemmK); }
Launch plan_gradients(const cp_gated_ffn_t* p, int pairs, bool dx, int in, bool down) {
  const int64_t T = p->T, D = p->D, F = p->F, O = p->D_out;
  const int k_dx = 2 * tiles(F, kGemmK), k = tiles(T, kGemmK);
  const bool first = dx_first(p);
  return plan_launch({{T, D, k_dx, dx && first}, {F, D, k, in}, {O, F, k, down},
                      {T, D, k_dx, dx && !first}},
                     GEMM_STORE, pairs, p->dtype == CP_F32);
}

enum : int { WANT_FWD = 1, WANT_BWD = 2 };
struct Plan {
  int sms = 0;
  Launch gate_up, down, dh, gradients;                      // tensor cores
  // shares of k on CUDA cores; d_in: of one weight
  int f32_gate_up = 1, f32_down = 1, f32_dh = 1, d_down = 1, d_in = 1, d_both = 1, dx = 1;
  size_t fwd_partial = 0, bwd_partial = 0;                  // bytes
  int pairs() const { return sms / 2; }
};

// Which gradients a call wants, as plan_gradients takes them.
struct Wanted {
  bool dx, down;
  int in;
};
// For one direction; a backward's for the gradients that are wanted, or, without them, as
// much workspace as any of them takes.
Plan make_plan(const cp_gated_ffn_t* p, int sms, int direction, const Wanted* wanted = nullptr) {
  Plan r;
  r.sms = sms;
  if (sms < 2 || p->T == 0) return r;   // without rows there is nothing to launch
  const int64_t T = p->T, D = p->D, F = p->F, O = p->D_out;
  const bool split = split_rows(p);
  if (p->dtype == CP_BF16 || split) {
    if (direction == WANT_FWD) {
      if (few_rows(p) || batch_rows(p)) return r;
      r.gate_up = plan_launch({{T, F, tiles(D, kGemmK), 1}}, GEMM_GLU, r.pairs(), split);
      r.down = plan_launch({{T, O, tiles(F, kGemmK), 1}}, GEMM_STORE, r.pairs(), split);
      r.fwd_partial = std::max(r.gate_up.partial, r.down.partial);
      return r;
    }
    r.dh = plan_launch({{T, F, tiles(O, kGemmK), 1}}, GEMM_DGLU, r.pairs(), split);
    r.bwd_partial = r.dh.partial;
    for (int which = 1; which < 12; ++which) {
      const Wanted w = wanted ? *wanted : Wanted{(which & 1) != 0, (which >> 1 & 1) != 0, which >> 2};
      r.gradients = plan_gradients(p, r.pairs(), w.dx, w.in, w.down);
      r.bwd_partial = std::max(r.bwd_partial, r.gradients.partial);
      if (wanted) break;
    }
    return r;
  }
  // gate and up always go through the workspace, and so does dh
  auto share = [&](int64_t M, int64_t N, int64_t K, int outputs, int phases, bool always,
                   size_t* most) {
    const int n = share_f32(M, N, K, outputs, phases, sms);
    if (always || n > 1) *most = std::max(*most, (size_t)outputs * n * M * N * 4);
    return n;
  };
  if (direction == WANT_FWD) {
    if (few_rows(p)) return r;
    r.f32_gate_up = share(T, F, D, 2, 1, true, &r.fwd_partial);
    r.f32_down = share(T, O, F, 1, 1, false, &r.fwd_partial);
    return r;
  }
  r.f32_dh = share(T, F, O, 1, 1, true, &r.bwd_partial);
  r.dx = share(T, D, F, 1, 2, false, &r.bwd_partial);
  r.d_down = share(O, F, T, 1, 1, false, &r.bwd_partial);
  r.d_in = share(F, D, T, 1, 1, false, &r.bwd_partial);
  r.d_both = share(F, D, T, 2, 1, false, &r.bwd_partial);
  return r;
}

// At the start of a workspace, cleared by every call: the status word, and the tickets
// of shared tiles (fewer than there are pairs of CTAs).
constexpr size_t kTicketsAt = 256;
size_t header_bytes(const Plan& plan) { return kTicketsAt + up256((size_t)plan.sms / 2 * kTickets * 4); }

// Three bf16 planes of an fp32 matrix.
size_t plane_bytes(int64_t rows, int64_t cols) { return up256((size_t)rows * cols * 6); }
size_t hidden_bytes(const cp_gated_ffn_t* p) {
  if (split_rows(p)) return plane_bytes(p->T, p->F);
  return up256((size_t)p->T * p->F * (p->dtype == CP_BF16 ? 2 : 4));
}
size_t operand_bytes(const cp_gated_ffn_t* p, bool backward) {   // planes of the call's inputs
  if (!split_rows(p)) return 0;
  return plane_bytes(p->T, p->D) + 2 * plane_bytes(p->F, p->D) + plane_bytes(p->D_out, p->F) +
         (backward ? plane_bytes(p->T, p->D_out) : 0);
}

size_t fwd_bytes(const cp_gated_ffn_t* p, const Plan& plan) {
  return header_bytes(plan) + hidden_bytes(p) + operand_bytes(p, false) + up256(plan.fwd_partial);
}
size_t bwd_bytes(const cp_gated_ffn_t* p, const Plan& plan) {
  return header_bytes(plan) + 3 * hidden_bytes(p) + operand_bytes(p, true) +
         up256(plan.bwd_partial);
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

// A launch of products under construction; failures stick.  What is set belongs to the
// product added last.
template <class Args>
struct Products {
  Args g = {};
  const Launch& plan;
  int epilogue;
  decltype(&g.p[0]) p = nullptr;
  int64_t units = 0;
  int slots = 0, shared = 0;
  const char* err = nullptr;

  Products(int epi, const Launch& l, uint8_t* ws, void* partial) : plan(l), epilogue(epi) {
    g.partial = static_cast<float*>(partial);
    g.status = reinterpret_cast<int32_t*>(ws);
    g.tickets = reinterpret_cast<int32_t*>(ws + kTicketsAt);
    g.wait_limit = device_wait_limit();
  }
  void add(int M, int N, bool a_mn, bool b_mn, int64_t K) {
    const GemmCut& c = plan.cut[g.problems];
    p = &g.p[g.problems++];
    p->M = M;
    p->N = N;
    p->a_mn = a_mn;
    p->b_mn = b_mn;
    p->m_tiles = p->m_split = tiles(M, kGemmM);
    p->n_tiles = tiles(N, epilogue == GEMM_GLU ? plan.tile_n / 2 : plan.tile_n);
    p->k_split = p->k_tiles = tiles(K, kGemmK);
    p->first = (int)units;
    p->whole = (int)c.whole;
    p->shares = c.shares;
    p->first_slot = slots;
    p->first_ticket = shared;
    const int cut = (int)(c.tiles - c.whole);
    units += c.whole + (int64_t)cut * c.shares;
    slots += cut * c.shares;
    shared += cut;
  }
  int a_rows() const { return p->a_mn ? 64 : kGemmM / 2; }   // of a box
  int b_rows() const { return p->b_mn ? 64 : plan.tile_n / 2; }
  cp_status_t ready(const char* what) {
    if (err) return entry_fail(CP_ERR_CUDA, std::string(what) + ": " + err);
    if (units >= (int64_t)1 << 30) return entry_fail(CP_ERR_SHAPE, "too many tiles");
    g.units = (int)units;
    return CP_OK;
  }
};

struct Bf16Products : Products<GemmArgs> {
  Bf16Products(int epi, const Launch& l, int follows, uint8_t* ws, void* partial)
      : Products(epi, l, ws, partial) {
    g.follows = follows;
  }
  void map(CUtensorMap* m, const Matrix& x, int elem, int cols, int rows) {
    const char* e = nullptr;
    if (!make_map(m, x, elem, cols, rows, &e) && !err) err = e;
  }
  void a(int i, const Matrix& m) { map(&p->a[i], m, 2, kGemmK, a_rows()); }
  void b(int i, const Matrix& m) { map(&p->b[i], m, 2, kGemmK, b_rows()); }
  void box(CUtensorMap* m, void* at, int elem, int64_t stride) {   // what an epilogue moves
    map(m, {at, p->M, p->N, stride}, elem, elem == 4 ? 32 : 64, 32);
  }
  void out(int i, void* at, bool f32 = false) {
    p->out_f32 = f32;
    box(&p->out[i], at, f32 ? 4 : 2, p->N);
  }
  void kept(void* gate, void* up) {
    g.keep = gate != nullptr;
    if (!gate) return;
    for (int i = 0; i < 2; ++i) {
      uint8_t* at = static_cast<uint8_t*>(i ? up : gate);
      CUtensorMap* m = i ? g.up : g.gate;
      box(&m[0], at, 2, p->N);
      map(&m[1], {at + kept_low(p->M, p->N), p->M, p->N, kept_pitch(p->N)}, 1, 64, 32);
    }
  }
  void gradients(void* dgate, void* dup) {
    box(&g.dgate, dgate, 2, p->N);
    box(&g.dup, dup, 2, p->N);
  }

  cp_status_t run(int sms, cudaStream_t st, const char* what) {
    const cp_status_t e = ready(what);
    if (e != CP_OK) return e;
    ENTRY_CUDA(launch_gemm_bf16(g, epilogue, plan.tile_n, sms, st), what);
    return CP_OK;
  }
};

// Planes of an fp32 matrix of the call.
struct Planes {
  void* p;
  int64_t rows, cols;
};
struct SplitProducts : Products<SplitArgs> {
  SplitProducts(int epi, const Launch& l, uint8_t* ws, void* partial)
      : Products(epi, l, ws, partial) {}
  void map(CUtensorMap* m, const Planes& x, int rows) {
    const char* e = nullptr;
    if (!make_tmap_planes(m, x.p, x.rows, x.cols, rows, &e) && !err) err = e;
  }
  void a(int i, const Planes& m) { map(&p->a[i], m, a_rows()); }
  void b(int i, const Planes& m) { map(&p->b[i], m, b_rows()); }
  cp_status_t run(int sms, cudaStream_t st, const char* what) {
    const cp_status_t e = ready(what);
    if (e != CP_OK) return e;
    ENTRY_CUDA(launch_gemm_split(g, epilogue, sms, st), what);
    return CP_OK;
  }
};

// The header is cleared by the call's first launch itself where that shares no tiles.
cp_status_t clear_header(const Plan& plan, Bf16Products& first, uint8_t* ws, cudaStream_t st) {
  if (first.plan.shared())
    ENTRY_CUDA(cudaMemsetAsync(ws, 0, header_bytes(plan), st), "clear the status word");
  else
    first.g.clear = (int)(header_bytes(plan) / 4);
  return CP_OK;
}

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
  auto launch = p->dtype == CP_F32 ? launch_ffn_rows_f32 : launch_ffn_rows;
  ENTRY_CUDA(launch(a, true, plan.sms, st), "gate and up projections");
  a.x = a.out;
  a.x_stride = p->F;
  a.w[0] = a.w[1] = wd;
  a.w_stride[0] = a.w_stride[1] = p->w_down_stride;
  a.out = y;
  a.N = p->D_out;
  a.K = p->F;
  ENTRY_CUDA(launch(a, false, plan.sms, st), "down projection");
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
  Bf16Products gu(GEMM_GLU, plan.gate_up, FOLLOWS_NONE, ws, partial);
  gu.add(T, F, false, false, D);
  gu.a(0, {x, T, D, p->x_stride});
  gu.b(0, {wg, F, D, p->w_gate_stride});
  gu.b(1, {wu, F, D, p->w_up_stride});
  gu.out(0, h);
  gu.g.act = p->activation;
  gu.kept(gate, up);
  if ((e = clear_header(plan, gu, ws, st)) != CP_OK) return e;
  if ((e = gu.run(plan.sms, st, "gate and up projections")) != CP_OK) return e;
  Bf16Products down(GEMM_STORE, plan.down, FOLLOWS_A, ws, partial);
  down.add(T, O, false, false, F);
  down.a(0, {h, T, F, F});
  down.b(0, {wd, O, F, p->w_down_stride});
  down.out(0, y);
  return down.run(plan.sms, st, "down projection");
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
  Bf16Products dh(GEMM_DGLU, plan.dh, FOLLOWS_NONE, ws, partial);
  dh.add(T, F, false, true, O);
  dh.a(0, {dy, T, O, p->dy_stride});
  dh.b(0, {wd, O, F, p->w_down_stride});
  dh.out(0, h);
  dh.g.act = p->activation;
  dh.kept(const_cast<void*>(gate), const_cast<void*>(up));
  dh.gradients(dg, du);
  if ((e = clear_header(plan, dh, ws, st)) != CP_OK) return e;
  if ((e = dh.run(plan.sms, st, "hidden gradients")) != CP_OK) return e;

  const int in = (dwg != nullptr) + (dwu != nullptr);
  Bf16Products q(GEMM_STORE, plan.gradients, dx && !in && !dwd ? FOLLOWS_A : FOLLOWS_BOTH, ws, partial);
  auto input = [&] {   // dg Wg + du Wu as one product, k running through both
    q.add(T, D, false, true, F);
    q.p->k_tiles *= 2;
    q.a(0, {dg, T, F, F});
    q.a(1, {du, T, F, F});
    q.b(0, {wg, F, D, p->w_gate_stride});
    q.b(1, {wu, F, D, p->w_up_stride});
    q.out(0, dx);
  };
  if (dx && dx_first(p)) input();
  if (in) {   // both weights as one product, m running through both
    q.add(F, D, true, true, T);
    q.a(0, {dwg ? dg : du, T, F, F});
    q.out(0, dwg ? dwg : dwu, wide);
    if (in == 2) {
      q.a(1, {du, T, F, F});
      q.out(1, dwu, wide);
      q.p->m_tiles *= 2;
    }
    q.b(0, {x, T, D, p->x_stride});
  }
  if (dwd) {
    q.add(O, F, true, true, T);
    q.a(0, {dy, T, O, p->dy_stride});
    q.b(0, {h, T, F, F});
    q.out(0, dwd, wide);
  }
  if (dx && !dx_first(p)) input();
  return q.run(plan.sms, st, "gradients");
}

// fp32 on the tensor cores: the inputs' planes in one launch, then the products.
struct Operands {
  SplitPass s = {};
  uint8_t* at;

  Operands(const Plan& plan, uint8_t* ws, size_t hidden) : at(ws + header_bytes(plan) + hidden) {
    s.status = reinterpret_cast<int32_t*>(ws);
    s.clear = (int)(header_bytes(plan) / 4);
  }
  Planes add(const void* src, int64_t rows, int64_t cols, int64_t stride, bool wanted = true) {
    const Planes r = {at, rows, cols};
    at += plane_bytes(rows, cols);
    if (!wanted) return r;
    auto& m = s.m[s.n++];
    m.src = static_cast<const float*>(src);
    m.planes = static_cast<__nv_bfloat16*>(r.p);
    m.rows = rows;
    m.cols = (int)cols;
    m.stride = rows > 1 ? stride : cols;
    return r;
  }
};

cp_status_t fwd_split(const cp_gated_ffn_t* p, const Plan& plan, const void* x, const void* wg,
                      const void* wu, const void* wd, void* y, void* gate, void* up, uint8_t* ws,
                      cudaStream_t st) {
  const int T = p->T, D = p->D, F = p->F, O = p->D_out;
  const Planes h = {ws + header_bytes(plan), T, F};
  Operands in(plan, ws, hidden_bytes(p));
  const Planes px = in.add(x, T, D, p->x_stride), pg = in.add(wg, F, D, p->w_gate_stride),
               pu = in.add(wu, F, D, p->w_up_stride), pd = in.add(wd, O, F, p->w_down_stride);
  void* partial = in.at;
  ENTRY_CUDA(launch_split(in.s, st), "planes of the inputs");
  cp_status_t e;
  SplitProducts gu(GEMM_GLU, plan.gate_up, ws, partial);
  gu.add(T, F, false, false, D);
  gu.a(0, px);
  gu.b(0, pg);
  gu.b(1, pu);
  gu.g.act = p->activation;
  gu.g.gate = static_cast<float*>(gate);
  gu.g.up = static_cast<float*>(up);
  gu.g.h = static_cast<__nv_bfloat16*>(h.p);
  if ((e = gu.run(plan.sms, st, "gate and up projections")) != CP_OK) return e;
  SplitProducts down(GEMM_STORE, plan.down, ws, partial);
  down.add(T, O, false, false, F);
  down.a(0, h);
  down.b(0, pd);
  down.p->out[0] = static_cast<float*>(y);
  return down.run(plan.sms, st, "down projection");
}

cp_status_t bwd_split(const cp_gated_ffn_t* p, const Plan& plan, const void* x, const void* wg,
                      const void* wu, const void* wd, const void* gate, const void* up,
                      const void* dy, void* dx, void* dwg, void* dwu, void* dwd, uint8_t* ws,
                      cudaStream_t st) {
  const int T = p->T, D = p->D, F = p->F, O = p->D_out;
  uint8_t* at = ws + header_bytes(plan);
  const size_t hidden = hidden_bytes(p);
  const Planes dg = {at, T, F}, du = {at + hidden, T, F}, h = {at + 2 * hidden, T, F};
  const int n_in = (dwg != nullptr) + (dwu != nullptr);
  Operands in(plan, ws, 3 * hidden);
  const Planes px = in.add(x, T, D, p->x_stride, n_in > 0),
               pg = in.add(wg, F, D, p->w_gate_stride, dx),
               pu = in.add(wu, F, D, p->w_up_stride, dx),
               pd = in.add(wd, O, F, p->w_down_stride), py = in.add(dy, T, O, p->dy_stride);
  void* partial = in.at;
  ENTRY_CUDA(launch_split(in.s, st), "planes of the inputs");
  cp_status_t e;
  SplitProducts dh(GEMM_DGLU, plan.dh, ws, partial);
  dh.add(T, F, false, true, O);
  dh.a(0, py);
  dh.b(0, pd);
  dh.g.act = p->activation;
  dh.g.gate = static_cast<float*>(const_cast<void*>(gate));
  dh.g.up = static_cast<float*>(const_cast<void*>(up));
  dh.g.h = static_cast<__nv_bfloat16*>(h.p);
  dh.g.dgate = static_cast<__nv_bfloat16*>(dg.p);
  dh.g.dup = static_cast<__nv_bfloat16*>(du.p);
  if ((e = dh.run(plan.sms, st, "hidden gradients")) != CP_OK) return e;

  SplitProducts q(GEMM_STORE, plan.gradients, ws, partial);
  auto input = [&] {
    q.add(T, D, false, true, F);
    q.p->k_tiles *= 2;
    q.a(0, dg);
    q.a(1, du);
    q.b(0, pg);
    q.b(1, pu);
    q.p->out[0] = static_cast<float*>(dx);
  };
  if (dx && dx_first(p)) input();
  if (n_in) {
    q.add(F, D, true, true, T);
    q.a(0, dwg ? dg : du);
    q.p->out[0] = static_cast<float*>(dwg ? dwg : dwu);
    if (n_in == 2) {
      q.a(1, du);
      q.p->out[1] = static_cast<float*>(dwu);
      q.p->m_tiles *= 2;
    }
    q.b(0, px);
  }
  if (dwd) {
    q.add(O, F, true, true, T);
    q.a(0, py);
    q.b(0, h);
    q.p->out[0] = static_cast<float*>(dwd);
  }
  if (dx && !dx_first(p)) input();
  return q.run(plan.sms, st, "gradients");
}

// fp32 products, their shares joined where there are several.
struct F32 {
  float* partial;
  cudaStream_t st;

  // The operands' order in memory: A and B row by row along k, or across it.
  static GemmF32Args args(int M, int N, int K, int64_t a_stride, bool a_mn, int64_t b_stride,
                          bool b_mn, int shares) {
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
    g.splits = shares;
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
  GemmF32Args g = F32::args(T, F, D, p->x_stride, false, p->w_gate_stride, false, plan.f32_gate_up);
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
  g = F32::args(T, O, F, F, false, p->w_down_stride, false, plan.f32_down);
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
  GemmF32Args g = F32::args(T, F, O, p->dy_stride, false, p->w_down_stride, true, plan.f32_dh);
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
  return sms > 0 ? fwd_bytes(desc, make_plan(desc, sms, WANT_FWD)) : 0;
}

size_t cp_gated_ffn_bwd_workspace_size(const cp_gated_ffn_t* desc) {
  const int sms = check_desc(desc) == CP_OK ? sm_count() : 0;
  return sms > 0 ? bwd_bytes(desc, make_plan(desc, sms, WANT_BWD)) : 0;
}

cp_status_t cp_gated_ffn_fwd(const cp_gated_ffn_t* given, const void* x, const void* w_gate,
                             const void* w_up, const void* w_down, void* y, void* gate, void* up,
                             void* workspace, size_t ws_bytes, void* stream) {
  ENTRY_TRY
  cp_status_t e = check_desc(given);
  if (e != CP_OK) return e;
  const cp_gated_ffn_t d = with_strides(given), *desc = &d;
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
  const Plan plan = make_plan(desc, sm_count(), WANT_FWD);
  if (plan.sms < 2) return entry_fail(CP_ERR_CUDA, "no CUDA device");
  if ((e = check_workspace(workspace, ws_bytes, fwd_bytes(desc, plan))) != CP_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (few_rows(desc))
    return fwd_rows(desc, plan, x, w_gate, w_up, w_down, y, gate, up, ws, st);
  if (desc->dtype == CP_BF16 && !batch_rows(desc))
    return fwd_bf16(desc, plan, x, w_gate, w_up, w_down, y, gate, up, ws, st);
  if (split_rows(desc))
    return fwd_split(desc, plan, x, w_gate, w_up, w_down, y, gate, up, ws, st);
  ENTRY_CUDA(cudaMemsetAsync(ws, 0, header_bytes(plan), st), "clear the status word");
  return batch_rows(desc) ? fwd_tokens(desc, plan, x, w_gate, w_up, w_down, y, gate, up, ws, st)
                          : fwd_f32(desc, plan, x, w_gate, w_up, w_down, y, gate, up, ws, st);
  ENTRY_CATCH
}

cp_status_t cp_gated_ffn_bwd(const cp_gated_ffn_t* given, const void* x, const void* w_gate,
                             const void* w_up, const void* w_down, const void* gate,
                             const void* up, const void* dy, void* dx, void* dw_gate, void* dw_up,
                             void* dw_down, void* workspace, size_t ws_bytes, void* stream) {
  ENTRY_TRY
  cp_status_t e = check_desc(given);
  if (e != CP_OK) return e;
  const cp_gated_ffn_t d = with_strides(given), *desc = &d;
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
  const Wanted wanted = {dx != nullptr, dw_down != nullptr,
                         (dw_gate != nullptr) + (dw_up != nullptr)};
  const Plan plan = make_plan(desc, sm_count(), WANT_BWD, &wanted);
  if (plan.sms < 2) return entry_fail(CP_ERR_CUDA, "no CUDA device");
  if ((e = check_workspace(workspace, ws_bytes, bwd_bytes(desc, plan))) != CP_OK) return e;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (desc->dtype == CP_BF16)
    return bwd_bf16(desc, plan, x, w_gate, w_up, w_down, gate, up, dy, dx, dw_gate, dw_up, dw_down,
                    ws, st);
  if (split_rows(desc))
    return bwd_split(desc, plan, x, w_gate, w_up, w_down, gate, up, dy, dx, dw_gate, dw_up,
                     dw_down, ws, st);
  ENTRY_CUDA(cudaMemsetAsync(ws, 0, header_bytes(plan), st), "clear the status word");
  return bwd_f32(desc, plan, x, w_gate, w_up, w_down, gate, up, dy, dx, dw_gate, dw_up, dw_down, ws,
                 st);
  ENTRY_CATCH
}

}  // extern "C"
