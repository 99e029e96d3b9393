// C ABI of attention with modified scores: plans, argument checks, workspace
// layout and the launch sequence.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>

#include "../../include/cpattn.h"
#include "entry.h"
#include "kernels.h"
#include "scored.h"
#include "scored_plan.h"
#include "tc.h"

using namespace cpattn;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int table_mid(int n_dist) { return n_dist + kTableSlack; }
int table_pitch(int n_dist) { return 2 * table_mid(n_dist) + 1; }

const ScorePlanHeader* header(const void* plan_h) {
  if (!plan_h || !aligned_to(plan_h, 8)) return nullptr;
  const ScorePlanHeader* h = static_cast<const ScorePlanHeader*>(plan_h);
  return h->magic == kScorePlanMagic ? h : nullptr;
}

// Offsets into the workspace of either direction.  What has to start at zero
// comes first, so that one memset clears it.
struct Ws {
  size_t status = 0, scales = 0, ranges = 0;
  size_t dtable = 0, dq = 0, dk = 0, dv = 0;   // backward (dq, dk, dv: bf16 results)
  size_t table = 0;
  size_t v16 = 0, part_out = 0, part_lse = 0;  // forward (parts: fp32 results)
  size_t lse2 = 0, D = 0, q16 = 0, k16 = 0;    // backward
  size_t total = 0;
};

inline int64_t ld_pitch(int64_t T) { return (T + 3) / 4 * 4; }

// The forward's partial results live in the workspace, so its split follows from
// the plan alone (n_sms is the plan's).
int f32_fwd_splits(const ScorePlanHeader& h) {
  return f32_splits((int64_t)h.n_tiles * h.H, h.max_walk, h.n_sms);
}

// The forward's P V on f16 operands, above softmax scale 0.25 as cp_attn_fwd, and with a
// learned bias that a backward will follow (out_lo): the bias's gradient is a sum of
// dS = P (dP - D) in which rows cancel, so that an error of D = dO . O shows.  Before
// its own rounding dbias is off by 1e-3 to 3e-3 (relative) with P in bf16, by 1e-4 to
// 2e-4 with P in f16.
// The backward's types do not follow the scale: dS is bf16, but f16 in the short samples
// whose range allows it (operand_range.cuh).  One power of two for all of a call's dS
// would leave a sample whose dout is 2^-20 of another's next to none of f16's bits (512
// tokens of 128: dq off by 8e-2 at 1e-6; in bf16 by 1.8e-3 at any ratio).
bool f16_operands(cp_dtype_t dt, float scale, bool bias_gradient) {
  return dt == CP_BF16 && (uses_f16_operands(scale) || bias_gradient);
}
bool has_ranges(const ScorePlanHeader& h, cp_dtype_t dt) { return dt == CP_BF16 && h.n_short > 0; }

Ws layout(const ScorePlanHeader& h, cp_dtype_t dt, int Hkv, int d, float scale, bool backward,
          bool bf16_grads) {
  Ws w;
  const bool f16 = !backward && f16_operands(dt, scale, h.n_dist > 0);
  const size_t T = h.T;
  size_t o = kStatusBytes;
  auto take = [&](size_t* at, bool need, size_t bytes) {
    *at = o;
    if (need) o = up256(o + bytes);
  };
  const bool ranges = backward && has_ranges(h, dt);
  take(&w.scales, f16, sizeof(OpScales));
  take(&w.ranges, ranges, (size_t)h.n_seqs * Hkv * sizeof(OperandRange));
  take(&w.dtable, backward && h.n_dist > 0, (size_t)h.H * h.n_dist * sizeof(float));
  take(&w.dq, backward && bf16_grads, T * h.H * d * sizeof(float));
  take(&w.dk, backward && bf16_grads, T * Hkv * d * sizeof(float));
  take(&w.dv, backward && bf16_grads, T * Hkv * d * sizeof(float));
  take(&w.table, h.n_dist > 0, (size_t)h.H * table_pitch(h.n_dist) * sizeof(float));
  if (!backward) {
    const size_t splits = dt == CP_F32 ? f32_fwd_splits(h) : 1;
    const size_t rows = dt == CP_BF16 ? h.run_rows : splits > 1 ? splits * T : 0;
    take(&w.v16, f16, T * Hkv * d * 2);
    take(&w.part_out, rows > 0, rows * h.H * d * sizeof(float));
    take(&w.part_lse, rows > 0, rows * h.H * sizeof(float));
  } else {
    const size_t plane = (size_t)ld_pitch(T) * h.H * sizeof(float);
    take(&w.lse2, true, 2 * plane);
    w.D = w.lse2 + plane;   // plane 1 directly after plane 0
    take(&w.q16, ranges, T * h.H * d * 2);
    take(&w.k16, ranges, T * Hkv * d * 2);
  }
  w.total = o;
  return w;
}

struct Call {
  const ScorePlanHeader* h = nullptr;
  bool bf16 = false, f16 = false;   // f16: the forward's P V on f16 operands
  int bias = SCORE_PLAIN;
  Ws ws;
};

// Checks everything that does not need a GPU.
cp_status_t check(const void* plan_h, const void* plan_d, const void* const* ptrs, int n_ptrs,
                  cp_dtype_t dt, int T, int H, int Hkv, int d, const cp_score_t* sc, float scale,
                  const void* out_lo, const void* ws, size_t ws_bytes, bool backward,
                  bool bf16_grads, Call* c) {
  c->h = header(plan_h);
  if (!c->h) return entry_fail(CP_ERR_INVALID_ARG, "plan_h is not a score plan");
  if (!sc) return entry_fail(CP_ERR_INVALID_ARG, "score is NULL");
  if (dt != CP_F32 && dt != CP_BF16)
    return entry_fail(CP_ERR_DTYPE, "dtype must be CP_F32 or CP_BF16");
  if (T != c->h->T) return entry_fail(CP_ERR_SHAPE, "T differs from the plan's cu_seqlens");
  if (H != c->h->H) return entry_fail(CP_ERR_SHAPE, "H differs from the plan's");
  if (Hkv < 1 || H % Hkv != 0)
    return entry_fail(CP_ERR_SHAPE, "H must be a positive multiple of H_kv");
  if (d != 64 && d != 128) return entry_fail(CP_ERR_SHAPE, "head_dim must be 64 or 128");
  // its inverse, and its quotients with the cap and the slopes, stay normal numbers
  if (!(scale >= 1e-10f && scale <= 1e10f))
    return entry_fail(CP_ERR_INVALID_ARG, "softmax_scale must be in [1e-10, 1e10]");
  if (!(sc->softcap >= 0.f) || !std::isfinite(sc->softcap))
    return entry_fail(CP_ERR_INVALID_ARG, "softcap must be finite and >= 0 (0: none)");
  // cap * log2(e), its inverse and that inverse's eighth power stay normal numbers
  if (sc->softcap != 0.f && (sc->softcap < 1e-3f || sc->softcap > 1e4f))
    return entry_fail(CP_ERR_INVALID_ARG, "softcap must be 0 or in [1e-3, 1e4]");
  if (sc->slopes && sc->rel_bias)
    return entry_fail(CP_ERR_INVALID_ARG, "slopes and rel_bias exclude one another");
  if (sc->slopes && !aligned_to(sc->slopes, 4))
    return entry_fail(CP_ERR_ALIGNMENT, "slopes are not aligned to their element type");
  if (sc->rel_bias) {
    if (c->h->n_dist == 0)
      return entry_fail(CP_ERR_INVALID_ARG, "rel_bias needs a plan with buckets");
    if (sc->bias_dtype != CP_F32 && sc->bias_dtype != CP_BF16)
      return entry_fail(CP_ERR_DTYPE, "bias_dtype must be CP_F32 or CP_BF16");
    if (sc->n_buckets < c->h->n_buckets)
      return entry_fail(CP_ERR_SHAPE, "the plan's buckets exceed n_buckets");
    if (!aligned_to(sc->rel_bias, sc->bias_dtype == CP_BF16 ? 2 : 4))
      return entry_fail(CP_ERR_ALIGNMENT, "rel_bias is not aligned to its element type");
  }
  c->bias = sc->slopes ? SCORE_SLOPES : sc->rel_bias ? SCORE_TABLE : SCORE_PLAIN;
  c->bf16 = dt == CP_BF16;
  c->f16 = !backward &&
           f16_operands(dt, scale, out_lo != nullptr && c->bias == SCORE_TABLE);
  c->ws = layout(*c->h, dt, Hkv, d, scale, backward, bf16_grads);
  if (out_lo && !c->bf16) return entry_fail(CP_ERR_DTYPE, "out_lo is for bf16 outputs only");
  if (T == 0) return CP_OK;
  if (!plan_d) return entry_fail(CP_ERR_INVALID_ARG, "plan_d is NULL");
  if (!aligned_to(plan_d, 256))
    return entry_fail(CP_ERR_ALIGNMENT, "plan_d must be 256-byte aligned");
  for (int i = 0; i < n_ptrs; ++i) {
    if (!ptrs[i]) return entry_fail(CP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (!aligned_to(ptrs[i], 16))
      return entry_fail(CP_ERR_ALIGNMENT, "tensor pointers must be 16-byte aligned");
  }
  if (!aligned_to(out_lo, 16)) return entry_fail(CP_ERR_ALIGNMENT, "out_lo alignment");
  if (!ws || ws_bytes < c->ws.total)
    return entry_fail(CP_ERR_WORKSPACE, "workspace smaller than cp_attn_scored_*_workspace_size()");
  if (!aligned_to(ws, 256))
    return entry_fail(CP_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  return CP_OK;
}

// As bwd_kv_split, for groups of any size: CTAs that share a group of query heads.
// (4096 tokens of 128, 6 heads over 2: 264 us with powers of two alone, 107 so;
// 8192, 5 over 1: 826 and 234.)
int group_split(int64_t n_items, int H, int Hkv, int sms) {
  const int G = H / Hkv;
  for (int s = 1; s < G; ++s)
    if (G % s == 0 && n_items * Hkv * s >= 4LL * sms) return s;
  return G;
}

cp_status_t check_gpu(bool bf16, int* sms) {
  int dev = 0, major = 0, minor = 0;
  ENTRY_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  ENTRY_CUDA(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev), "SM count");
  ENTRY_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev), "cc major");
  ENTRY_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev), "cc minor");
  if (bf16 && (major != 10 || minor != 3))
    return entry_fail(CP_ERR_UNSUPPORTED,
                      "the bf16 path is built for sm_103a (compute capability 10.3)");
  return CP_OK;
}

// The tensor-core kernels' view of the scores; lays the table out by distance.
cp_status_t prepare_scores(const Call& c, const cp_score_t* sc, float scale, const char* plan,
                           char* w, ScoreArgs* s, cudaStream_t st) {
  *s = ScoreArgs{};
  s->cap_log2 = sc->softcap * kLog2e;
  s->inv_cap_log2 = sc->softcap > 0.f ? 1.f / s->cap_log2 : 0.f;
  if (sc->softcap > 0.f) fill_cap_polynomial(s, scale * kLog2e);
  s->slopes = sc->slopes;
  if (c.bias == SCORE_TABLE) {
    s->n_dist = c.h->n_dist;
    s->table_mid = table_mid(s->n_dist);
    s->table_pitch = table_pitch(s->n_dist);
    float* table = reinterpret_cast<float*>(w + c.ws.table);
    s->table = table;
    ENTRY_CUDA(launch_expand_bias(sc->rel_bias, sc->bias_dtype == CP_BF16, sc->bias_stride_h,
                                  sc->bias_stride_b,
                                  reinterpret_cast<const int32_t*>(plan + c.h->buckets), s->n_dist,
                                  c.h->H, c.bf16 ? kLog2e : 1.f, table, s->table_mid,
                                  s->table_pitch, st),
               "bias by distance");
  }
  return CP_OK;
}

F32Args f32_args(const Call& c, const cp_score_t* sc, const char* plan, const ScoreArgs& s, int Hkv,
                 float scale) {
  F32Args a{};
  a.tiles = reinterpret_cast<const Tile32*>(plan + c.h->tiles);
  a.n_tiles = c.h->n_tiles;
  a.H = c.h->H;
  a.Hkv = Hkv;
  a.T = c.h->T;
  a.scale = scale;
  a.softcap = sc->softcap;
  a.inv_cap = sc->softcap > 0.f ? 1.f / sc->softcap : 0.f;
  a.slopes = sc->slopes;
  a.table = s.table;
  a.table_pitch = s.table_pitch;
  a.table_mid = s.table_mid;
  a.n_dist = s.n_dist;
  return a;
}

}  // namespace

extern "C" {

size_t cp_score_plan_size(const int32_t* cu, int n_seqs, const int32_t* prefix_lens,
                          int bidirectional, int H, int n_sms, const int32_t* buckets,
                          int n_dist) {
  try {
    ScorePlanHeader h;
    const std::string err = score_plan_layout(cu, n_seqs, prefix_lens, bidirectional != 0, H, n_sms,
                                              buckets, n_dist, &h);
    if (err.empty()) return h.total;
    set_last_error(err);
  } catch (const std::exception& ex) {   // its lists may not fit in memory
    set_last_error(ex.what());
  }
  return 0;
}

cp_status_t cp_score_plan_build(const int32_t* cu, int n_seqs, const int32_t* prefix_lens,
                                int bidirectional, int H, int n_sms, const int32_t* buckets,
                                int n_dist, void* block, size_t bytes) {
  ENTRY_TRY
  ScorePlanHeader h;
  const std::string err = score_plan_layout(cu, n_seqs, prefix_lens, bidirectional != 0, H, n_sms,
                                            buckets, n_dist, &h);
  if (!err.empty()) return entry_fail(CP_ERR_SHAPE, err);
  if (!block || bytes < h.total)
    return entry_fail(CP_ERR_WORKSPACE, "block smaller than cp_score_plan_size()");
  if (!aligned_to(block, 8)) return entry_fail(CP_ERR_ALIGNMENT, "block must be 8-byte aligned");
  score_plan_build(h, cu, prefix_lens, buckets, block);
  return CP_OK;
  ENTRY_CATCH
}

cp_status_t cp_score_plan_pairs(const void* plan_h, int64_t* fwd, int64_t* bwd, int64_t* tiles) {
  const ScorePlanHeader* h = header(plan_h);
  if (!h) return entry_fail(CP_ERR_INVALID_ARG, "plan_h is not a score plan");
  const char* b = static_cast<const char*>(plan_h);
  int64_t nf = 0, nb = 0, nt = 0;
  const FwdItem* fi = reinterpret_cast<const FwdItem*>(b + h->fwd);
  for (int i = 0; i < h->n_fwd; ++i)
    for (int t = 0; t < fi[i].q_len; ++t) {
      const Seg& s = fi[i].seg[0];
      nf += s.causal ? std::max<int64_t>(0, std::min<int64_t>(s.len, (int64_t)t + s.delta + 1))
                     : s.len;
    }
  const BwdItem* bi = reinterpret_cast<const BwdItem*>(b + h->bwd);
  const Seg* runs = reinterpret_cast<const Seg*>(b + h->runs);
  for (int i = 0; i < h->n_bwd; ++i)
    for (int u = 0; u < bi[i].k_len; ++u) {
      const Seg& s = runs[bi[i].run0];
      nb += s.causal ? std::min<int64_t>(s.len, std::max<int64_t>(0, s.len - (u - s.delta)))
                     : s.len;
    }
  const Tile32* ti = reinterpret_cast<const Tile32*>(b + h->tiles);
  for (int i = 0; i < h->n_tiles; ++i)
    for (int t = 0; t < ti[i].len; ++t) {
      const int64_t pos = ti[i].row0 - ti[i].seq0 + t;
      nt += std::max<int64_t>(pos + 1, pos < ti[i].prefix ? ti[i].prefix : 0);
    }
  if (fwd) *fwd = nf;
  if (bwd) *bwd = nb;
  if (tiles) *tiles = nt;
  return CP_OK;
}

size_t cp_attn_scored_fwd_workspace_size(const void* plan_h, cp_dtype_t dt, int Hkv, int d,
                                         float scale) {
  const ScorePlanHeader* h = header(plan_h);
  if (!h || Hkv < 1 || d < 1) return 0;
  return layout(*h, dt, Hkv, d, scale, false, false).total;
}

size_t cp_attn_scored_bwd_workspace_size(const void* plan_h, cp_dtype_t dt, int Hkv, int d,
                                         float scale, cp_dtype_t grad_dt) {
  const ScorePlanHeader* h = header(plan_h);
  if (!h || Hkv < 1 || d < 1) return 0;
  return layout(*h, dt, Hkv, d, scale, true, grad_dt == CP_BF16).total;
}

cp_status_t cp_attn_scored_fwd(const void* plan_h, const void* plan_d, const void* q,
                               const void* k, const void* v, cp_dtype_t dt, int T, int H, int Hkv,
                               int d, const cp_score_t* score, float scale, void* out, float* lse,
                               void* out_lo, void* ws, size_t ws_bytes, void* stream) {
  ENTRY_TRY
  const void* ptrs[5] = {q, k, v, out, lse};
  Call c;
  cp_status_t e = check(plan_h, plan_d, ptrs, 5, dt, T, H, Hkv, d, score, scale, out_lo, ws,
                        ws_bytes, false, false, &c);
  if (e != CP_OK) return e;
  if (T == 0) return CP_OK;
  int sms = 0;
  if ((e = check_gpu(c.bf16, &sms)) != CP_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  const char* plan = static_cast<const char*>(plan_d);
  ENTRY_CUDA(cudaMemsetAsync(w, 0, c.ws.dtable, st), "clear status and operand scales");
  ScoreArgs s;
  if ((e = prepare_scores(c, score, scale, plan, w, &s, st)) != CP_OK) return e;
  if (!c.bf16) {
    F32Args a = f32_args(c, score, plan, s, Hkv, scale);
    a.q = static_cast<const float*>(q);
    a.k = static_cast<const float*>(k);
    a.v = static_cast<const float*>(v);
    a.splits = f32_fwd_splits(*c.h);
    const bool parts = a.splits > 1;
    a.out = parts ? reinterpret_cast<float*>(w + c.ws.part_out) : static_cast<float*>(out);
    a.lse = parts ? reinterpret_cast<float*>(w + c.ws.part_lse) : lse;
    ProfileScope prof(6, st, parts ? 2 : 1);
    ENTRY_CUDA(launch_f32_fwd(a, d, st), "fp32 scored forward");
    if (parts)
      ENTRY_CUDA(launch_lse_merge(a.splits, a.out, a.lse, T, H, d, out, false, lse, st),
                 "merge of partial results");
    return CP_OK;
  }
  const void* vsrc = v;
  OpScales* sc = reinterpret_cast<OpScales*>(w + c.ws.scales);
  if (c.f16) {   // V's scaled copy
    const int64_t n = (int64_t)T * Hkv * d;
    void* v16 = w + c.ws.v16;
    ProfileScope prof(1, st, 2);
    ENTRY_CUDA(launch_absmax_bf16(&v, &n, 1, sc, st), "max |V|");
    ENTRY_CUDA(launch_to_f16_scaled(&v, &v16, &n, 1, sc, false, d, st), "f16 copy of V");
    vsrc = v16;
  }
  TcFwdArgs a{};
  const char* terr = nullptr;
  if (!make_tmap_thd(&a.tm_q_nat, q, T, H, d, 128, &terr) ||
      !make_tmap_thd(&a.tm_k_nat, k, T, Hkv, d, 128, &terr) ||
      !make_tmap_thd(&a.tm_v_nat, vsrc, T, Hkv, d, 128, &terr, c.f16))
    return entry_fail(CP_ERR_CUDA, std::string("tensor map: ") + (terr ? terr : "?"));
  a.tm_q_text = a.tm_q_nat;   // no run of these plans is rank-local
  a.tm_k_text = a.tm_k_nat;
  a.tm_v_text = a.tm_v_nat;
  a.items = reinterpret_cast<const FwdItem*>(plan + c.h->fwd);
  a.n_items = c.h->n_fwd;
  if (c.h->n_units > 0) {
    a.units = reinterpret_cast<const int32_t*>(plan + c.h->units);
    a.cta_off = a.units + c.h->n_units;
    a.n_ctas = c.h->grid;
  }
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.scale_log2 = scale * kLog2e;
  a.f16_pv = c.f16 ? 1 : 0;
  a.op_scales = c.f16 ? sc : nullptr;
  a.out = out;
  a.lse = lse;
  a.T = T;
  a.out_lo = out_lo;
  a.status = reinterpret_cast<int32_t*>(w);
  a.wait_limit = device_wait_limit();
  a.text_rows = T;
  a.isolate = 1;
  a.score = s;
  a.o_run = reinterpret_cast<float*>(w + c.ws.part_out);
  a.lse_run = reinterpret_cast<float*>(w + c.ws.part_lse);
  a.run_rows = c.h->run_rows;
  ProfileScope prof(2, st, c.h->n_joins > 0 ? 2 : 1);
  ENTRY_CUDA(launch_tc_fwd_scored(a, c.bias, st), "tensor-core scored forward");
  if (c.h->n_joins > 0)
    ENTRY_CUDA(launch_join_parts(reinterpret_cast<const Join*>(plan + c.h->joins), c.h->n_joins,
                                 a.o_run, a.lse_run, a.run_rows, H, d, T, out, out_lo, lse, st),
               "join of partial results");
  return CP_OK;
  ENTRY_CATCH
}

cp_status_t cp_attn_scored_bwd(const void* plan_h, const void* plan_d, const void* q,
                               const void* k, const void* v, const void* out, const void* out_lo,
                               const float* lse, const void* dout, cp_dtype_t dt, int T, int H,
                               int Hkv, int d, const cp_score_t* score, float scale, void* dq_out,
                               void* dk_out, void* dv_out, cp_dtype_t grad_dt, void* dbias,
                               cp_dtype_t dbias_dt, void* ws, size_t ws_bytes, void* stream) {
  ENTRY_TRY
  const void* ptrs[9] = {q, k, v, out, lse, dout, dq_out, dk_out, dv_out};
  Call c;
  cp_status_t e = check(plan_h, plan_d, ptrs, 9, dt, T, H, Hkv, d, score, scale, out_lo, ws,
                        ws_bytes, true, grad_dt == CP_BF16, &c);
  if (e != CP_OK) return e;
  if (grad_dt != CP_F32 && (grad_dt != CP_BF16 || dt != CP_BF16))
    return entry_fail(CP_ERR_DTYPE, "grad_dtype must be CP_F32, or CP_BF16 for bf16 inputs");
  if (dbias && dbias_dt != CP_F32 && dbias_dt != CP_BF16)
    return entry_fail(CP_ERR_DTYPE, "dbias_dtype must be CP_F32 or CP_BF16");
  if (dbias && c.bias != SCORE_TABLE)
    return entry_fail(CP_ERR_INVALID_ARG, "dbias without rel_bias");
  if (!aligned_to(dbias, dbias_dt == CP_BF16 ? 2 : 4))
    return entry_fail(CP_ERR_ALIGNMENT, "dbias alignment");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (dbias)
      ENTRY_CUDA(cudaMemsetAsync(dbias, 0,
                                 (size_t)H * score->n_buckets * (dbias_dt == CP_BF16 ? 2 : 4), st),
                 "clear dbias");
    return CP_OK;
  }
  int sms = 0;
  if ((e = check_gpu(c.bf16, &sms)) != CP_OK) return e;
  char* w = static_cast<char*>(ws);
  const char* plan = static_cast<const char*>(plan_d);
  // bf16 gradients are summed in fp32 in the workspace and rounded at the end
  const bool bf16_grads = grad_dt == CP_BF16;
  float* dq = static_cast<float*>(dq_out);
  float* dk = static_cast<float*>(dk_out);
  float* dv = static_cast<float*>(dv_out);
  const int kv_split = c.bf16 ? group_split(c.h->n_bwd, H, Hkv, sms) : 1;
  const int f32_split = c.bf16 ? 1 : f32_splits((int64_t)c.h->n_tiles * H, c.h->max_walk, sms);
  const bool add_dq = c.bf16 || f32_split > 1;
  const bool add_dkdv = c.bf16 ? kv_split > 1 || c.h->bwd_cut : f32_split > 1 || H > Hkv;
  // (dK and dV of whole groups come out of the tensor cores complete: straight to bf16)
  const bool bf16_dkdv = bf16_grads && !add_dkdv;
  if (bf16_grads) {
    dq = reinterpret_cast<float*>(w + c.ws.dq);
    if (add_dkdv) {
      dk = reinterpret_cast<float*>(w + c.ws.dk);
      dv = reinterpret_cast<float*>(w + c.ws.dv);
    }
  }
  const size_t zero = !bf16_grads ? c.ws.dq : add_dkdv ? c.ws.table : c.ws.dk;
  ENTRY_CUDA(cudaMemsetAsync(w, 0, zero, st), "clear status and sums");
  if (!bf16_grads && add_dq)
    ENTRY_CUDA(cudaMemsetAsync(dq, 0, (size_t)T * H * d * sizeof(float), st), "clear dq");
  if (!bf16_grads && add_dkdv) {
    ENTRY_CUDA(cudaMemsetAsync(dk, 0, (size_t)T * Hkv * d * sizeof(float), st), "clear dk");
    ENTRY_CUDA(cudaMemsetAsync(dv, 0, (size_t)T * Hkv * d * sizeof(float), st), "clear dv");
  }
  ScoreArgs s;
  if ((e = prepare_scores(c, score, scale, plan, w, &s, st)) != CP_OK) return e;
  if (c.bias == SCORE_TABLE) s.dtable = reinterpret_cast<float*>(w + c.ws.dtable);
  float* Dd = reinterpret_cast<float*>(w + c.ws.D);
  float* lse2 = reinterpret_cast<float*>(w + c.ws.lse2);
  const int64_t pitch = ld_pitch(T);
  const bool item_types = has_ranges(*c.h, dt);
  OperandRange* ranges = reinterpret_cast<OperandRange*>(w + c.ws.ranges);
  void* q16 = w + c.ws.q16;
  void* k16 = w + c.ws.k16;
  {
    ProfileScope prof(3, st, item_types ? 3 : 1);
    ENTRY_CUDA(launch_bwd_preprocess(out, out_lo, dout, c.bf16, lse, T, H, d, Dd, lse2, pitch, st),
               "bwd preprocess");
    if (item_types) {   // S, dQ and dK of short samples on f16 operands
      const Tile32* tiles = reinterpret_cast<const Tile32*>(plan + c.h->tiles);
      ENTRY_CUDA(launch_operand_ranges(tiles, c.h->n_tiles, q, k, v, dout, H, Hkv, d, ranges, st),
                 "ranges of short samples");
      ENTRY_CUDA(launch_f16_operands(tiles, c.h->n_tiles, q, k, H, Hkv, d, ranges, q16, k16, st),
                 "f16 copies of short samples");
    }
  }
  if (!c.bf16) {
    F32Args a = f32_args(c, score, plan, s, Hkv, scale);
    a.q = static_cast<const float*>(q);
    a.k = static_cast<const float*>(k);
    a.v = static_cast<const float*>(v);
    a.dout = static_cast<const float*>(dout);
    a.lse_in = lse;
    a.D = Dd;
    a.pitch_d = pitch;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dtable = s.dtable;
    a.splits = f32_split;
    a.add_dq = add_dq;
    a.add_dkdv = add_dkdv;
    ProfileScope prof(7, st, 2);
    ENTRY_CUDA(launch_f32_bwd(a, d, st), "fp32 scored backward");
  } else {
    TcBwdArgs a{};
    const char* terr = nullptr;
    if (!make_tmap_thd(&a.tm_q, q, T, H, d, 128, &terr) ||
        !make_tmap_thd(&a.tm_k, k, T, Hkv, d, kBwdTileK, &terr) ||
        (item_types && (!make_tmap_thd(&a.tm_q16, q16, T, H, d, 128, &terr, true) ||
                        !make_tmap_thd(&a.tm_k16, k16, T, Hkv, d, kBwdTileK, &terr, true))) ||
        !make_tmap_thd(&a.tm_v, v, T, Hkv, d, kBwdTileK, &terr) ||
        !make_tmap_thd(&a.tm_do, dout, T, H, d, 128, &terr) ||
        !make_tmap_ld(&a.tm_ld, lse2, pitch, H, 128 + 4, &terr) ||
        !make_tmap_f32_sw128(&a.tm_dq, dq, T, H, d, 32, &terr))
      return entry_fail(CP_ERR_CUDA, std::string("tensor map: ") + (terr ? terr : "?"));
    a.items = reinterpret_cast<const BwdItem*>(plan + c.h->bwd);
    a.runs = reinterpret_cast<const Seg*>(plan + c.h->runs);
    a.n_items = c.h->n_bwd;
    a.H = H;
    a.Hkv = Hkv;
    a.d = d;
    a.scale = scale;
    a.scale_log2 = scale * kLog2e;
    a.T = T;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dkv_bf16 = bf16_dkdv ? 1 : 0;
    a.status = reinterpret_cast<int32_t*>(w);
    a.wait_limit = device_wait_limit();
    a.kv_split = kv_split;
    a.add_dkdv = add_dkdv ? 1 : 0;
    a.isolate = 1;
    a.item_major = item_major((int64_t)c.h->n_bwd * Hkv * kv_split, sms) ? 1 : 0;
    a.ranges = item_types ? ranges : nullptr;
    a.n_samples = c.h->n_seqs;
    a.score = s;
    ProfileScope prof(4, st);
    ENTRY_CUDA(launch_tc_bwd_scored(a, c.bias, st), "tensor-core scored backward");
  }
  if (bf16_grads) {
    const float* const src[3] = {dq, dk, dv};
    void* const dst[3] = {dq_out, dk_out, dv_out};
    const int64_t nkv = bf16_dkdv ? 0 : (int64_t)T * Hkv * d;
    const int64_t n[3] = {(int64_t)T * H * d, nkv, nkv};
    ENTRY_CUDA(launch_cast_bf16(src, dst, n, sms, st), "bf16 gradients");
  }
  if (dbias)
    ENTRY_CUDA(launch_reduce_dbias(s.dtable, reinterpret_cast<const int32_t*>(plan + c.h->buckets),
                                   s.n_dist, score->n_buckets, H, dbias, dbias_dt == CP_BF16, st),
               "bias gradient by bucket");
  return CP_OK;
  ENTRY_CATCH
}

}  // extern "C"
