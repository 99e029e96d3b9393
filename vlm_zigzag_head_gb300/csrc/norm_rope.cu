// RMS norm of every query and key head and the position rotation, in one pass
// over q and k, and its gradient.
//
//   r = 1 / sqrt(mean_e x_e^2 + eps),  n = x r,  z = n w
//   y = R z: for rotated pair p of axis a with angle t = pos[a] * freq_p,
//       (y_i, y_j) = (z_i cos t - z_j sin t, z_j cos t + z_i sin t),
//   (i, j) = (p, p + rot / 2), or (2p, 2p + 1) when interleaved; elements from
//   rot on are not rotated.
// Gradient, with g = R^T dy:
//   dw_e = sum over rows of g_e n_e,   dx = r (g w - n mean_e(g w n)).
//
// The passes are bound by memory: forward reads and writes every element once,
// backward reads x and dy and writes dx (r and the angles are recomputed).  So
// a lane moves eight neighbouring elements (16 bytes of bf16), d / 8 lanes
// share a head, and a warp keeps the cosines, sines and weights of its lane's
// elements in registers while it walks the heads of one token: the angles cost
// one evaluation per token and pair, not per head.  Several heads are loaded
// before the first is used, to cover the memory latency.
//
// Angles.  A 32-bit product pos * freq is off by 2^-24 of the angle, which at
// position 100000 is 0.006 radians.  The turns per position are therefore held
// as a 64-bit fraction of 2^64; the integer product with the position drops
// whole turns exactly, and its upper 32 bits are the angle to 2^-32 of a turn.
#include <cuda_bf16.h>

#include <type_traits>

#include "norm_rope.h"

namespace cpattn {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Eight elements as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
  template <bool kVec>
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    if constexpr (kVec) {
      v = ld_stream(p);
    } else {
      const unsigned short* s = reinterpret_cast<const unsigned short*>(p);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (uint32_t)s[2 * i] | ((uint32_t)s[2 * i + 1] << 16);
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // a bf16 is the upper half of its fp32
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  uint4 v[2];
  __device__ __forceinline__ void clear() { v[0] = v[1] = make_uint4(0, 0, 0, 0); }
  template <bool kVec>
  __device__ __forceinline__ void load(const float* p) {
    if constexpr (kVec) {
      v[0] = ld_stream(p);
      v[1] = ld_stream(p + 4);
    } else {
      const uint32_t* s = reinterpret_cast<const uint32_t*>(p);
      v[0] = make_uint4(s[0], s[1], s[2], s[3]);
      v[1] = make_uint4(s[4], s[5], s[6], s[7]);
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
};

// Outputs are contiguous and 16-byte aligned.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ void load_weights(const NormRopeArgs& a, int s, int e0, float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = a.w[s] == nullptr ? 1.f
           : a.w_bf16        ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.w[s])[e0 + i])
                             : static_cast<const float*>(a.w[s])[e0 + i];
  }
}

// Cosine and sine of every rotated pair of token t into the warp's table.
__device__ __forceinline__ void token_angles(const NormRopeArgs& a, int64_t t, int lane,
                                             float2* cs) {
  for (int p = lane; p < a.rot / 2; p += 32) {
    int ax = 0;
#pragma unroll
    for (int i = 0; i < kRopeMaxAxes - 1; ++i) ax += i + 1 < a.n_axes && p >= a.sec_end[i];
    const int64_t pos = a.pos[ax * a.T + t];
    const uint64_t turns = (uint64_t)pos * a.freq[p];   // whole turns wrap away
    // upper half as a signed fraction: half turns in [-1, 1)
    const float half_turns = (float)(int32_t)(turns >> 32) * (1.f / 2147483648.f);
    float s, c;
    sincospif(half_turns, &s, &c);
    cs[p] = make_float2(c, s);
  }
}

// The lane's rotation: element i of the rotated head is z_i c[i] + partner_i s[i].
// Half layout: the partner elements sit `shift` lanes away (rot / 2 elements);
// interleaved: the partner of an even element is the next one.
template <bool kInter>
__device__ __forceinline__ void lane_rotation(const float2* cs, int e0, int rot, float (&c)[8],
                                              float (&s)[8]) {
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const bool in = e0 < rot;
      const float2 v = in ? cs[(e0 + i) / 2] : make_float2(1.f, 0.f);
      c[i] = c[i + 1] = v.x;
      s[i] = -v.y;
      s[i + 1] = v.y;
    }
  } else {
    const int half = rot / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = e0 < rot;
      const float2 v = in ? cs[e0 < half ? e0 + i : e0 + i - half] : make_float2(1.f, 0.f);
      c[i] = v.x;
      s[i] = e0 < half ? -v.y : v.y;
    }
  }
}

// y = R z, or R^T z with kBack (the sines change sign).
template <bool kInter, bool kBack>
__device__ __forceinline__ void rotate(const float (&z)[8], const float (&c)[8],
                                       const float (&s)[8], int partner, float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float other = kInter ? z[i ^ 1] : __shfl_sync(0xffffffffu, z[i], partner);
    y[i] = fmaf(other, kBack ? -s[i] : s[i], z[i] * c[i]);
  }
}

template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Geometry shared by both directions: where lane's elements of head g live.
template <int D>
struct Lane {
  static constexpr int kLanes = D / 8;          // lanes of one head
  static constexpr int kHeads = 32 / kLanes;    // heads of one warp pass
  int e0, sel, partner;
  __device__ __forceinline__ Lane(int lane, int rot) {
    const int sub = lane % kLanes;
    e0 = sub * 8;
    sel = lane / kLanes;
    const int shift = rot / 16;                 // rot / 2 elements, in lanes
    int p = e0 < rot / 2 ? sub + shift : sub - shift;
    if (e0 >= rot) p = sub;
    partner = sel * kLanes + p;
  }
};

// One warp: heads [g0, g1) of one token (query heads first, then key heads).
template <typename T, int D, bool kInter, bool kVec>
__global__ void __launch_bounds__(kWarps * 32)
    norm_rope_fwd_kernel(const __grid_constant__ NormRopeArgs a) {
  __shared__ float2 cs_all[kWarps][64];
  using G = Lane<D>;
  constexpr int kUnroll = sizeof(T) == 2 ? 4 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = unit / a.n_chunks;
  if (t >= a.T) return;   // whole warps only: the block has no barrier
  const int total = a.heads[0] + a.heads[1];
  const int g0 = (int)(unit % a.n_chunks) * a.chunk;
  const int g1 = min(g0 + a.chunk, total);
  const G ln(lane, a.rot);
  auto src = [&](int g) {
    const int s = g >= a.heads[0];
    return static_cast<const T*>(a.x[s]) + t * a.st[s] +
           (int64_t)(g - (s ? a.heads[0] : 0)) * a.sh[s] + ln.e0;
  };
  // the first heads' loads go out before the angles are computed
  Raw<T> raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int g = g0 + u * G::kHeads + ln.sel;
    raw[u].clear();
    if (g < g1) raw[u].template load<kVec>(src(g));
  }
  float2* cs = cs_all[warp];
  token_angles(a, t, lane, cs);
  __syncwarp();
  float c[8], s[8], wq[8], wk[8];
  lane_rotation<kInter>(cs, ln.e0, a.rot, c, s);
  load_weights(a, 0, ln.e0, wq);
  load_weights(a, 1, ln.e0, wk);
  for (int gb = g0; gb < g1; gb += kUnroll * G::kHeads) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int g = gb + u * G::kHeads + ln.sel;
      float x[8];
      raw[u].get(x);
      const int gn = g + kUnroll * G::kHeads;
      raw[u].clear();
      if (gn < g1) raw[u].template load<kVec>(src(gn));
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
      const float r = rsqrtf(head_sum<G::kLanes>(ss) * (1.f / D) + a.eps);
      const bool is_k = g >= a.heads[0];
      float z[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = x[i] * r * (is_k ? wk[i] : wq[i]);
      rotate<kInter, false>(z, c, s, ln.partner, y);
      if (g < g1) {
        T* dst = is_k ? static_cast<T*>(a.y[1]) + (t * a.heads[1] + g - a.heads[0]) * D
                      : static_cast<T*>(a.y[0]) + (t * a.heads[0] + g) * D;
        store8(dst + ln.e0, y);
      }
    }
  }
}

// Warps walk (token, chunk) units gridDim.x * kWarps apart and keep the weight
// gradients of their lane's elements in registers; a block adds its warps' in
// warp order and writes one row of partial sums, which a second small launch
// adds in block order: the result does not depend on timing.
template <typename T, int D, bool kInter, bool kVec>
__global__ void __launch_bounds__(kWarps * 32)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a) {
  __shared__ float2 cs_all[kWarps][64];
  __shared__ float red[kWarps][2][D];
  using G = Lane<D>;
  constexpr int kUnroll = sizeof(T) == 2 ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int total = a.heads[0] + a.heads[1];
  const G ln(lane, a.rot);
  float2* cs = cs_all[warp];
  float wq[8], wk[8], dwq[8], dwk[8];
  load_weights(a, 0, ln.e0, wq);
  load_weights(a, 1, ln.e0, wk);
#pragma unroll
  for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.f;
  const int64_t units = a.T * a.n_chunks;
  for (int64_t unit = (int64_t)blockIdx.x * kWarps + warp; unit < units;
       unit += (int64_t)gridDim.x * kWarps) {
    const int64_t t = unit / a.n_chunks;
    const int g0 = (int)(unit % a.n_chunks) * a.chunk;
    const int g1 = min(g0 + a.chunk, total);
    auto load = [&](int g, Raw<T>& rx, Raw<T>& rg) {
      rx.clear();
      rg.clear();
      if (g < g1) {
        const int s = g >= a.heads[0];
        const int h = g - (s ? a.heads[0] : 0);
        rx.template load<kVec>(static_cast<const T*>(a.x[s]) + t * a.st[s] +
                               (int64_t)h * a.sh[s] + ln.e0);
        rg.template load<true>(static_cast<const T*>(a.dy[s]) +
                               (t * a.heads[s] + h) * D + ln.e0);
      }
    };
    Raw<T> rx[kUnroll], rg[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load(g0 + u * G::kHeads + ln.sel, rx[u], rg[u]);
    __syncwarp();   // the previous token's angles are read
    token_angles(a, t, lane, cs);
    __syncwarp();
    float c[8], s[8];
    lane_rotation<kInter>(cs, ln.e0, a.rot, c, s);
    for (int gb = g0; gb < g1; gb += kUnroll * G::kHeads) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int g = gb + u * G::kHeads + ln.sel;
        float x[8], dy[8], gr[8];
        rx[u].get(x);
        rg[u].get(dy);
        load(g + kUnroll * G::kHeads, rx[u], rg[u]);
        rotate<kInter, true>(dy, c, s, ln.partner, gr);
        const bool is_k = g >= a.heads[0];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(x[i], x[i], ss);
          dot = fmaf(gr[i] * (is_k ? wk[i] : wq[i]), x[i], dot);
        }
        const float r = rsqrtf(head_sum<G::kLanes>(ss) * (1.f / D) + a.eps);
        // mean of (g w) n = r * mean of (g w) x
        const float m = head_sum<G::kLanes>(dot) * (1.f / D) * r;
        float dx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = x[i] * r;
          const float gn = g < g1 ? gr[i] * n : 0.f;
          dwq[i] += is_k ? 0.f : gn;
          dwk[i] += is_k ? gn : 0.f;
          dx[i] = r * fmaf(gr[i], is_k ? wk[i] : wq[i], -n * m);
        }
        if (g < g1) {
          T* dst = is_k ? static_cast<T*>(a.y[1]) + (t * a.heads[1] + g - a.heads[0]) * D
                        : static_cast<T*>(a.y[0]) + (t * a.heads[0] + g) * D;
          store8(dst + ln.e0, dx);
        }
      }
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = G::kLanes; o < 32; o <<= 1) {   // the heads of one pass
      dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
      dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
    }
    if (ln.sel == 0) {
      red[warp][0][ln.e0 + i] = dwq[i];
      red[warp][1][ln.e0 + i] = dwk[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][i / D][i % D];
    a.partial[(int64_t)blockIdx.x * 2 * D + i] = v;
  }
}

// One warp column per output: 32 columns x 8 row groups per block.
__global__ void __launch_bounds__(256)
    norm_rope_dw_kernel(const float* partial, int blocks, int d, float* dqw, float* dkw) {
  __shared__ float red[8][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), grp = threadIdx.x >> 5;
  float v = 0.f;
  for (int b = grp; b < blocks; b += 8) v += partial[(int64_t)b * 2 * d + col];
  red[grp][threadIdx.x & 31] = v;
  __syncthreads();
  if (grp == 0) {
    for (int g = 1; g < 8; ++g) v += red[g][threadIdx.x & 31];
    if (col < d) { if (dqw) dqw[col] = v; }
    else if (dkw) dkw[col - d] = v;
  }
}

template <typename T, int D, bool kInter, bool kVec>
cudaError_t fwd_t(const NormRopeArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.T * a.n_chunks + kWarps - 1) / kWarps;
  norm_rope_fwd_kernel<T, D, kInter, kVec><<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int D, bool kInter, bool kVec>
cudaError_t bwd_t(const NormRopeArgs& a, int blocks, cudaStream_t st) {
  norm_rope_bwd_kernel<T, D, kInter, kVec><<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

// f(T{}, head size, interleaved, vec), the last three as integral constants
template <typename F>
cudaError_t dispatch(bool bf16, int d, bool inter, bool vec, F f) {
  auto by_vec = [&](auto t, auto dd, auto i) {
    return vec ? f(t, dd, i, std::true_type{}) : f(t, dd, i, std::false_type{});
  };
  auto by_inter = [&](auto t, auto dd) {
    return inter ? by_vec(t, dd, std::true_type{}) : by_vec(t, dd, std::false_type{});
  };
  auto by_d = [&](auto t) {
    return d == 64 ? by_inter(t, std::integral_constant<int, 64>{})
                   : by_inter(t, std::integral_constant<int, 128>{});
  };
  return bf16 ? by_d(__nv_bfloat16{}) : by_d(float{});
}

}  // namespace

void norm_rope_split(int64_t T, int heads, int d, int sms, int* chunk, int* n_chunks) {
  // A token's heads stay with one warp (its angles are computed once) unless
  // that leaves fewer than 32 warps per SM; then they are shared out, down to
  // one pass per warp.
  const int per_pass = 32 / (d / 8);
  const int passes = (heads + per_pass - 1) / per_pass;
  const int64_t want = 32LL * sms;
  int64_t n = (want + T - 1) / T;
  if (n > passes) n = passes;
  const int each = (passes + (int)n - 1) / (int)n;
  *chunk = each * per_pass;
  *n_chunks = (passes + each - 1) / each;
}

int norm_rope_bwd_max_blocks(int sms) { return 2 * sms; }   // resident blocks

int norm_rope_bwd_blocks(int64_t T, int n_chunks, int sms) {
  const int64_t need = (T * n_chunks + kWarps - 1) / kWarps;
  const int64_t most = norm_rope_bwd_max_blocks(sms);
  return (int)(need < most ? need : most);
}

cudaError_t launch_norm_rope_fwd(const NormRopeArgs& a, bool bf16, int d, bool interleaved,
                                 bool vec, cudaStream_t st) {
  return dispatch(bf16, d, interleaved, vec, [&](auto t, auto dd, auto i, auto v) {
    return fwd_t<decltype(t), decltype(dd)::value, decltype(i)::value, decltype(v)::value>(a, st);
  });
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, bool bf16, int d, bool interleaved,
                                 bool vec, int blocks, cudaStream_t st) {
  return dispatch(bf16, d, interleaved, vec, [&](auto t, auto dd, auto i, auto v) {
    return bwd_t<decltype(t), decltype(dd)::value, decltype(i)::value, decltype(v)::value>(
        a, blocks, st);
  });
}

cudaError_t launch_norm_rope_dw(const float* partial, int blocks, int d, float* dqw, float* dkw,
                                cudaStream_t st) {
  norm_rope_dw_kernel<<<2 * d / 32, 256, 0, st>>>(partial, blocks, d, dqw, dkw);
  return cudaGetLastError();
}

}  // namespace cpattn
