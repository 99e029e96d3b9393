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
// backward reads x and dy and writes dx (r and the angles are recomputed).  To
// stay there a pass has few instructions per element: a lane owns two groups of
// four elements that rotate against one another (elements 4 l and rot / 2 + 4 l
// on), so that the rotation needs no exchange between lanes; d / 8 lanes share a
// head; the cosines, sines and weights of a lane's elements are multiplied once
// per token into the coefficients that every head of the token uses; arithmetic
// runs two elements per instruction.  Several heads are loaded before the first
// is used, to cover the memory latency.  Measured on bf16 heads of 128: forward
// 6.7 TB/s at 131072 tokens x 40 heads and 6.1 at 18688 x 64 (a plain copy: 6.8);
// backward 5.8 and 5.4 with two blocks of eight warps per SM (5.5 and 5.0 with
// three, whose 80 registers leave fewer loads in flight).
#include <type_traits>

#include "norm_rope.h"
#include "rope.cuh"

namespace cpattn {

namespace {

using namespace ptx;

constexpr int kWarps = 8;

__device__ __forceinline__ Four load_weights(const NormRopeArgs& a, int s, int e) {
  float w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = a.w[s] == nullptr ? 1.f
           : a.w_bf16        ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.w[s])[e + i])
                             : static_cast<const float*>(a.w[s])[e + i];
  }
  return {{pack2(w[0], w[1]), pack2(w[2], w[3])}};
}

template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float sum2(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}

// The forward's coefficients with the weights folded in: y = r (x A + other B).
template <int D, bool kInter>
struct Turn {
  uint64_t A[4], B[4];
  __device__ __forceinline__ Turn(const Lane<D, kInter>& ln, const float2* cs, const Four& wx,
                                  const Four& wz) {
    uint64_t c[4], s[4];
    ln.coefficients(cs, c, s);
    if constexpr (kInter) {
      const uint64_t w[4] = {wx.p[0], wx.p[1], wz.p[0], wz.p[1]};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        A[i] = mul2(w[i], c[i]);
        B[i] = mul2(swap2(w[i]), s[i]);   // of the pair's other element
      }
    } else {
      const uint64_t neg = pack2(-1.f, -1.f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        A[i] = mul2(wx.p[i], c[i]);
        A[2 + i] = mul2(wz.p[i], c[i]);
        B[i] = mul2(mul2(wz.p[i], s[i]), neg);
        B[2 + i] = mul2(wx.p[i], s[i]);
      }
    }
  }
  __device__ __forceinline__ void apply(const Four& x, const Four& z, float r, Four& y0,
                                        Four& y1) const {
    const uint64_t r2 = pack2(r, r);
    const uint64_t v[4] = {x.p[0], x.p[1], z.p[0], z.p[1]};
    uint64_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t other = kInter ? swap2(v[i]) : v[i ^ 2];
      y[i] = mul2(fma2(other, B[i], mul2(v[i], A[i])), r2);
    }
    y0 = {{y[0], y[1]}};
    y1 = {{y[2], y[3]}};
  }
};

// One warp: heads [g0, g1) of one token (query heads first, then key heads).
template <typename T, int D, bool kInter, bool kVec>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 4 : 2)
    norm_rope_fwd_kernel(const __grid_constant__ NormRopeArgs a) {
  __shared__ float2 cs_all[kWarps][64];
  using G = Lane<D, kInter>;
  constexpr int kUnroll = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = unit / a.n_chunks;
  if (t >= a.T) return;   // whole warps only: the block has no barrier
  const int g0 = (int)(unit % a.n_chunks) * a.chunk, g1 = g0 + a.chunk;
  const G ln(lane, a.rot);
  float2* cs = cs_all[warp];
  bool angles = false;
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    // the chunk's heads of this tensor
    const int h0 = max(0, g0 - (s ? a.heads[0] : 0));
    const int h1 = min(a.heads[s], g1 - (s ? a.heads[0] : 0));
    if (h0 >= h1) continue;
    // running pointers to this lane's elements of the pass's head
    const int64_t step = G::kHeads * a.sh[s];
    const int gap = ln.e1 - ln.e0;
    int h = h0 + ln.sel, hn = h;   // head of the pass, and of the next load
    const T* src = static_cast<const T*>(a.x[s]) + t * a.st[s] + h * a.sh[s] + ln.e0;
    T* dst = static_cast<T*>(a.y[s]) + (t * a.heads[s] + h) * D + ln.e0;
    // the first heads' loads go out before the angles are computed
    Raw<T> rx[kUnroll], rz[kUnroll];
    auto load = [&](int u) {
      if (hn < h1) {
        rx[u].template load<kVec>(src);
        rz[u].template load<kVec>(src + gap);
      }
      hn += G::kHeads;
      src += step;
    };
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      rx[u].clear();
      rz[u].clear();
      load(u);
    }
    if (!angles) {
      token_angles(a, t, lane, cs);
      __syncwarp();
      angles = true;
    }
    const Turn<D, kInter> turn(ln, cs, load_weights(a, s, ln.e0), load_weights(a, s, ln.e1));
    for (int hb = h0; hb < h1; hb += kUnroll * G::kHeads) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const Four x = rx[u].get(), z = rz[u].get();
        load(u);
        uint64_t ss = mul2(x.p[0], x.p[0]);
        ss = fma2(x.p[1], x.p[1], ss);
        ss = fma2(z.p[0], z.p[0], ss);
        ss = fma2(z.p[1], z.p[1], ss);
        const float r = rsqrtf(head_sum<G::kLanes>(sum2(ss)) * (1.f / D) + a.eps);
        Four y0, y1;
        turn.apply(x, z, r, y0, y1);
        if (h < h1) {
          store4(dst, y0);
          store4(dst + gap, y1);
        }
        h += G::kHeads;
        dst += G::kHeads * D;
      }
    }
  }
}

// Warps walk (token, chunk) units gridDim.x * kWarps apart and keep the weight
// gradients of their lane's elements in registers; a block adds its warps' in
// warp order and writes one row of partial sums, which a second small launch
// adds in block order: the result does not depend on timing.
template <typename T, int D, bool kInter, bool kVec>
__global__ void __launch_bounds__(kWarps * 32, 2)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a) {
  __shared__ float2 cs_all[kWarps][64];
  __shared__ float red[kWarps][2][D];
  using G = Lane<D, kInter>;
  constexpr int kUnroll = 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const G ln(lane, a.rot);
  float2* cs = cs_all[warp];
  uint64_t dw[2][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i / 4][i % 4] = pack2(0.f, 0.f);
  const int64_t units = a.T * a.n_chunks;
  for (int64_t unit = (int64_t)blockIdx.x * kWarps + warp; unit < units;
       unit += (int64_t)gridDim.x * kWarps) {
    const int64_t t = unit / a.n_chunks;
    const int g0 = (int)(unit % a.n_chunks) * a.chunk, g1 = g0 + a.chunk;
    __syncwarp();   // the previous token's angles are read
    bool angles = false;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int h0 = max(0, g0 - (s ? a.heads[0] : 0));
      const int h1 = min(a.heads[s], g1 - (s ? a.heads[0] : 0));
      if (h0 >= h1) continue;
      const int64_t step = G::kHeads * a.sh[s];
      const int gap = ln.e1 - ln.e0;
      int h = h0 + ln.sel, hn = h;   // head of the pass, and of the next load
      const int64_t row = (t * a.heads[s] + h) * D + ln.e0;
      const T* src = static_cast<const T*>(a.x[s]) + t * a.st[s] + h * a.sh[s] + ln.e0;
      const T* gsrc = static_cast<const T*>(a.dy[s]) + row;
      T* dst = static_cast<T*>(a.y[s]) + row;
      Raw<T> rx[kUnroll], rz[kUnroll], rgx[kUnroll], rgz[kUnroll];
      auto load = [&](int u) {
        if (hn < h1) {
          rx[u].template load<kVec>(src);
          rz[u].template load<kVec>(src + gap);
          rgx[u].template load<true>(gsrc);
          rgz[u].template load<true>(gsrc + gap);
        }
        hn += G::kHeads;
        src += step;
        gsrc += G::kHeads * D;
      };
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        rx[u].clear();
        rz[u].clear();
        rgx[u].clear();
        rgz[u].clear();
        load(u);
      }
      if (!angles) {
        token_angles(a, t, lane, cs);
        __syncwarp();
        angles = true;
      }
      uint64_t c[4], sn[4];
      ln.coefficients(cs, c, sn);
      const Four wx = load_weights(a, s, ln.e0), wz = load_weights(a, s, ln.e1);
      const uint64_t w[4] = {wx.p[0], wx.p[1], wz.p[0], wz.p[1]};
      const uint64_t neg = pack2(-1.f, -1.f);
      for (int hb = h0; hb < h1; hb += kUnroll * G::kHeads) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const Four x0 = rx[u].get(), x1 = rz[u].get(), d0 = rgx[u].get(), d1 = rgz[u].get();
          load(u);
          const uint64_t x[4] = {x0.p[0], x0.p[1], x1.p[0], x1.p[1]};
          const uint64_t dy[4] = {d0.p[0], d0.p[1], d1.p[0], d1.p[1]};
          // g = R^T dy
          uint64_t g[4], gx[4];
          if constexpr (kInter) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              g[i] = fma2(mul2(swap2(dy[i]), sn[i]), neg, mul2(dy[i], c[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              g[i] = fma2(dy[2 + i], sn[i], mul2(dy[i], c[i]));
              g[2 + i] = fma2(mul2(dy[i], sn[i]), neg, mul2(dy[2 + i], c[i]));
            }
          }
          uint64_t ss = mul2(x[0], x[0]), dot = pack2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i > 0) ss = fma2(x[i], x[i], ss);
            gx[i] = mul2(g[i], x[i]);
            dot = fma2(gx[i], w[i], dot);
          }
          const float r = rsqrtf(head_sum<G::kLanes>(sum2(ss)) * (1.f / D) + a.eps);
          // n mean(g w n) = x r^2 mean(g w x)
          const float k = head_sum<G::kLanes>(sum2(dot)) * (1.f / D) * r * r;
          if (h < h1) {
            const uint64_t r2 = pack2(r, r), k2 = pack2(-k, -k);
            uint64_t dx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              dw[s][i] = fma2(gx[i], r2, dw[s][i]);
              dx[i] = mul2(fma2(x[i], k2, mul2(g[i], w[i])), r2);
            }
            store4(dst, {{dx[0], dx[1]}});
            store4(dst + gap, {{dx[2], dx[3]}});
          }
          h += G::kHeads;
          dst += G::kHeads * D;
        }
      }
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[2];
      unpack2(dw[s][i], v[0], v[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int o = G::kLanes; o < 32; o <<= 1)   // the heads of one pass
          v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
        if (ln.sel == 0) red[warp][s][(i < 2 ? ln.e0 : ln.e1) + (i & 1) * 2 + j] = v[j];
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

// 32 outputs per block; a warp adds the rows of its share, then the warps' sums
// meet in warp order.
constexpr int kDwWarps = 32;
__global__ void __launch_bounds__(kDwWarps * 32)
    norm_rope_dw_kernel(const float* partial, int blocks, int d, float* dqw, float* dkw) {
  __shared__ float red[kDwWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
#pragma unroll 4
  for (int b = warp; b < blocks; b += kDwWarps) v += partial[(int64_t)b * 2 * d + col];
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int g = 1; g < kDwWarps; ++g) v += red[g][lane];
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
  norm_rope_dw_kernel<<<2 * d / 32, kDwWarps * 32, 0, st>>>(partial, blocks, d, dqw, dkw);
  return cudaGetLastError();
}

}  // namespace cpattn
