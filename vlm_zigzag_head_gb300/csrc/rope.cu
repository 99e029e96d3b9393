// Rotation of every query and key head by its position, in one pass over q and k.
//
//   for rotated pair p of axis a, with angle t = pos[a] * freq_p and amplitude m:
//       (y_i, y_j) = m (x_i cos t - x_j sin t, x_j cos t + x_i sin t),
//   (i, j) = (p, p + rot / 2), or (2p, 2p + 1) when interleaved; elements from
//   rot on are copied as they are.
// The gradient is the same map with the angles turned round.
//
// Bound by memory: every element is read and written once.  A lane owns two
// groups of four elements that rotate against one another, so the rotation needs
// no exchange between lanes, and it has read both before it writes either: the
// output may be the input.  The cosines and sines of a token are worked out once
// by the warp that takes its heads.
#include <type_traits>

#include "rope.cuh"

namespace cpattn {

namespace {

constexpr int kWarps = 8;

// Four elements from memory that this launch may also write (in place), so not
// through the read-only path.
template <bool kVec>
__device__ __forceinline__ void load_shared(Raw<__nv_bfloat16>& r, const __nv_bfloat16* p) {
  if constexpr (kVec)
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(r.v.x), "=r"(r.v.y)
                 : "l"(p));
  else r.template load<false>(p);
}
template <bool kVec>
__device__ __forceinline__ void load_shared(Raw<float>& r, const float* p) {
  if constexpr (kVec)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.v.x), "=r"(r.v.y), "=r"(r.v.z), "=r"(r.v.w)
                 : "l"(p));
  else r.template load<false>(p);
}

// Raw elements as they are.
template <bool kVec>
__device__ __forceinline__ void store_raw(__nv_bfloat16* p, uint2 v) {
  if constexpr (kVec) {
    *reinterpret_cast<uint2*>(p) = v;
  } else {
    unsigned short* s = reinterpret_cast<unsigned short*>(p);
    s[0] = (unsigned short)v.x;
    s[1] = (unsigned short)(v.x >> 16);
    s[2] = (unsigned short)v.y;
    s[3] = (unsigned short)(v.y >> 16);
  }
}
template <bool kVec>
__device__ __forceinline__ void store_raw(float* p, uint4 v) {
  if constexpr (kVec) {
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    uint32_t* s = reinterpret_cast<uint32_t*>(p);
    s[0] = v.x;
    s[1] = v.y;
    s[2] = v.z;
    s[3] = v.w;
  }
}
__device__ __forceinline__ void round_to(uint2& v, const Four& f) {
  float a, b, c, d;
  unpack2(f.p[0], a, b);
  unpack2(f.p[1], c, d);
  v = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}
__device__ __forceinline__ void round_to(uint4& v, const Four& f) {
  float a, b, c, d;
  unpack2(f.p[0], a, b);
  unpack2(f.p[1], c, d);
  v = make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}

// One warp: heads [g0, g1) of one token (query heads first, then key heads).
template <typename T, int D, bool kInter, bool kVec>
__global__ void __launch_bounds__(kWarps * 32, 4)
    rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 cs_all[kWarps][64];
  using G = Lane<D, kInter>;
  constexpr int kUnroll = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = unit / a.n_chunks;
  if (t >= a.T) return;   // whole warps only: the block has no barrier
  const int g0 = (int)(unit % a.n_chunks) * a.chunk, g1 = g0 + a.chunk;
  const G ln(lane, a.rot);
  const bool turned = ln.pair >= 0;
  const int gap = ln.e1 - ln.e0;
  float2* cs = cs_all[warp];
  uint64_t c[4], sn[4];
  bool angles = false;
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    // the chunk's heads of this tensor
    const int h0 = max(0, g0 - (s ? a.heads[0] : 0));
    const int h1 = min(a.heads[s], g1 - (s ? a.heads[0] : 0));
    if (h0 >= h1) continue;
    // running pointers to this lane's elements of the pass's head
    const int64_t step = G::kHeads * a.sh[s], ystep = G::kHeads * a.ysh[s];
    int h = h0 + ln.sel, hn = h;   // head of the pass, and of the next load
    const T* src = static_cast<const T*>(a.x[s]) + t * a.st[s] + h * a.sh[s] + ln.e0;
    T* dst = static_cast<T*>(a.y[s]) + t * a.yst[s] + h * a.ysh[s] + ln.e0;
    Raw<T> rx[kUnroll], rz[kUnroll];
    auto load = [&](int u) {
      if (hn < h1) {
        load_shared<kVec>(rx[u], src);
        load_shared<kVec>(rz[u], src + gap);
      }
      hn += G::kHeads;
      src += step;
    };
    // the first heads' loads go out before the angles are computed
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      rx[u].clear();
      rz[u].clear();
      load(u);
    }
    if (!angles) {
      token_angles(a, t, lane, cs);
      __syncwarp();
      ln.coefficients(cs, c, sn);
      const uint64_t m = pack2(a.amp, a.amp), ms = pack2(a.sin_amp, a.sin_amp);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!kInter && i >= 2) break;   // the half layout has two pairs of coefficients
        c[i] = mul2(c[i], m);
        sn[i] = mul2(sn[i], ms);
      }
      angles = true;
    }
    const uint64_t neg = pack2(-1.f, -1.f);
    for (int hb = h0; hb < h1; hb += kUnroll * G::kHeads) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        Raw<T> ox = rx[u], oz = rz[u];
        const Four x = ox.get(), z = oz.get();
        load(u);
        if (turned) {   // others stay as they are, to the bit
          const uint64_t v[4] = {x.p[0], x.p[1], z.p[0], z.p[1]};
          uint64_t y[4];
          if constexpr (kInter) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = fma2(swap2(v[i]), sn[i], mul2(v[i], c[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              y[i] = fma2(mul2(v[2 + i], neg), sn[i], mul2(v[i], c[i]));
              y[2 + i] = fma2(v[i], sn[i], mul2(v[2 + i], c[i]));
            }
          }
          round_to(ox.v, {{y[0], y[1]}});
          round_to(oz.v, {{y[2], y[3]}});
        }
        if (h < h1) {
          store_raw<kVec>(dst, ox.v);
          store_raw<kVec>(dst + gap, oz.v);
        }
        h += G::kHeads;
        dst += ystep;
      }
    }
  }
}

template <typename T, int D, bool kInter, bool kVec>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.T * a.n_chunks + kWarps - 1) / kWarps;
  rope_kernel<T, D, kInter, kVec><<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_d(const RopeArgs& a, bool inter, bool vec, cudaStream_t st) {
  if (inter) return vec ? launch_t<T, D, true, true>(a, st) : launch_t<T, D, true, false>(a, st);
  return vec ? launch_t<T, D, false, true>(a, st) : launch_t<T, D, false, false>(a, st);
}

}  // namespace

void rope_split(int64_t T, int heads, int d, int sms, int* chunk, int* n_chunks) {
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

cudaError_t launch_rope(const RopeArgs& a, bool bf16, int d, bool interleaved, bool vec,
                        cudaStream_t st) {
  if (bf16)
    return d == 64 ? launch_d<__nv_bfloat16, 64>(a, interleaved, vec, st)
                   : launch_d<__nv_bfloat16, 128>(a, interleaved, vec, st);
  return d == 64 ? launch_d<float, 64>(a, interleaved, vec, st)
                 : launch_d<float, 128>(a, interleaved, vec, st);
}

}  // namespace cpattn
