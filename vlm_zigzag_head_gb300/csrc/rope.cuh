// Pieces of the kernels that rotate query and key heads: loads and stores of
// four elements, the angles of a token, and where a lane's elements of a head lie.
//
// Angles.  A 32-bit product pos * freq is off by 2^-24 of the angle, which at
// position 100000 is 0.006 radians.  The turns per position are therefore held
// as a 64-bit fraction of 2^64; the integer product with the position drops
// whole turns exactly, and its upper 32 bits are the angle to 2^-32 of a turn.
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "rope.h"

namespace cpattn {

namespace {

using namespace ptx;

// Four elements as two pairs of floats, and their load as stored.
struct Four {
  uint64_t p[2];
};
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void clear() { v = make_uint2(0, 0); }
  template <bool kVec>
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    if constexpr (kVec) {
      asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                   : "=r"(v.x), "=r"(v.y)
                   : "l"(p));
    } else {
      const unsigned short* s = reinterpret_cast<const unsigned short*>(p);
      v = make_uint2((uint32_t)s[0] | ((uint32_t)s[1] << 16),
                     (uint32_t)s[2] | ((uint32_t)s[3] << 16));
    }
  }
  __device__ __forceinline__ Four get() const {   // a bf16 is the upper half of its fp32
    return {{pack2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u)),
             pack2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u))}};
  }
};
template <>
struct Raw<float> {
  uint4 v;
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
  template <bool kVec>
  __device__ __forceinline__ void load(const float* p) {
    if constexpr (kVec) {
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "l"(p));
    } else {
      const uint32_t* s = reinterpret_cast<const uint32_t*>(p);
      v = make_uint4(s[0], s[1], s[2], s[3]);
    }
  }
  __device__ __forceinline__ Four get() const {
    return {{pack2(__uint_as_float(v.x), __uint_as_float(v.y)),
             pack2(__uint_as_float(v.z), __uint_as_float(v.w))}};
  }
};

// Outputs are contiguous and 16-byte aligned.
__device__ __forceinline__ void store4(__nv_bfloat16* p, const Four& f) {
  float a, b, c, d;
  unpack2(f.p[0], a, b);
  unpack2(f.p[1], c, d);
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}
__device__ __forceinline__ void store4(float* p, const Four& f) {
  float4 v;
  unpack2(f.p[0], v.x, v.y);
  unpack2(f.p[1], v.z, v.w);
  *reinterpret_cast<float4*>(p) = v;
}

__device__ __forceinline__ uint64_t swap2(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return pack2(b, a);
}

// Cosine and sine of every rotated pair of token t into the warp's table.
__device__ __forceinline__ void token_angles(const RopeAngles& a, int64_t t, int lane,
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

// Where a lane's elements of a head live: two groups of four, x from e0 and z
// from e1.  Rotated lanes of the half layout hold partners, (x[i], z[i]); all
// other lanes hold eight neighbouring elements.
template <int D, bool kInter>
struct Lane {
  static constexpr int kLanes = D / 8;          // lanes of one head
  static constexpr int kHeads = 32 / kLanes;    // heads of one warp pass
  int e0, e1, sel, pair;   // pair: first rotated pair, or -1
  __device__ __forceinline__ Lane(int lane, int rot) {
    const int sub = lane % kLanes;
    sel = lane / kLanes;
    const bool in = sub * 8 < rot;
    e0 = sub * 8;
    e1 = e0 + 4;
    pair = in ? sub * 4 : -1;
    if (!kInter && in) {
      e0 = sub * 4;
      e1 = rot / 2 + sub * 4;
    }
  }
  // the pairs' cosines and sines as coefficients of two elements each:
  // half layout: of (x, z) elements 0, 1 and 2, 3; interleaved: cosine twice,
  // and (-sine, sine), for the two elements of each of four pairs
  __device__ __forceinline__ void coefficients(const float2* cs, uint64_t (&c)[4],
                                               uint64_t (&s)[4]) const {
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair >= 0 ? cs[pair + i] : make_float2(1.f, 0.f);
    if constexpr (kInter) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = pack2(v[i].x, v[i].x);
        s[i] = pack2(-v[i].y, v[i].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        c[i] = pack2(v[2 * i].x, v[2 * i + 1].x);
        s[i] = pack2(v[2 * i].y, v[2 * i + 1].y);
      }
    }
  }
};

}  // namespace

}  // namespace cpattn
