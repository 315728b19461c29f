// rope.cuh -- rotary positions: the angle of a (position, pair) and the
// rotation of vectors of pairs, shared by the kernels that rotate.
//
// A pair (x1, x2) at position p with frequency f (radians a position) becomes
//   y1 = a (x1 cos(p f) - x2 sin(p f)),  y2 = a (x2 cos(p f) + x1 sin(p f)).
// The angle is formed in turns as a 64-bit binary fraction: with
// t = round(2^64 frac(f / 2 pi)) the product p t, taken mod 2^64, is the angle's
// fraction of a turn to 2^-33 for any 32-bit p, whole turns dropping out by
// themselves. So far positions cost and lose nothing (an fp32 product p f is 0.06
// radians off at a million), no table is read, and the sine and cosine are taken
// of an eighth of a turn at most, where fp32 holds the angle to 5e-8.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/pa.h"

namespace pa {

__device__ __forceinline__ void rope_cos_sin(uint64_t turns, int32_t pos, float amplitude, float& c, float& s) {
  const uint32_t part = (uint32_t)((turns * (uint64_t)(int64_t)pos) >> 32);  // of a turn, in 2^-32
  const uint32_t quarter = (part + 0x20000000u) >> 30;                      // nearest, mod 4
  const int32_t rest = (int32_t)(part - (quarter << 30));                   // -1/8 .. 1/8 of a turn
  float sn, cs;
  sincospif((float)rest * 0x1p-31f, &sn, &cs);
  const float u = (quarter & 1) ? sn : cs, v = (quarter & 1) ? cs : sn;
  c = (quarter == 1 || quarter == 2) ? -amplitude * u : amplitude * u;
  s = (quarter & 2) ? -amplitude * v : amplitude * v;
}

// A unit of VEC pairs of one row: pairs VEC u .. VEC u + VEC - 1 of rot / 2.
// Interleaved pairs are neighbours (2 VEC elements in one run); half pairs lie
// rot / 2 apart (two runs of VEC elements).
template <typename T, int VEC, bool INTER>
struct RopeUnit {
  static constexpr int W = VEC * 2 * (int)sizeof(T) / 4;  // 32-bit words
  uint32_t w[W];

  template <int N>
  static __device__ __forceinline__ void get(uint32_t* to, const T* p) {
    if constexpr (N == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      to[0] = v.x, to[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        to[i] = v.x, to[i + 1] = v.y, to[i + 2] = v.z, to[i + 3] = v.w;
      }
    }
  }
  template <int N>
  static __device__ __forceinline__ void put(T* p, const uint32_t* v) {
    if constexpr (N == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  }
  __device__ __forceinline__ void load(const T* row, int u, int half) {
    if constexpr (INTER) {
      get<W>(w, row + u * (2 * VEC));
    } else {
      get<W / 2>(w, row + u * VEC);
      get<W / 2>(w + W / 2, row + half + u * VEC);
    }
  }
  __device__ __forceinline__ void store(T* row, int u, int half) const {
    if constexpr (INTER) {
      put<W>(row + u * (2 * VEC), w);
    } else {
      put<W / 2>(row + u * VEC, w);
      put<W / 2>(row + half + u * VEC, w + W / 2);
    }
  }
  __device__ __forceinline__ void rotate(const float (&c)[VEC], const float (&s)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if constexpr (sizeof(T) == 4) {
        uint32_t &wa = INTER ? w[2 * i] : w[i], &wb = INTER ? w[2 * i + 1] : w[W / 2 + i];
        const float a = __uint_as_float(wa), b = __uint_as_float(wb);
        wa = __float_as_uint(a * c[i] - b * s[i]);
        wb = __float_as_uint(b * c[i] + a * s[i]);
      } else if constexpr (INTER) {
        const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
        w[i] = pack(a * c[i] - b * s[i], b * c[i] + a * s[i]);
      } else if (i % 2 == 0) {
        uint32_t &wa = w[i / 2], &wb = w[W / 2 + i / 2];
        const float a0 = __uint_as_float(wa << 16), a1 = __uint_as_float(wa & 0xFFFF0000u);
        const float b0 = __uint_as_float(wb << 16), b1 = __uint_as_float(wb & 0xFFFF0000u);
        wa = pack(a0 * c[i] - b0 * s[i], a1 * c[i + 1] - b1 * s[i + 1]);
        wb = pack(b0 * c[i] + a0 * s[i], b1 * c[i + 1] + a1 * s[i + 1]);
      }
    }
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// Eight elements that are not rotated.
template <typename T>
struct PlainUnit {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
};

}  // namespace pa
