// rope.cuh -- rotary positions: the angle of a (position, pair) and the
// rotation of vectors of pairs, shared by the kernels that rotate.
//
// A pair (x1, x2) at position p with frequency f (radians a position) becomes
//   y1 = a (x1 cos(p f) - x2 sin(p f)),  y2 = a (x2 cos(p f) + x1 sin(p f)).
// The angle is formed in turns as a 64-bit binary fraction: with
// t = 2^64 frac(f / 2 pi) to a unit, the product p t, taken mod 2^64, is the angle's
// fraction of a turn to 2^-33 for any 32-bit p, whole turns dropping out by
// themselves; its upper 32 bits, cut off there, are used (2^-32 of a turn, 1.5e-9 radians). So far
// positions cost and lose nothing (an fp32 product p f is 0.06
// radians off at a million), no table is read, and the sine and cosine are taken
// of an eighth of a turn at most, where fp32 holds the angle to 5e-8.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/pa.h"

namespace pa {

// On an eighth of a turn, |x| <= pi / 4, the series of sine up to x^9 and of cosine up to x^8
// leave out less than 2e-9 and 3e-8, below fp32's half steps there.
__device__ __forceinline__ void rope_cos_sin(uint64_t turns, int32_t pos, float amplitude, float& c, float& s) {
  const uint32_t lo = (uint32_t)turns, hi = (uint32_t)(turns >> 32), p = (uint32_t)pos;
  const uint32_t part = __umulhi(lo, p) + hi * p - (pos < 0 ? lo : 0u);  // of a turn, in 2^-32
  const uint32_t quarter = (part + 0x20000000u) >> 30;                    // the nearest one, mod 4
  const float x = (float)(int32_t)(part - (quarter << 30)) * 1.462918079e-9f;  // 2 pi / 2^32
  const float x2 = x * x;
  float sn = fmaf(x2, 1.f / 362880, -1.f / 5040);
  sn = fmaf(x2, sn, 1.f / 120);
  sn = fmaf(x2, sn, -1.f / 6);
  sn = fmaf(x * x2, sn, x);
  float cs = fmaf(x2, 1.f / 40320, -1.f / 720);
  cs = fmaf(x2, cs, 1.f / 24);
  cs = fmaf(x2, cs, -0.5f);
  cs = fmaf(x2, cs, 1.f);
  // a quarter turn swaps the two; the sign of the cosine turns at 1/4 and 3/4, the sine's at 1/2
  const float u = (quarter & 1) ? sn : cs, v = (quarter & 1) ? cs : sn;
  c = __uint_as_float(__float_as_uint(amplitude * u) ^ (((quarter + 1) & 2) << 30));
  s = __uint_as_float(__float_as_uint(amplitude * v) ^ ((quarter & 2) << 30));
}

// The unit of a row that a thread holds: two vectors of VEC elements. Of the rotated part
// it is VEC pairs (half pairs: elements VEC u .. and rot / 2 + VEC u ..; interleaved ones: 2 VEC
// neighbours), of the rest 2 VEC neighbours, whose second half may lie past the row's end.
struct RopeUnits {
  int units, turning;  // per row, the `turning` ones first
};
inline RopeUnits rope_units(int D, int rot, int vec, bool rest) {
  const int turning = rot / (2 * vec);
  return {turning + (rest ? (D - rot + 2 * vec - 1) / (2 * vec) : 0), turning};
}

template <typename T, int VEC, bool INTER>
struct RopeUnit {
  static constexpr int BYTES = VEC * (int)sizeof(T), W = BYTES / 4;  // of a vector
  int a, b;   // where in a row the vectors lie
  bool turn;  // pairs to be rotated
  bool two;   // the second vector exists
  __device__ __forceinline__ RopeUnit(int D, int rot, int turning, int u) {
    turn = u < turning;
    a = turn ? (INTER ? 2 * u * VEC : u * VEC) : rot + 2 * VEC * (u - turning);
    b = turn && !INTER ? rot / 2 + u * VEC : a + VEC;
    two = b < D;
  }
  static __device__ __forceinline__ void get(uint32_t (&w)[2 * W], int at, const T* p) {
    if constexpr (BYTES == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[at] = v.x, w[at + 1] = v.y;
    } else if constexpr (BYTES == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[at] = v.x, w[at + 1] = v.y, w[at + 2] = v.z, w[at + 3] = v.w;
    } else {
      asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[at]), "=r"(w[at + 1]), "=r"(w[at + 2]), "=r"(w[at + 3]), "=r"(w[at + 4]), "=r"(w[at + 5]),
                     "=r"(w[at + 6]), "=r"(w[at + 7])
                   : "l"(p)
                   : "memory");
    }
  }
  static __device__ __forceinline__ void put(const uint32_t (&w)[2 * W], int at, T* p) {
    if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[at], w[at + 1]);
    } else if constexpr (BYTES == 16) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[at], w[at + 1], w[at + 2], w[at + 3]);
    } else {
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[at]), "r"(w[at + 1]), "r"(w[at + 2]),
                   "r"(w[at + 3]), "r"(w[at + 4]), "r"(w[at + 5]), "r"(w[at + 6]), "r"(w[at + 7])
                   : "memory");
    }
  }
  __device__ __forceinline__ void load(uint32_t (&w)[2 * W], const T* row) const {
    get(w, 0, row + a);
    if (two) get(w, W, row + b);
  }
  __device__ __forceinline__ void store(const uint32_t (&w)[2 * W], T* row) const {
    put(w, 0, row + a);
    if (two) put(w, W, row + b);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ void rotate(uint32_t (&w)[2 * W], const float (&c)[VEC], const float (&s)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if constexpr (sizeof(T) == 4) {
        uint32_t &wa = INTER ? w[2 * i] : w[i], &wb = INTER ? w[2 * i + 1] : w[W + i];
        const float x = __uint_as_float(wa), y = __uint_as_float(wb);
        wa = __float_as_uint(x * c[i] - y * s[i]);
        wb = __float_as_uint(y * c[i] + x * s[i]);
      } else if constexpr (INTER) {
        const float x = __uint_as_float(w[i] << 16), y = __uint_as_float(w[i] & 0xFFFF0000u);
        w[i] = pack(x * c[i] - y * s[i], y * c[i] + x * s[i]);
      } else if (i % 2 == 0) {
        uint32_t &wa = w[i / 2], &wb = w[W + i / 2];
        const float x0 = __uint_as_float(wa << 16), x1 = __uint_as_float(wa & 0xFFFF0000u);
        const float y0 = __uint_as_float(wb << 16), y1 = __uint_as_float(wb & 0xFFFF0000u);
        wa = pack(x0 * c[i] - y0 * s[i], x1 * c[i + 1] - y1 * s[i + 1]);
        wb = pack(y0 * c[i] + x0 * s[i], y1 * c[i + 1] + x1 * s[i + 1]);
      }
    }
  }
  // n heads of one row, xs and ys elements apart, several loads in flight
  __device__ __forceinline__ void move(const T* x, int64_t xs, T* y, int64_t ys, int n, bool rotating, const float (&c)[VEC],
                                       const float (&s)[VEC]) const {
    constexpr int U = BYTES == 32 ? 2 : 4;
#pragma unroll 1
    for (int h = 0; h < n; h += U, x += U * xs, y += U * ys) {
      uint32_t w[U][2 * W];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < n) load(w[i], x + i * xs);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < n) {
          if (rotating) rotate(w[i], c, s);
          store(w[i], y + i * ys);
        }
    }
  }
};

}  // namespace pa
