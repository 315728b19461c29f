// ckpt.cu -- activations kept in 8 bits between the forward and the backward:
// save, load, and the step that starts the attention backward from them.
//
// A row of C elements is cut into blocks of G (the last may be short). Per block
//   s    = max |x| / top                 top = 127 (int8) or 448 (e4m3), fp32
//   code = x / s rounded once, to nearest even (int8 in -127..127, or e4m3)
//   y    = code * s                      (fp32, then rounded to the tensor's type)
// A block of zeros has s = 0; one that holds an infinity or a NaN has s = NaN
// and codes 0, so that all of it comes back as NaN instead of hiding the fault.
//
// All of it is bound by memory: 3 bytes an element in bf16 either way, 1/G of
// a float for the scale. A thread takes vectors of 16 elements (a 32-byte load
// of bf16, a 16-byte store of codes) where every row is a whole number of
// blocks without gaps and the tensor starts on 32 bytes, else of 8, with
// several loads in flight, and a block's lanes share its maximum by shuffles.
// What a block needs once (its scale, the reciprocal) is computed by every lane
// that holds a part of it, so longer vectors also mean fewer instructions: saving
// 8192 x 4096 bf16 as int8 took 25.6 us with vectors of 8 and 18.4 us with vectors
// of 16 (5.6 TB/s), loading it 19.5 and 13.3 us.
//
// The rounding is exact without a division per element: q = x * (1 / s) is
// within 2^-23 of x / s relatively, so only a quotient that lies that close
// to the border t between two codes is undecided, and there the sign of
// fma(-t, s, x), which rounds once, says on which side of it x / s is.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "sm103.cuh"

namespace pa {
namespace {

constexpr int kCkptThreads = 256;
// Vectors in flight per thread, in a save and in a load.
template <int VEC>
constexpr int kUnroll = VEC == 16 ? 2 : 4;
constexpr int kLoadUnroll = 4;

// n / d for n < 2^31 as a product (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994): q = (mulhi(m, n) + n) >> s.
struct FastDiv {
  uint32_t d, m, s;
};
FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{d, (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1), s};
}
__device__ __forceinline__ uint32_t quot(uint32_t n, const FastDiv& f) { return (__umulhi(f.m, n) + n) >> f.s; }

struct Tensor {
  const void* x;  // save: source; load: destination
  void* codes;
  float* scales;
  uint32_t blocks0;     // thread blocks of the tensors before this one
  uint32_t vecs;        // vectors in all (save: short blocks filled up to G elements)
  int C;                // elements per row
  int nb;               // blocks of G per row
  FastDiv row_vecs, N, H;
  int64_t sb, sh, sn;   // element strides; contiguous rows: sn = C, and N, H unused
  int contiguous;
};
struct Tensors {
  Tensor t[PA_CKPT_MAX_TENSORS];
  int count;
};

__device__ __forceinline__ size_t row_offset(const Tensor& t, uint32_t row) {
  if (t.contiguous) return (size_t)row * t.C;
  const uint32_t bh = quot(row, t.N), n = row - bh * t.N.d, b = quot(bh, t.H), h = bh - b * t.H.d;
  return (size_t)b * t.sb + (size_t)h * t.sh + (size_t)n * t.sn;
}

// Where vector i of a tensor lies: its elements, its codes and its block's
// scale (2^shift vectors a block). FLAT: rows without gaps or short blocks, so
// that vector i is simply the elements from VEC i on.
struct Place {
  size_t x, code, scale;
  bool on;
};
template <int VEC, bool FLAT, bool SAVE>
__device__ __forceinline__ Place place_of(const Tensor& t, uint32_t i, int shift) {
  Place p;
  if (FLAT) {
    p.on = i < t.vecs;
    p.x = p.code = (size_t)i * VEC;
    p.scale = i >> shift;
  } else {
    const uint32_t row = quot(i, t.row_vecs), at = i - row * t.row_vecs.d;
    p.on = i < t.vecs && (!SAVE || (int)at * VEC < t.C);  // a save counts short blocks as whole
    p.x = row_offset(t, row) + at * VEC;
    p.code = (size_t)row * t.C + at * VEC;
    p.scale = (size_t)row * t.nb + (at >> shift);
  }
  return p;
}

// 32 bytes of one lane in one access (aligned to them).
__device__ __forceinline__ void ld_32(const void* p, uint32_t* w) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void st_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// VEC elements as they lie in memory (WIDE: taken 32 bytes at a time, which they
// are then aligned to), their largest magnitude as the bits of an
// fp32 value (NaN and infinity order above every number), and as fp32.
template <typename T, int VEC, bool WIDE = VEC == 16>
struct Vec {
  static constexpr int W = VEC * sizeof(T) / 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const void* base, size_t e) {
    const T* p = static_cast<const T*>(base) + e;
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < W; i += 8) ld_32(reinterpret_cast<const uint32_t*>(p) + i, w + i);
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void store(void* base, size_t e) const {
    T* p = static_cast<T*>(base) + e;
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < W; i += 8) st_32(reinterpret_cast<uint32_t*>(p) + i, w + i);
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < W; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      return max(m << 16, m & 0xFFFF0000u);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    return m;
  }
  // elements 8 part .. 8 part + 7
  __device__ __forceinline__ void floats(int part, float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (sizeof(T) == 2) {
        const uint32_t x = w[4 * part + i / 2];
        f[i] = __uint_as_float(i & 1 ? x & 0xFFFF0000u : x << 16);
      } else {
        f[i] = __uint_as_float(w[(8 * part + i) % W]);
      }
    }
  }
  __device__ __forceinline__ void set(int part, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (sizeof(T) == 2) {
        if (i & 1) w[4 * part + i / 2] = pack_bf16x2(f[i - 1], f[i]);
      } else {
        w[(8 * part + i) % W] = __float_as_uint(f[i]);
      }
    }
  }
};

// ------------------------------------------------------------------- formats
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3_values(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

template <int FMT>
struct Format;

template <>
struct Format<PA_CKPT_INT8> {
  static constexpr float kTop = 127.f;
  // Codes of x[0..7], with r = 1 / s rounded: x r is within 2^-24 of x / s,
  // relatively, and at most 127 (1 + 2^-23).
  static __device__ __forceinline__ uint2 encode(const float (&x)[8], float s, float r) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a sum's low bits are the nearest integer
    const uint64_t r2 = f2(r, r), magic2 = f2(kMagic, kMagic), minus1 = f2(-1.f, -1.f);
    uint32_t u[8];
    float far = 0.f;  // the largest distance of an x r from its code
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t x2 = f2(x[i], x[i + 1]), y = fma2(x2, r2, magic2);
      const float2 d = f2_split(fma2(x2, r2, fma2(y, minus1, magic2))), yy = f2_split(y);
      u[i] = __float_as_uint(yy.x);
      u[i + 1] = __float_as_uint(yy.y);
      far = fmax3(far, fabsf(d.x), fabsf(d.y));
    }
    if (far > 0.4999f) {  // x r is off by 127 * 2^-24 at most, and the distance by a rounding
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float k = fmaf(x[i], r, kMagic) - kMagic, d = fmaf(x[i], r, -k);
        if (fabsf(d) > 0.4999f) {
          const float up = d > 0.f ? 1.f : -1.f, side = up * fmaf(-(k + 0.5f * up), s, x[i]);
          const bool odd = __float_as_uint(k + kMagic) & 1u;
          u[i] = __float_as_uint((side > 0.f || (side == 0.f && odd) ? k + up : k) + kMagic);
        }
      }
    }
    return make_uint2(__byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410));
  }
  static __device__ __forceinline__ void decode(uint2 c, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the byte with its sign bit flipped, under 2^23's exponent: 2^23 + 128 + code
      const uint32_t w = (i < 4 ? c.x : c.y) ^ 0x80808080u;
      f[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 | (i & 3))) - 8388736.f;
    }
  }
};

template <>
struct Format<PA_CKPT_E4M3> {
  static constexpr float kTop = 448.f;
  static __device__ __forceinline__ uint2 encode(const float (&x)[8], float s, float r) {
    uint32_t c[4], near = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // the quotient a little too small and a little too large: where the
      // codes agree, so does that of the exact quotient between them
      const float a = x[2 * i] * r, b = x[2 * i + 1] * r;
      c[i] = e4m3_pair(fmaf(a, -0x1p-21f, a), fmaf(b, -0x1p-21f, b));
      near |= c[i] ^ e4m3_pair(fmaf(a, 0x1p-21f, a), fmaf(b, 0x1p-21f, b));
    }
    if (near) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = fabsf(x[i] * r);
        const uint32_t two = e4m3_pair(fmaf(q, -0x1p-21f, q), fmaf(q, 0x1p-21f, q));
        uint32_t lo = two & 0xFFu;
        const uint32_t hi = two >> 8;
        if (lo != hi) {
          const float2 v = e4m3_values(two);
          const float side = fmaf(-0.5f * (v.x + v.y), s, fabsf(x[i]));  // v.x + v.y is exact
          if (side > 0.f || (side == 0.f && (lo & 1u))) lo = hi;
        }
        lo |= __float_as_uint(x[i]) >> 31 << 7;
        const int at = 8 * (i & 1);
        c[i >> 1] = (c[i >> 1] & ~(0xFFu << at)) | lo << at;
      }
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
  static __device__ __forceinline__ void decode(uint2 c, float (&f)[8]) {
    const float2 a = e4m3_values(c.x & 0xFFFFu), b = e4m3_values(c.x >> 16);
    const float2 d = e4m3_values(c.y & 0xFFFFu), e = e4m3_values(c.y >> 16);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = d.x, f[5] = d.y, f[6] = e.x, f[7] = e.y;
  }
};

__device__ __forceinline__ const Tensor& tensor_of(const Tensors& a, uint32_t block, uint32_t per_block, uint32_t* first) {
  int i = 0;
  while (i + 1 < a.count && block >= a.t[i + 1].blocks0) ++i;
  *first = (block - a.t[i].blocks0) * per_block;
  return a.t[i];
}

// max / top, rounded correctly: a first quotient from the rounded reciprocal of
// top, its remainder exactly, and one correction (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000", 1990). Below 2^-100 the
// remainder could be lost, and the division is left to the compiler.
template <int FMT>
__device__ __forceinline__ float scale_of(float m) {
  constexpr float kTop = Format<FMT>::kTop, kInv = 1.f / kTop;
  if (m < 0x1p-100f) return __fdiv_rn(m, kTop);
  const float q = m * kInv;
  return fmaf(fmaf(-q, kTop, m), kInv, q);
}

// LG lanes hold one block of LG * VEC elements.
template <typename T, int FMT, int VEC, int LG, bool WIDE>
__global__ void __launch_bounds__(kCkptThreads) ckpt_save_kernel(const __grid_constant__ Tensors a) {
  using F = Format<FMT>;
  constexpr int U = kUnroll<VEC>, kShift = LG == 2 ? 1 : LG == 4 ? 2 : LG == 8 ? 3 : 4;
  uint32_t first;
  const Tensor& t = tensor_of(a, blockIdx.x, kCkptThreads * U, &first);
  Vec<T, VEC, WIDE> v[U];
  Place at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at[u] = place_of<VEC, VEC == 16, true>(t, first + u * kCkptThreads + threadIdx.x, kShift);
    if (at[u].on)
      v[u].load(t.x, at[u].x);
    else
      v[u].zero();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t m = v[u].top();
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
    if (!at[u].on) continue;
    const bool finite = m < 0x7F800000u;
    float s = finite ? scale_of<FMT>(__uint_as_float(m)) : __uint_as_float(0x7FC00000u);
    if (threadIdx.x % LG == 0) t.scales[at[u].scale] = s;
    uint2 c[VEC / 8];
    const bool small = s < 0x1p-100f;
    if (small) s *= 0x1p100f;  // 1 / s could overflow: both by 2^100, which changes no bits of either
    const float r = __frcp_rn(s);
#pragma unroll
    for (int h = 0; h < VEC / 8; ++h) {
      float f[8];
      v[u].floats(h, f);
      if (small) {
        // a scale below the normal range has been rounded to few bits: quotients
        // past the largest code are cut there
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i] * 0x1p100f, -F::kTop * s), F::kTop * s);
      }
      c[h] = finite && s > 0.f ? F::encode(f, s, r) : make_uint2(0u, 0u);
    }
    uint8_t* out = static_cast<uint8_t*>(t.codes) + at[u].code;
    if (VEC == 16)
      *reinterpret_cast<uint4*>(out) = make_uint4(c[0].x, c[0].y, c[VEC / 8 - 1].x, c[VEC / 8 - 1].y);
    else
      *reinterpret_cast<uint2*>(out) = c[0];
  }
}

// Vectors first .. of one tensor: codes and scales to T. shift = log2 of the
// vectors in a block.
template <typename T, int FMT, int VEC, bool WIDE>
__device__ __forceinline__ void load_vectors(const Tensor& t, uint32_t first, int shift) {
  using F = Format<FMT>;
  constexpr int U = kLoadUnroll;
  uint2 c[U][VEC / 8];
  float s[U];
  Place at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at[u] = place_of<VEC, VEC == 16, false>(t, first + u * kCkptThreads + threadIdx.x, shift);
    s[u] = 0.f;
#pragma unroll
    for (int h = 0; h < VEC / 8; ++h) c[u][h] = make_uint2(0u, 0u);
    if (!at[u].on) continue;
    const uint8_t* from = static_cast<const uint8_t*>(t.codes) + at[u].code;
    if (VEC == 16) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(from));
      c[u][0] = make_uint2(w.x, w.y);
      c[u][VEC / 8 - 1] = make_uint2(w.z, w.w);
    } else {
      c[u][0] = __ldg(reinterpret_cast<const uint2*>(from));
    }
    s[u] = __ldg(t.scales + at[u].scale);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!at[u].on) continue;
    Vec<T, VEC, WIDE> v;
#pragma unroll
    for (int h = 0; h < VEC / 8; ++h) {
      float f[8];
      F::decode(c[u][h], f);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 y = f2_split(mul2(f2(f[i], f[i + 1]), f2(s[u], s[u])));
        f[i] = y.x;
        f[i + 1] = y.y;
      }
      v.set(h, f);
    }
    v.store(const_cast<void*>(t.x), at[u].x);
  }
}
template <typename T, int FMT, int VEC, bool WIDE>
__global__ void __launch_bounds__(kCkptThreads) ckpt_load_kernel(const __grid_constant__ Tensors a, int shift) {
  uint32_t first;
  const Tensor& t = tensor_of(a, blockIdx.x, kCkptThreads * kLoadUnroll, &first);
  load_vectors<T, FMT, VEC, WIDE>(t, first, shift);
}

// Start of the attention backward from 8-bit tensors, in one launch: the
// first thread blocks bring q, k and v back as bf16 (the operand type of the
// products), the rest form delta = rowsum(dO * O) with O straight from its
// codes, O itself never being stored, and lse * log2(e). Bound by memory; the
// packed 8k row (Hq 32, Hkv 8, D 128; 251 MB) takes 43.5 us, 5.8 TB/s: five blocks
// an SM and two rows a thread in flight; with four rows a thread and three
// blocks it took 53.5 us.
struct DeltaArgs {
  const uint8_t* codes;  // (B, H, Nr, D)
  const float* scales;
  const __nv_bfloat16* dout;
  const float* lse;
  float* delta;
  float* lse2;
  uint32_t rows;  // B * H * N, N padded to whole tiles
  FastDiv N, H;
  int Nr, nb, shift;   // shift: log2 of a block's groups of 16
  int64_t sb, sh, sn;  // of dout
};
// A row's groups of 16 elements on a power of two of lanes, and rows in flight
// per thread.
constexpr int row_lanes(int D) { return D == 128 ? 8 : D == 64 ? 4 : 2; }
constexpr int row_unroll(int D) { return D == 96 ? 1 : 2; }
constexpr int block_rows(int D) { return kCkptThreads / row_lanes(D) * row_unroll(D); }

// VEC: of the load. WIDE: dout's rows start on 32 bytes.
template <int D, int FMT, int VEC, bool WIDE>
__global__ void __launch_bounds__(kCkptThreads, VEC == 16 ? 5 : 4)
    bwd_ckpt_prologue_kernel(const __grid_constant__ Tensors a, uint32_t load_blocks, const DeltaArgs p, int shift) {
  if (blockIdx.x < load_blocks) {
    uint32_t first;
    const Tensor& t = tensor_of(a, blockIdx.x, kCkptThreads * kLoadUnroll, &first);
    load_vectors<__nv_bfloat16, FMT, VEC, VEC == 16>(t, first, shift);
    return;
  }
  using F = Format<FMT>;
  constexpr int LPR = row_lanes(D), NL = D / 16 / LPR, R = row_unroll(D);
  const uint32_t row0 = (blockIdx.x - load_blocks) * block_rows(D) + threadIdx.x / LPR;
  const int sub = threadIdx.x % LPR;
  uint4 c[R][NL];
  float s[R][NL];
  Vec<__nv_bfloat16, 16> g[R][NL];
  bool live[R];
#pragma unroll
  for (int u = 0; u < R; ++u) {
    const uint32_t row = row0 + u * (kCkptThreads / LPR);
    const uint32_t bh = quot(row, p.N), n = row - bh * p.N.d, b = quot(bh, p.H), h = bh - b * p.H.d;
    // rows past the caller's N get P = 0 (lse = +inf) and delta = 0, so they add nothing
    live[u] = row < p.rows && n < (uint32_t)p.Nr;
    const size_t r = (size_t)bh * p.Nr + n;
    const __nv_bfloat16* dout = p.dout + (size_t)b * p.sb + (size_t)h * p.sh + (size_t)n * p.sn;
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const int v = sub + k * LPR;
      if (live[u]) {
        c[u][k] = __ldg(reinterpret_cast<const uint4*>(p.codes + r * D) + v);
        s[u][k] = __ldg(p.scales + r * p.nb + (v >> p.shift));
        if (WIDE) {
          ld_32(dout + v * 16, g[u][k].w);
        } else {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(dout + v * 16)), y = __ldg(reinterpret_cast<const uint4*>(dout + v * 16) + 1);
          g[u][k].w[0] = x.x, g[u][k].w[1] = x.y, g[u][k].w[2] = x.z, g[u][k].w[3] = x.w;
          g[u][k].w[4] = y.x, g[u][k].w[5] = y.y, g[u][k].w[6] = y.z, g[u][k].w[7] = y.w;
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < R; ++u) {
    float acc = 0.f;
    if (live[u]) {
#pragma unroll
      for (int k = 0; k < NL; ++k) {
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float o[8], d[8];
          F::decode(h ? make_uint2(c[u][k].z, c[u][k].w) : make_uint2(c[u][k].x, c[u][k].y), o);
          g[u][k].floats(h, d);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(o[i], d[i], sum);
        }
        acc = fmaf(s[u][k], sum, acc);
      }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(~0u, acc, o);
    const uint32_t row = row0 + u * (kCkptThreads / LPR);
    if (sub == 0 && row < p.rows) {
      const uint32_t bh = quot(row, p.N), n = row - bh * p.N.d;
      p.delta[row] = acc;
      p.lse2[row] = live[u] ? p.lse[(size_t)bh * p.Nr + n] * 1.4426950408889634f : INFINITY;
    }
  }
  // This kernel runs beside the tile table's, on which nothing here depends;
  // the one after it needs both, so the last block waits for the other's end.
  if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Whether all the tensors can be taken in vectors of 16 without looking at rows.
bool all_flat(const CkptTensor* x, int count, int G) {
  for (int i = 0; i < count; ++i) {
    const bool contiguous = (x[i].N == 1 || x[i].s_n == x[i].C) && (x[i].H == 1 || x[i].s_h == (int64_t)x[i].N * x[i].C) &&
                            (x[i].B == 1 || x[i].s_b == (int64_t)x[i].H * x[i].N * x[i].C);
    if (!contiguous || x[i].C % G != 0 || !aligned32(x[i].x)) return false;
  }
  return true;
}

// The tensors' descriptions in vectors of VEC elements and thread blocks of
// `per_block` vectors; a save counts short blocks as whole.
uint32_t describe(const CkptTensor* x, int count, int G, int VEC, uint32_t per_block, bool save, Tensors* a) {
  uint32_t blocks = 0;
  a->count = count;
  for (int i = 0; i < count; ++i) {
    Tensor& t = a->t[i];
    t.x = x[i].x;
    t.codes = x[i].codes;
    t.scales = x[i].scales;
    t.blocks0 = blocks;
    t.C = x[i].C;
    t.nb = (x[i].C + G - 1) / G;
    const uint32_t rv = save ? (uint32_t)t.nb * (G / VEC) : (uint32_t)x[i].C / VEC;
    t.vecs = (uint32_t)((int64_t)x[i].B * x[i].H * x[i].N) * rv;
    t.row_vecs = fast_div(rv);
    t.N = fast_div(x[i].N);
    t.H = fast_div(x[i].H);
    t.sb = x[i].s_b;
    t.sh = x[i].s_h;
    t.sn = x[i].s_n;
    t.contiguous = (x[i].N == 1 || t.sn == t.C) && (x[i].H == 1 || t.sh == (int64_t)x[i].N * t.C) &&
                   (x[i].B == 1 || t.sb == (int64_t)x[i].H * x[i].N * t.C);
    blocks += (uint32_t)(((uint64_t)t.vecs + per_block - 1) / per_block);
  }
  return blocks;
}
int log2_of(int n) { return n == 2 ? 1 : n == 4 ? 2 : n == 8 ? 3 : 4; }

// Whether vectors of eight fp32 elements start on 32 bytes.
bool all_wide(const CkptTensor* x, int count) {
  for (int i = 0; i < count; ++i)
    if (!aligned32(x[i].x) || (x[i].N > 1 && x[i].s_n % 8) || (x[i].H > 1 && x[i].s_h % 8) || (x[i].B > 1 && x[i].s_b % 8))
      return false;
  return true;
}

template <typename T, int FMT, int VEC, bool WIDE>
void save_launch(const CkptTensor* x, int count, int G, cudaStream_t st) {
  Tensors a{};
  const uint32_t blocks = describe(x, count, G, VEC, kCkptThreads * kUnroll<VEC>, true, &a);
  if (G == 32)
    ckpt_save_kernel<T, FMT, VEC, 32 / VEC, WIDE><<<blocks, kCkptThreads, 0, st>>>(a);
  else if (G == 64)
    ckpt_save_kernel<T, FMT, VEC, 64 / VEC, WIDE><<<blocks, kCkptThreads, 0, st>>>(a);
  else
    ckpt_save_kernel<T, FMT, VEC, 128 / VEC, WIDE><<<blocks, kCkptThreads, 0, st>>>(a);
}
template <typename T, int FMT>
void save_any(const CkptTensor* x, int count, int G, cudaStream_t st) {
  if (all_flat(x, count, G))
    save_launch<T, FMT, 16, true>(x, count, G, st);
  else if (sizeof(T) == 4 && all_wide(x, count))
    save_launch<T, FMT, 8, sizeof(T) == 4>(x, count, G, st);
  else
    save_launch<T, FMT, 8, false>(x, count, G, st);
}

template <typename T, int FMT, int VEC, bool WIDE>
void load_launch(const CkptTensor* x, int count, int G, cudaStream_t st) {
  Tensors a{};
  const uint32_t blocks = describe(x, count, G, VEC, kCkptThreads * kLoadUnroll, false, &a);
  ckpt_load_kernel<T, FMT, VEC, WIDE><<<blocks, kCkptThreads, 0, st>>>(a, log2_of(G / VEC));
}
template <typename T, int FMT>
void load_any(const CkptTensor* x, int count, int G, cudaStream_t st) {
  if (all_flat(x, count, G))
    load_launch<T, FMT, 16, true>(x, count, G, st);
  else if (sizeof(T) == 4 && all_wide(x, count))
    load_launch<T, FMT, 8, sizeof(T) == 4>(x, count, G, st);
  else
    load_launch<T, FMT, 8, false>(x, count, G, st);
}

template <int D, int VEC>
cudaError_t prologue_launch(const CkptTensor* qkv, int format, int G, const DeltaArgs& d, cudaStream_t st) {
  Tensors a{};
  const uint32_t load_blocks = describe(qkv, 3, G, VEC, kCkptThreads * kLoadUnroll, false, &a);
  const bool wide = aligned32(d.dout) && d.sb % 16 == 0 && d.sh % 16 == 0 && d.sn % 16 == 0;
  const bool i8 = format == PA_CKPT_INT8;
  const auto kfn = wide ? (i8 ? bwd_ckpt_prologue_kernel<D, PA_CKPT_INT8, VEC, true> : bwd_ckpt_prologue_kernel<D, PA_CKPT_E4M3, VEC, true>)
                        : (i8 ? bwd_ckpt_prologue_kernel<D, PA_CKPT_INT8, VEC, false> : bwd_ckpt_prologue_kernel<D, PA_CKPT_E4M3, VEC, false>);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(load_blocks + (d.rows + block_rows(D) - 1) / block_rows(D));
  cfg.blockDim = dim3(kCkptThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr = programmatic_launch();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, a, load_blocks, d, log2_of(G / VEC));
}

}  // namespace

cudaError_t launch_ckpt_save(const CkptTensor* x, int count, bool f32, int format, int block, cudaStream_t st) {
  if (format == PA_CKPT_INT8)
    f32 ? save_any<float, PA_CKPT_INT8>(x, count, block, st) : save_any<__nv_bfloat16, PA_CKPT_INT8>(x, count, block, st);
  else
    f32 ? save_any<float, PA_CKPT_E4M3>(x, count, block, st) : save_any<__nv_bfloat16, PA_CKPT_E4M3>(x, count, block, st);
  return cudaGetLastError();
}

cudaError_t launch_ckpt_load(const CkptTensor* x, int count, bool f32, int format, int block, cudaStream_t st) {
  if (format == PA_CKPT_INT8)
    f32 ? load_any<float, PA_CKPT_INT8>(x, count, block, st) : load_any<__nv_bfloat16, PA_CKPT_INT8>(x, count, block, st);
  else
    f32 ? load_any<float, PA_CKPT_E4M3>(x, count, block, st) : load_any<__nv_bfloat16, PA_CKPT_E4M3>(x, count, block, st);
  return cudaGetLastError();
}

cudaError_t launch_bwd_ckpt_prologue(const AttnParams& p, int D, const RowStrides& rs, const CkptTensor (&qkv)[3],
                                     const void* out_codes, const float* out_scales, int format, int block,
                                     cudaStream_t st) {
  DeltaArgs d{};
  d.codes = static_cast<const uint8_t*>(out_codes);
  d.scales = out_scales;
  d.dout = p.dout;
  d.lse = p.lse_in;
  d.delta = p.delta;
  d.lse2 = p.lse2;
  d.rows = (uint32_t)((int64_t)p.B * p.Hq * p.N);
  d.N = fast_div(p.N);
  d.H = fast_div(p.Hq);
  d.Nr = p.Nr;
  d.nb = (D + block - 1) / block;
  d.shift = log2_of(block / 16);
  d.sb = rs.q_b;
  d.sh = rs.q_h;
  d.sn = rs.q_n;
  const bool flat = all_flat(qkv, 3, block);
  if (D == 64) return flat ? prologue_launch<64, 16>(qkv, format, block, d, st) : prologue_launch<64, 8>(qkv, format, block, d, st);
  if (D == 96) return flat ? prologue_launch<96, 16>(qkv, format, block, d, st) : prologue_launch<96, 8>(qkv, format, block, d, st);
  return flat ? prologue_launch<128, 16>(qkv, format, block, d, st) : prologue_launch<128, 8>(qkv, format, block, d, st);
}

}  // namespace pa
