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
// a float for the scale. A thread takes vectors of 8 elements (16-byte loads
// of bf16, 8-byte stores of codes), four of them at a time so that enough
// loads are in flight, and a block's G / 8 lanes share its maximum by shuffles.
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

namespace pa {
namespace {

constexpr int kCkptThreads = 256, kCkptUnroll = 4;

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
  uint32_t vecs;        // vectors in all (save: short blocks filled up to G / 8 vectors)
  uint32_t rows;
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

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight elements as they lie in memory, their largest magnitude as the bits
// of an fp32 value (NaN and infinity order above every number), and as fp32.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* p, size_t e) {
    w = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + e));
  }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t top() const {
    constexpr uint32_t k = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    f[0] = bf_lo(w.x), f[1] = bf_hi(w.x), f[2] = bf_lo(w.y), f[3] = bf_hi(w.y);
    f[4] = bf_lo(w.z), f[5] = bf_hi(w.z), f[6] = bf_lo(w.w), f[7] = bf_hi(w.w);
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, size_t e) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
    a = __ldg(s);
    b = __ldg(s + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ uint32_t top() const {
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, size_t e, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p + e) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, size_t e, const float (&f)[8]) {
  float4* d = reinterpret_cast<float4*>(p + e);
  d[0] = make_float4(f[0], f[1], f[2], f[3]);
  d[1] = make_float4(f[4], f[5], f[6], f[7]);
}

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
  // Codes of x[0..7], with r within 2^-23 of 1 / s and |x| r <= 127.5 or so.
  static __device__ __forceinline__ uint2 encode(const float (&x)[8], float s, float r) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the nearest integer
    uint32_t u[8];
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = fminf(fmaxf(x[i] * r, -127.f), 127.f), y = q + kMagic;
      u[i] = __float_as_uint(y);
      near |= fabsf(q - (y - kMagic)) > 0.4999f;  // q is off by 1.6e-5 at most
    }
    if (near) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = fminf(fmaxf(x[i] * r, -127.f), 127.f), k = (q + kMagic) - kMagic, d = q - k;
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

__device__ __forceinline__ const Tensor& tensor_of(const Tensors& a, uint32_t block, uint32_t* first) {
  int i = 0;
  while (i + 1 < a.count && block >= a.t[i + 1].blocks0) ++i;
  *first = (block - a.t[i].blocks0) * (kCkptThreads * kCkptUnroll);
  return a.t[i];
}

// LG = G / 8 lanes hold one block.
template <typename T, int FMT, int LG>
__global__ void __launch_bounds__(kCkptThreads) ckpt_save_kernel(const __grid_constant__ Tensors a) {
  using F = Format<FMT>;
  uint32_t first;
  const Tensor& t = tensor_of(a, blockIdx.x, &first);
  Vec8<T> v[kCkptUnroll];
  uint32_t row[kCkptUnroll], at[kCkptUnroll];
  bool on[kCkptUnroll];
#pragma unroll
  for (int u = 0; u < kCkptUnroll; ++u) {
    const uint32_t i = first + u * kCkptThreads + threadIdx.x;
    row[u] = quot(i, t.row_vecs);
    at[u] = i - row[u] * t.row_vecs.d;  // vector within the row, short blocks filled up
    on[u] = i < t.vecs && (int)at[u] * 8 < t.C;
    if (on[u])
      v[u].load(t.x, row_offset(t, row[u]) + at[u] * 8);
    else
      v[u].zero();
  }
#pragma unroll
  for (int u = 0; u < kCkptUnroll; ++u) {
    uint32_t m = v[u].top();
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
    if (!on[u]) continue;
    const bool finite = m < 0x7F800000u;
    float s = finite ? __fdiv_rn(__uint_as_float(m), F::kTop) : __uint_as_float(0x7FC00000u);
    if (threadIdx.x % LG == 0) t.scales[(size_t)row[u] * t.nb + at[u] / LG] = s;
    uint2 c = make_uint2(0u, 0u);
    if (finite && s > 0.f) {
      float f[8];
      v[u].floats(f);
      if (s < 0x1p-100f) {  // 1 / s could overflow: both by 2^100, which changes no bits of either
        s *= 0x1p100f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= 0x1p100f;
      }
      c = F::encode(f, s, __frcp_rn(s));
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.codes) + (size_t)row[u] * t.C + at[u] * 8) = c;
  }
}

// Vectors first .. of one tensor: codes and scales to T. shift = log2(G / 8).
template <typename T, int FMT>
__device__ __forceinline__ void load_vectors(const Tensor& t, uint32_t first, int shift) {
  using F = Format<FMT>;
  uint2 c[kCkptUnroll];
  float s[kCkptUnroll];
  uint32_t row[kCkptUnroll], at[kCkptUnroll];
  bool on[kCkptUnroll];
#pragma unroll
  for (int u = 0; u < kCkptUnroll; ++u) {
    const uint32_t i = first + u * kCkptThreads + threadIdx.x;
    on[u] = i < t.vecs;
    row[u] = quot(i, t.row_vecs);
    at[u] = i - row[u] * t.row_vecs.d;
    c[u] = make_uint2(0u, 0u);
    s[u] = 0.f;
    if (on[u]) {
      c[u] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.codes) + (size_t)row[u] * t.C + at[u] * 8));
      s[u] = __ldg(t.scales + (size_t)row[u] * t.nb + (at[u] >> shift));
    }
  }
#pragma unroll
  for (int u = 0; u < kCkptUnroll; ++u) {
    if (!on[u]) continue;
    float f[8];
    F::decode(c[u], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= s[u];
    store8(static_cast<T*>(const_cast<void*>(t.x)), row_offset(t, row[u]) + at[u] * 8, f);
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kCkptThreads) ckpt_load_kernel(const __grid_constant__ Tensors a, int shift) {
  uint32_t first;
  const Tensor& t = tensor_of(a, blockIdx.x, &first);
  load_vectors<T, FMT>(t, first, shift);
}

// Start of the attention backward from 8-bit tensors, in one launch: the
// first thread blocks bring q, k and v back as bf16 (the operand type of the
// products), the rest form delta = rowsum(dO * O) with O straight from its
// codes, O itself never being stored, and lse * log2(e).
struct DeltaArgs {
  const uint8_t* codes;  // (B, H, Nr, D)
  const float* scales;
  const __nv_bfloat16* dout;
  const float* lse;
  float* delta;
  float* lse2;
  uint32_t rows;  // B * H * N, N padded to whole tiles
  FastDiv N, H;
  int Nr, nb;
  int64_t sb, sh, sn;  // of dout
};
constexpr int row_lanes(int D) { return D == 128 ? 16 : D == 64 ? 8 : 4; }  // divides D / 8 and a warp

template <int D, int FMT>
__global__ void __launch_bounds__(kCkptThreads)
    bwd_ckpt_prologue_kernel(const __grid_constant__ Tensors a, uint32_t load_blocks, const DeltaArgs p, int shift) {
  if (blockIdx.x < load_blocks) {
    uint32_t first;
    const Tensor& t = tensor_of(a, blockIdx.x, &first);
    load_vectors<__nv_bfloat16, FMT>(t, first, shift);
    return;
  }
  using F = Format<FMT>;
  constexpr int VEC = D / 8, LPR = row_lanes(D), RPB = kCkptThreads / LPR;
  const uint32_t row = (blockIdx.x - load_blocks) * RPB + threadIdx.x / LPR;
  const int sub = threadIdx.x % LPR;
  const bool in = row < p.rows;
  const uint32_t bh = quot(in ? row : 0u, p.N), n = (in ? row : 0u) - bh * p.N.d;
  const uint32_t b = quot(bh, p.H), h = bh - b * p.H.d;
  // rows past the caller's N get P = 0 (lse = +inf) and delta = 0, so they add nothing
  const bool live = in && n < (uint32_t)p.Nr;
  const size_t r = (size_t)bh * p.Nr + n;
  const __nv_bfloat16* dout = p.dout + (size_t)b * p.sb + (size_t)h * p.sh + (size_t)n * p.sn;
  float acc = 0.f;
  if (live) {
#pragma unroll
    for (int v = sub; v < VEC; v += LPR) {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(p.codes + r * D) + v);
      const float s = __ldg(p.scales + r * p.nb + (v >> shift));
      Vec8<__nv_bfloat16> g;
      g.load(dout, v * 8);
      float o[8], d[8];
      F::decode(c, o);
      g.floats(d);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(o[i], d[i], sum);
      acc = fmaf(s, sum, acc);
    }
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(~0u, acc, o);
  if (in && sub == 0) {
    p.delta[row] = acc;
    p.lse2[row] = live ? p.lse[r] * 1.4426950408889634f : INFINITY;
  }
}

// The tensors' descriptions; vectors per row counted with whole blocks for a save.
uint32_t describe(const CkptTensor* x, int count, int G, bool save, Tensors* a) {
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
    const uint32_t rv = save ? (uint32_t)t.nb * (G / 8) : (uint32_t)x[i].C / 8;
    t.rows = (uint32_t)((int64_t)x[i].B * x[i].H * x[i].N);
    t.vecs = t.rows * rv;
    t.row_vecs = fast_div(rv);
    t.N = fast_div(x[i].N);
    t.H = fast_div(x[i].H);
    t.sb = x[i].s_b;
    t.sh = x[i].s_h;
    t.sn = x[i].s_n;
    t.contiguous = (x[i].N == 1 || t.sn == t.C) && (x[i].H == 1 || t.sh == (int64_t)x[i].N * t.C) &&
                   (x[i].B == 1 || t.sb == (int64_t)x[i].H * x[i].N * t.C);
    blocks += (uint32_t)(((uint64_t)t.vecs + kCkptThreads * kCkptUnroll - 1) / (kCkptThreads * kCkptUnroll));
  }
  return blocks;
}
int lane_shift(int G) { return G == 32 ? 2 : G == 64 ? 3 : 4; }

template <typename T, int FMT>
void save_launch(const Tensors& a, uint32_t blocks, int G, cudaStream_t st) {
  if (G == 32)
    ckpt_save_kernel<T, FMT, 4><<<blocks, kCkptThreads, 0, st>>>(a);
  else if (G == 64)
    ckpt_save_kernel<T, FMT, 8><<<blocks, kCkptThreads, 0, st>>>(a);
  else
    ckpt_save_kernel<T, FMT, 16><<<blocks, kCkptThreads, 0, st>>>(a);
}

template <int D>
void prologue_launch(int format, const Tensors& a, uint32_t load_blocks, const DeltaArgs& d, int shift, cudaStream_t st) {
  constexpr int RPB = kCkptThreads / row_lanes(D);
  const uint32_t blocks = load_blocks + (d.rows + RPB - 1) / RPB;
  if (format == PA_CKPT_INT8)
    bwd_ckpt_prologue_kernel<D, PA_CKPT_INT8><<<blocks, kCkptThreads, 0, st>>>(a, load_blocks, d, shift);
  else
    bwd_ckpt_prologue_kernel<D, PA_CKPT_E4M3><<<blocks, kCkptThreads, 0, st>>>(a, load_blocks, d, shift);
}

}  // namespace

cudaError_t launch_ckpt_save(const CkptTensor* x, int count, bool f32, int format, int block, cudaStream_t st) {
  Tensors a{};
  const uint32_t blocks = describe(x, count, block, true, &a);
  if (f32)
    format == PA_CKPT_INT8 ? save_launch<float, PA_CKPT_INT8>(a, blocks, block, st)
                           : save_launch<float, PA_CKPT_E4M3>(a, blocks, block, st);
  else
    format == PA_CKPT_INT8 ? save_launch<__nv_bfloat16, PA_CKPT_INT8>(a, blocks, block, st)
                           : save_launch<__nv_bfloat16, PA_CKPT_E4M3>(a, blocks, block, st);
  return cudaGetLastError();
}

cudaError_t launch_ckpt_load(const CkptTensor* x, int count, bool f32, int format, int block, cudaStream_t st) {
  Tensors a{};
  const uint32_t blocks = describe(x, count, block, false, &a);
  const int shift = lane_shift(block);
  if (f32 && format == PA_CKPT_INT8)
    ckpt_load_kernel<float, PA_CKPT_INT8><<<blocks, kCkptThreads, 0, st>>>(a, shift);
  else if (f32)
    ckpt_load_kernel<float, PA_CKPT_E4M3><<<blocks, kCkptThreads, 0, st>>>(a, shift);
  else if (format == PA_CKPT_INT8)
    ckpt_load_kernel<__nv_bfloat16, PA_CKPT_INT8><<<blocks, kCkptThreads, 0, st>>>(a, shift);
  else
    ckpt_load_kernel<__nv_bfloat16, PA_CKPT_E4M3><<<blocks, kCkptThreads, 0, st>>>(a, shift);
  return cudaGetLastError();
}

cudaError_t launch_bwd_ckpt_prologue(const AttnParams& p, int D, const RowStrides& rs, const CkptTensor (&qkv)[3],
                                     const void* out_codes, const float* out_scales, int format, int block,
                                     cudaStream_t st) {
  Tensors a{};
  const uint32_t load_blocks = describe(qkv, 3, block, false, &a);
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
  d.sb = rs.q_b;
  d.sh = rs.q_h;
  d.sn = rs.q_n;
  const int shift = lane_shift(block);
  if (D == 64)
    prologue_launch<64>(format, a, load_blocks, d, shift, st);
  else if (D == 96)
    prologue_launch<96>(format, a, load_blocks, d, shift, st);
  else
    prologue_launch<128>(format, a, load_blocks, d, shift, st);
  return cudaGetLastError();
}

}  // namespace pa
