// rope.cu -- positions of packed rows, and rotary positions applied to queries
// and keys, forward and backward.
//
// Both are bound by memory: the rotation reads and writes each element once.
// A thread holds the cosines and sines of one unit of pairs at one token
// (rope.cuh) and takes that unit of many heads, so that they are computed once
// for a run of heads; several heads' loads are in flight at a time. The backward is
// the rotation by minus the angle (a rotation's transpose), times the same
// amplitude.
//
// Measured: 8,192 tokens of 32 and 8 bf16 heads of 128 take 25.7 us, 0.96 of the copy
// bandwidth, the gradients of 16,384 tokens with half of each head turned 49.2 us, all of it
// (88 us with vectors of 16 bytes and a form of its own for the part that stays). Small
// calls are their launches: 666 tokens in fp32 with their positions 6.2 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "rope.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 128;

struct RopeArgs {
  pa_rotary rope;
  RopeTensor t[PA_ROPE_MAX_TENSORS];
  int count, heads;  // tensors, and their heads in all
  int run;           // heads per block
  int tokens;        // B * N
  int N, D;
  RopeUnits u;
  const int32_t* positions;
  float sign;
};

template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per = kRopeThreads / p.u.units;
  const int at = threadIdx.x / p.u.units, u = threadIdx.x - at * p.u.units;
  const int64_t here = (int64_t)blockIdx.x * per + at;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (at >= per || here >= p.tokens) return;
  const int token = (int)here, b = token / p.N, n = token - b * p.N;
  const RopeUnit<T, VEC, INTER> r(p.D, p.rope.rot, p.u.turning, u);
  float c[VEC], s[VEC];
  if (r.turn) {
    const int32_t pos = p.positions ? p.positions[token] : n;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      rope_cos_sin(p.rope.turns[u * VEC + i], pos, p.rope.amplitude, c[i], s[i]);
      s[i] *= p.sign;
    }
  }
  int h = blockIdx.y * p.run;  // among all tensors' heads
  const int end = min(h + p.run, p.heads);
  int k = 0, first = 0;  // tensor, and its first head
  while (h < end) {
    while (h >= first + p.t[k].H) first += p.t[k++].H;
    const RopeTensor& t = p.t[k];
    const int stop = min(end, first + t.H);
    r.move(static_cast<const T*>(t.x) + b * t.x_b + n * t.x_n + (int64_t)(h - first) * t.x_h, t.x_h,
           static_cast<T*>(t.y) + b * t.y_b + n * t.y_n + (int64_t)(h - first) * t.y_h, t.y_h, stop - h, r.turn, c, s);
    h = stop;
  }
}

template <typename T, int VEC>
cudaError_t launch_vec(RopeArgs& a, bool rest, cudaStream_t st) {
  a.u = rope_units(a.D, a.rope.rot, VEC, rest);
  const int per = kRopeThreads / a.u.units;
  const int64_t blocks = ((int64_t)a.tokens + per - 1) / per;
  // Heads of a block: all of them, or fewer where the tokens alone do not fill the device.
  const int64_t want = 152 * 8;
  a.run = (int)std::min<int64_t>(a.heads, std::max<int64_t>(4, (int64_t)a.heads * blocks / want));
  cudaLaunchAttribute attr = programmatic_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)((a.heads + a.run - 1) / a.run));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, a.rope.layout == PA_ROPE_INTERLEAVED ? rope_kernel<T, VEC, true> : rope_kernel<T, VEC, false>, a);
}

// Position of each token in its run of equal ids. A block takes 1,024 tokens of a row; a
// thread's latest start of a run at or before each of its four tokens comes from a scan
// of maxima. The start of the run that the block's first token continues lies before the
// block: the 4,096 ids there are read along with its own, those further back only if
// none of them starts one. Bound by the round trips: one, and one more for each 4,096 tokens of
// a longer run. Over long rows that would be quadratic, so there a kernel goes ahead that leaves each block's
// last start in the place of its last token's position, as a negative number, and what lies further back
// than 4,096 tokens is looked up in those, 1,024 blocks at a time. A place may hold its position
// by then: that gives the start of its run as well, and with it the end of the search.
constexpr int kPosThreads = 256, kPosPer = 4, kPosTile = kPosThreads * kPosPer, kPosBack = 16, kPosMarks = 4;
// The first kernel costs 1.2 us of a row of short runs (32,768 tokens 4.8 -> 6.0 us) and saves 3 us for each 4,096
// tokens of a long one (one run of 32,768 tokens 25.6 -> 6.4 us, of 2^20 1,054 -> 15, of 2^24 153,500 -> 200).
constexpr int kPosLong = 32768;

// The latest start of a run among a block's tokens, or -1: m in the place of the last one's position.
__device__ __forceinline__ int32_t pos_mark(int m) { return -2 - m; }
__device__ __forceinline__ int pos_start(int32_t word, int n) { return word < 0 ? -2 - word : n - word; }

__global__ void __launch_bounds__(kPosThreads) positions_mark_kernel(const int32_t* __restrict__ seg, int32_t* positions, int N,
                                                                     int tiles) {
  __shared__ int sh[kPosThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x / tiles, n0 = (blockIdx.x - b * tiles) * kPosTile;
  const int32_t* row = seg + (int64_t)b * N;
  int last = -1;
#pragma unroll
  for (int i = 0; i < kPosPer; ++i) {
    const int n = n0 + i * kPosThreads + (int)threadIdx.x;
    if (n < N && (n == 0 || row[n] != row[n - 1])) last = n;
  }
  last = __reduce_max_sync(~0u, last);
  if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = last;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < kPosThreads / 32; ++w) last = max(last, sh[w]);
    positions[(int64_t)b * N + min((int64_t)n0 + kPosTile, (int64_t)N) - 1] = pos_mark(last);
  }
}

__global__ void __launch_bounds__(kPosThreads) positions_kernel(const int32_t* __restrict__ seg, int32_t* positions, int N,
                                                                int tiles, bool marked) {
  __shared__ int sh[kPosThreads / 32], back[kPosThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x / tiles, n0 = (blockIdx.x - b * tiles) * kPosTile;
  const int32_t* row = seg + (int64_t)b * N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // whether a run starts at n; false outside the row
  const auto starts = [&](int n) { return n >= 0 && n < N && (n == 0 || row[n] != row[n - 1]); };
  // the latest start among the kPosBack * kPosThreads tokens before hi that this thread sees
  const auto look_back = [&](int hi) {
    bool at[kPosBack];
#pragma unroll
    for (int j = 0; j < kPosBack; ++j) at[j] = starts(hi - 1 - (j * kPosThreads + (int)threadIdx.x));
    int found = -1;
#pragma unroll
    for (int j = kPosBack - 1; j >= 0; --j)
      if (at[j]) found = hi - 1 - (j * kPosThreads + (int)threadIdx.x);
    return found;
  };
  bool own[kPosPer];
#pragma unroll
  for (int i = 0; i < kPosPer; ++i) own[i] = starts(n0 + threadIdx.x * kPosPer + i);
  int found = look_back(n0);
  int at[kPosPer];  // latest start at or before token n0 + 4 thread + i, as far as this thread sees
  int last = -1;
#pragma unroll
  for (int i = 0; i < kPosPer; ++i) {
    if (own[i]) last = n0 + threadIdx.x * kPosPer + i;
    at[i] = last;
  }
  int before = last;  // inclusive scan over the warp, then over the block
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, before, o);
    if (lane >= o) before = max(before, v);
  }
  found = __reduce_max_sync(~0u, found);
  if (lane == 31) {
    sh[warp] = before;
    back[warp] = found;
  }
  int excl = __shfl_up_sync(~0u, before, 1);
  if (lane == 0) excl = -1;
  __syncthreads();
  int from = -1;
#pragma unroll
  for (int w = 0; w < kPosThreads / 32; ++w) {
    if (w < warp) excl = max(excl, sh[w]);
    from = max(from, back[w]);
  }
  const auto look_up = [&](int hi) {  // the same among the marks of the kPosMarks * kPosThreads tiles before tile hi
    int start = -1;
#pragma unroll
    for (int j = 0; j < kPosMarks; ++j) {
      const int t = hi - 1 - (j * kPosThreads + (int)threadIdx.x), n = t * kPosTile + kPosTile - 1;
      if (t >= 0) start = max(start, pos_start(*(const volatile int32_t*)(positions + (int64_t)b * N + n), n));
    }
    return start;
  };
  const int unit = marked ? kPosTile : 1, step = marked ? kPosThreads * kPosMarks : kPosThreads * kPosBack;
  for (int hi = (n0 - kPosThreads * kPosBack) / unit; hi > 0 && from < 0; hi -= step) {
    found = __reduce_max_sync(~0u, marked ? look_up(hi) : look_back(hi));
    __syncthreads();
    if (lane == 0) back[warp] = found;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPosThreads / 32; ++w) from = max(from, back[w]);
  }
#pragma unroll
  for (int i = 0; i < kPosPer; ++i) {
    const int n = n0 + threadIdx.x * kPosPer + i;
    if (n < N) positions[(int64_t)b * N + n] = n - max(max(at[i], excl), from);
  }
}

}  // namespace

cudaError_t launch_rope(const pa_rotary& rope, const RopeTensor* t, int count, int B, int N, int D, bool f32, bool backward,
                        const int32_t* positions, cudaStream_t st) {
  RopeArgs a{};
  a.rope = rope;
  a.count = count;
  bool in_place = true;
  uint64_t bits = 0;  // of every address and stride, in bytes
  const int size = f32 ? 4 : 2;
  for (int i = 0; i < count; ++i) {
    a.t[i] = t[i];
    a.heads += t[i].H;
    in_place = in_place && t[i].x == t[i].y;
    bits |= reinterpret_cast<uintptr_t>(t[i].x) | reinterpret_cast<uintptr_t>(t[i].y);
    if (B > 1) bits |= (uint64_t)(t[i].x_b | t[i].y_b) * size;
    if (t[i].H > 1) bits |= (uint64_t)(t[i].x_h | t[i].y_h) * size;
    if (N > 1) bits |= (uint64_t)(t[i].x_n | t[i].y_n) * size;
  }
  a.tokens = (int)((int64_t)B * N);
  a.N = N;
  a.D = D;
  a.positions = positions;
  a.sign = backward ? -1.f : 1.f;
  // Vectors of 32 bytes where every row starts on them and both parts of it are whole numbers
  // of units, else of 16, else (a rotated part of 8 pairs and 8 more) of 8. In place the rest stays.
  const auto fits = [&](int vec) {
    const uint64_t bytes = (uint64_t)vec * size;
    return rope.rot % (2 * vec) == 0 && (in_place || (D - rope.rot) % vec == 0) && (bits % bytes) == 0 && (uint64_t)D * size % bytes == 0;
  };
  if (f32) return fits(8) ? launch_vec<float, 8>(a, !in_place, st) : launch_vec<float, 4>(a, !in_place, st);
  if (fits(16)) return launch_vec<__nv_bfloat16, 16>(a, !in_place, st);
  return fits(8) ? launch_vec<__nv_bfloat16, 8>(a, !in_place, st) : launch_vec<__nv_bfloat16, 4>(a, !in_place, st);
}

cudaError_t launch_positions(int B, int N, const int32_t* seg, int32_t* positions, cudaStream_t st) {
  const int tiles = (int)(((int64_t)N + kPosTile - 1) / kPosTile);
  cudaLaunchAttribute attr = programmatic_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)B * tiles));
  cfg.blockDim = dim3(kPosThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool marked = N > kPosLong;
  if (marked) {
    const cudaError_t e = cudaLaunchKernelEx(&cfg, positions_mark_kernel, seg, positions, N, tiles);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, positions_kernel, seg, positions, N, tiles, marked);
}

}  // namespace pa
