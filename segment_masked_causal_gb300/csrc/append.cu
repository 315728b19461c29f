// append.cu -- new tokens' keys and values into a paged cache, with the rotation
// of keys and queries on the way.
//
// Bound by memory (q, k and v read once, q_out and the places written once) from a
// few hundred tokens on, by latency below: a token's place hangs on its sequence's
// row of q_start, its length and its page number, one after the other. A block
// finds the sequences of its tokens in a copy of q_start in shared memory (in
// global memory past kStarts of them); its threads then hold the cosines and
// sines of one unit of pairs of a token for a run of heads, as in rope.cu. Measured:
// 8,000 tokens of 32 and 8 heads of 128 31.8 us, 0.91 of the copy bandwidth; one
// token each of 17 sequences 4.5 us with its launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "kernels.h"
#include "paged.cuh"
#include "rope.cuh"

namespace pa {
namespace {

constexpr int kAppendThreads = 128, kStarts = 1024;

struct AppendArgs {
  PagedArgs p;
  pa_rotary rope;  // rot 0: nothing is rotated
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_pages, *v_pages;
  int64_t n_t, n_h;
  const int32_t* positions;
  int heads, run;      // q's, k's and v's heads one behind the other, and how many a block takes
  RopeUnits u;
};

template <int VEC, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ int starts[kStarts + 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const PagedArgs& p = a.p;
  const int per = kAppendThreads / a.u.units;
  const int at = threadIdx.x / a.u.units, u = threadIdx.x - at * a.u.units;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool small = p.S <= kStarts;
  if (small) {
    for (int i = threadIdx.x; i <= p.S; i += kAppendThreads) starts[i] = p.q_start[i];
    __syncthreads();
  }
  const int t = blockIdx.x * per + at;
  if (at >= per || t >= p.T) return;
  const int* from = small ? starts : p.q_start;
  // the last sequence that starts at or before row t, the empty ones among those skipped
  int s = -1;
  for (int hi = p.S; hi - s > 1;) {
    const int mid = (s + hi) >> 1;
    if (from[mid] <= t)
      s = mid;
    else
      hi = mid;
  }
  if (s < 0 || from[s + 1] <= t) return;  // nobody's row
  const SeqRows r = seq_rows(p, s);
  const int slot = r.base() + (t - r.a);
  int64_t place = -1;
  if (slot >= 0 && slot / p.page < p.width) {
    const int id = p.page_table[(int64_t)s * p.width + slot / p.page];
    if (id >= 0 && id < p.pages) place = id * p.p_p + (int64_t)(slot % p.page) * p.p_n;
  }
  const RopeUnit<__nv_bfloat16, VEC, INTER> unit(p.D, a.rope.rot, a.u.turning, u);
  float c[VEC], sn[VEC];
  if (unit.turn) {
    const int32_t pos = a.positions ? a.positions[t] : slot;
#pragma unroll
    for (int i = 0; i < VEC; ++i) rope_cos_sin(a.rope.turns[u * VEC + i], pos, a.rope.amplitude, c[i], sn[i]);
  }
  // this block's heads of q, k and v, one behind the other
  const int nq = a.q ? p.Hq : 0, begin = blockIdx.y * a.run, end = min(begin + a.run, a.heads);
#pragma unroll 1
  for (int which = 0; which < 3; ++which) {
    const int first = which == 0 ? 0 : nq + (which - 1) * p.Hkv, last = which == 0 ? nq : first + p.Hkv;
    const int h0 = max(begin, first), n = min(end, last) - h0, h = h0 - first;
    if (n <= 0 || (which > 0 && place < 0)) continue;
    const __nv_bfloat16* x = which == 0 ? a.q + t * p.q_t + h * p.q_h : (which == 1 ? a.k : a.v) + t * a.n_t + h * a.n_h;
    __nv_bfloat16* y = which == 0 ? a.q_out + t * p.o_t + h * p.o_h : (which == 1 ? a.k_pages : a.v_pages) + place + h * p.p_h;
    unit.move(x, which == 0 ? p.q_h : a.n_h, y, which == 0 ? p.o_h : p.p_h, n, unit.turn && which < 2, c, sn);
  }
}

}  // namespace

cudaError_t launch_append(const PagedArgs& p, const pa_rotary* rope, const void* q, const void* k, const void* v, int64_t n_t,
                          int64_t n_h, const int32_t* positions, void* q_out, void* k_pages, void* v_pages, cudaStream_t st) {
  AppendArgs a{};
  a.p = p;
  if (rope) a.rope = *rope;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  a.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  a.n_t = n_t;
  a.n_h = n_h;
  a.positions = positions;
  a.heads = (q ? p.Hq : 0) + 2 * p.Hkv;
  // vectors as in rope.cu
  uint64_t bits = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(q) |
                  reinterpret_cast<uintptr_t>(q_out) | reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages);
  for (int64_t s : {n_t, n_h, p.p_p, p.p_h, p.p_n}) bits |= (uint64_t)s * 2;
  if (q)
    for (int64_t s : {p.q_t, p.q_h, p.o_t, p.o_h}) bits |= (uint64_t)s * 2;
  const auto fits = [&](int vec) {
    return a.rope.rot % (2 * vec) == 0 && (p.D - a.rope.rot) % vec == 0 && bits % (2 * vec) == 0;
  };
  const int vec = fits(16) ? 16 : fits(8) ? 8 : 4;
  a.u = rope_units(p.D, a.rope.rot, vec, true);
  const int per = kAppendThreads / a.u.units, blocks = (p.T + per - 1) / per;
  const int64_t want = 152 * 8;
  a.run = (int)std::min<int64_t>(a.heads, std::max<int64_t>(4, (int64_t)a.heads * blocks / want));
  const bool inter = rope && rope->layout == PA_ROPE_INTERLEAVED;
  const auto kfn = vec == 16  ? (inter ? append_kernel<16, true> : append_kernel<16, false>)
                   : vec == 8 ? (inter ? append_kernel<8, true> : append_kernel<8, false>)
                              : (inter ? append_kernel<4, true> : append_kernel<4, false>);
  cudaLaunchAttribute attr = programmatic_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)((a.heads + a.run - 1) / a.run));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, a);
}

}  // namespace pa
