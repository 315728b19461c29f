// append.cu -- new tokens' keys and values into a paged cache, with the rotation
// of keys and queries on the way.
//
// Bound by memory (q, k and v read once, q_out and the places written once) from a
// few hundred tokens on, by latency below: a token's place hangs on its sequence's
// row of q_start, its length and its page number, one after the other. A block
// finds the sequences of its tokens in a copy of q_start in shared memory (in
// global memory past kStarts of them); its threads then hold the cosines and
// sines of one unit of pairs of a token for a run of heads, as in rope.cu.
#include <cuda_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "paged.cuh"
#include "rope.cuh"

namespace pa {
namespace {

constexpr int kAppendThreads = 256, kStarts = 1024;

struct AppendArgs {
  PagedArgs p;
  pa_rotary rope;  // rot 0: nothing is rotated
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_pages, *v_pages;
  int64_t n_t, n_h;
  const int32_t* positions;
  int heads, run;      // q's, k's and v's heads one behind the other, and how many a block takes
  int units, turning;  // units per row: `turning` ones of pairs, then eight elements each
};

// Heads h .. stop - 1 of one token: `turn` units rotated, others copied.
template <int VEC, bool INTER>
__device__ __forceinline__ void move_heads(const __nv_bfloat16* x, int64_t xs, __nv_bfloat16* y, int64_t ys, int n, bool pairs,
                                           bool turn, int u, int half, int e, const float (&c)[VEC], const float (&s)[VEC]) {
  constexpr int U = 4;
  if (pairs) {
    for (int h = 0; h < n; h += U, x += U * xs, y += U * ys) {
      RopeUnit<__nv_bfloat16, VEC, INTER> r[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < n) r[i].load(x + i * xs, u, half);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < n) {
          if (turn) r[i].rotate(c, s);
          r[i].store(y + i * ys, u, half);
        }
    }
  } else {
    for (int h = 0; h < n; h += U, x += U * xs, y += U * ys) {
      PlainUnit<__nv_bfloat16> r[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < n) r[i].load(x + i * xs + e);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < n) r[i].store(y + i * ys + e);
    }
  }
}

template <int VEC, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ int starts[kStarts + 1];
  const PagedArgs& p = a.p;
  const int per = kAppendThreads / a.units;
  const int at = threadIdx.x / a.units, u = threadIdx.x - at * a.units;
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
  const int rot = a.rope.rot, half = rot / 2, e = rot + 8 * (u - a.turning);
  const bool pairs = u < a.turning;
  float c[VEC], sn[VEC];
  if (pairs) {
    const int32_t pos = a.positions ? a.positions[t] : slot;
#pragma unroll
    for (int i = 0; i < VEC; ++i) rope_cos_sin(a.rope.turns[u * VEC + i], pos, a.rope.amplitude, c[i], sn[i]);
  }
  const int nq = a.q ? p.Hq : 0;
  int h = blockIdx.y * a.run;
  const int end = min(h + a.run, a.heads);
  if (h < nq) {
    const int stop = min(end, nq);
    move_heads<VEC, INTER>(a.q + t * p.q_t + h * p.q_h, p.q_h, a.q_out + t * p.o_t + h * p.o_h, p.o_h, stop - h, pairs, true, u,
                           half, e, c, sn);
    h = stop;
  }
  if (place < 0) return;
  for (int which = 0; which < 2; ++which) {  // keys, values
    const int first = nq + which * p.Hkv, stop = min(end, first + p.Hkv);
    if (h >= first && h < stop) {
      move_heads<VEC, INTER>((which ? a.v : a.k) + t * a.n_t + (h - first) * a.n_h, a.n_h,
                             (which ? a.v_pages : a.k_pages) + place + (h - first) * p.p_h, p.p_h, stop - h, pairs, which == 0,
                             u, half, e, c, sn);
      h = stop;
    }
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
  const int vec = a.rope.rot % 16 ? 4 : 8;  // as in rope.cu
  a.turning = a.rope.rot / (2 * vec);
  a.units = a.turning + (p.D - a.rope.rot) / 8;
  const int per = kAppendThreads / a.units, blocks = (p.T + per - 1) / per;
  const int64_t want = 152 * 8;
  a.run = (int)std::min<int64_t>(a.heads, std::max<int64_t>(4, (int64_t)a.heads * blocks / want));
  const dim3 grid((unsigned)blocks, (unsigned)((a.heads + a.run - 1) / a.run));
  const bool inter = rope && rope->layout == PA_ROPE_INTERLEAVED;
  const auto kfn = vec == 8 ? (inter ? append_kernel<8, true> : append_kernel<8, false>)
                            : (inter ? append_kernel<4, true> : append_kernel<4, false>);
  kfn<<<grid, kAppendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
