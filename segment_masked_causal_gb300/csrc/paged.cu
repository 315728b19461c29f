// paged.cu -- attention of a step's new tokens over a paged cache.
//
// One warp per (row of the step, query head): it walks the keys that the row
// sees, 32 lanes over the head dim, with the running maximum and sum of the
// softmax.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"

namespace pa {
namespace {

struct FwdArgs {
  PagedArgs p;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* out;
  float* lse;
};

template <int D>
__global__ void __launch_bounds__(128) paged_kernel(const __grid_constant__ FwdArgs a) {
  const PagedArgs& p = a.p;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(item / p.Hq), h = (int)(item % p.Hq), hk = h / p.G;
  if (t >= p.T) return;
  int s = -1;
  for (int hi = p.S; hi - s > 1;) {
    const int mid = (s + hi) >> 1;
    if (p.q_start[mid] <= t)
      s = mid;
    else
      hi = mid;
  }
  if (s < 0 || p.q_start[s + 1] <= t) return;
  const SeqRows r = seq_rows(p, s);
  const int seen = min(r.base() + (t - r.a) + 1, p.width * p.page);
  constexpr int E = D / 32;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[t * p.q_t + h * p.q_h + e * 32 + lane]) * p.scale_log2, o[e] = 0.f;
  for (int j0 = 0; j0 < seen; j0 += p.page) {
    const int id = p.page_table[(int64_t)s * p.width + j0 / p.page];
    if (id < 0 || id >= p.pages) continue;
    const int64_t at = id * p.p_p + hk * p.p_h + lane;
    const int n = min(p.page, seen - j0);
    for (int j = 0; j < n; ++j) {
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x = fmaf(q[e], __bfloat162float(a.k[at + j * p.p_n + e * 32]), x);
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(~0u, x, i);
      const float mn = fmaxf(m, x), f = exp2f(m - mn), w = exp2f(x - mn);
      l = fmaf(l, f, w);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f, w * __bfloat162float(a.v[at + j * p.p_n + e * 32]));
      m = mn;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[t * p.o_t + h * p.o_h + e * 32 + lane] = __float2bfloat16(o[e] * inv);
  if (lane == 0) a.lse[(int64_t)t * p.Hq + h] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

size_t paged_ws_bytes(int D) { return 256; }

cudaError_t launch_paged_fwd(const PagedArgs& p, const void* q, const void* k_pages, const void* v_pages, void* out, float* lse,
                             void* ws, cudaStream_t st) {
  FwdArgs a{p, static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k_pages),
            static_cast<const __nv_bfloat16*>(v_pages), static_cast<__nv_bfloat16*>(out), lse};
  if (cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(uint32_t), st)) return e;
  const int64_t items = (int64_t)p.T * p.Hq;
  const auto kfn = p.D == 64 ? paged_kernel<64> : p.D == 96 ? paged_kernel<96> : paged_kernel<128>;
  kfn<<<(unsigned)((items + 3) / 4), 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
