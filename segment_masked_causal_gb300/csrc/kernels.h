// kernels.h -- host-side launchers of the packed-attention kernels (internal).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/pa.h"
#include "common.cuh"

namespace pa {

// PA_OK when the current device is compute capability 10.3 with enough
// opt-in shared memory for the kernels, else PA_ERR_ARCH (or PA_ERR_CUDA if
// the query itself fails). Cached per device.
pa_status device_check();

// Launch attribute with which a kernel may start before the one ahead of it on
// the stream has ended, once every block of that one has started and said so
// (griddepcontrol.launch_dependents). It runs griddepcontrol.wait before it
// reads what that one writes, and somewhere before its end in any case, so that
// what follows on the stream finds both finished.
inline cudaLaunchAttribute programmatic_launch() {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

// Launch attribute: clusters of two CTAs along x.
inline cudaLaunchAttribute cluster_pair() {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = 2;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
  return a;
}

// Element strides of the (B, H, N, D) tensors the kernels read and write in
// place (D contiguous): q, out, dout and dq use the q_* strides, k, v, dk and
// dv the k_* strides.
struct RowStrides {
  int64_t q_n, q_h, q_b, k_n, k_h, k_b;
};
inline RowStrides contiguous_rows(int Hq, int Hkv, int N, int D) {
  return RowStrides{D, (int64_t)N * D, (int64_t)Hq * N * D, D, (int64_t)N * D, (int64_t)Hkv * N * D};
}
inline bool is_contiguous(const RowStrides& s, int Hq, int Hkv, int N, int D) {
  const RowStrides c = contiguous_rows(Hq, Hkv, N, D);
  return s.q_n == c.q_n && s.q_h == c.q_h && s.q_b == c.q_b && s.k_n == c.k_n && s.k_h == c.k_h && s.k_b == c.k_b;
}

// Tile table (B, T) x {smin, smax, kv_lo, q_hi} and the two work lists; also
// clears the status word.
cudaError_t launch_tile_table(const AttnParams& p, int4* tiles, cudaStream_t st);
// delta[b, h, i] = sum_c dO[b, h, i, c] * O[b, h, i, c] (fp32), and lse2 = lse * log2(e);
// also zeroes the rows of p.dq_acc when it is non-null.
cudaError_t launch_delta(const AttnParams& p, int D, const RowStrides& rs, cudaStream_t st);
// Self-test of the bounded waits: one warp waits on an mbarrier nothing arrives on.
cudaError_t launch_wait_timeout_selftest(uint32_t* status, cudaStream_t st);
cudaError_t launch_exp2_fma_selftest(const float* x, float* y, int64_t n, cudaStream_t st);
cudaError_t launch_fwd(const AttnParams& p, int D, const RowStrides& rs, const void* q, const void* k, const void* v,
                       cudaStream_t st);
// in: the strides of q, k and v where they are not those of dout and the gradients.
// fp32_p: dS from P before its rounding to bf16 (see bwd_dkv.cu).
// beside: launch dQ programmatically behind the kernel ahead of it (dK/dV),
// of which it needs nothing.
cudaError_t launch_bwd_dq(const AttnParams& p, int D, const RowStrides& rs, const void* q, const void* k,
                          const void* v, const void* dout, cudaStream_t st, const RowStrides* in = nullptr,
                          bool beside = false);
cudaError_t launch_bwd_dkv(const AttnParams& p, int D, const RowStrides& rs, const void* q, const void* k,
                           const void* v, const void* dout, cudaStream_t st, const RowStrides* in = nullptr,
                           bool fp32_p = false);
// Single-pass backward: dK, dV and the fp32 dQ accumulator p.dq_acc (zeroed
// beforehand), then p.dq = the accumulator rounded to bf16.
cudaError_t launch_bwd_fused(const AttnParams& p, int D, const RowStrides& rs, const void* q, const void* k,
                             const void* v, const void* dout, cudaStream_t st);
cudaError_t launch_dq_round(const AttnParams& p, int D, cudaStream_t st);

// A (B, H, N, D) bf16 or fp32 tensor with element strides sb, sh, sn (16-byte
// multiples) and contiguous D, against the kernels' contiguous bf16
// (B, H, Np, D) copy; vec = D / 8 bf16 16-byte vectors per token row.
struct RowsView {
  int B, H, N, Np, vec;
  int64_t sb, sh, sn;
};
// Copies in (tail rows n >= N zero) and out (real rows only); f32: the
// caller's tensor is fp32 (rounded to bf16 in, widened out).
cudaError_t launch_stage_rows_in(void* dst, const void* src, const RowsView& v, bool f32, cudaStream_t st);
cudaError_t launch_stage_rows_out(void* dst, const void* src, const RowsView& v, bool f32, cudaStream_t st);
// (R, N) 32-bit words to (R, Np) with a tail of 0 or of the row's last word, and back.
cudaError_t launch_stage_words_in(void* dst, const void* src, uint64_t R, int N, int Np, bool repeat_last,
                                  cudaStream_t st);
cudaError_t launch_stage_words_out(void* dst, const void* src, uint64_t R, int N, int Np, cudaStream_t st);

// Fused linear cross-entropy forward. The vocabulary's 128-row tiles are cut
// into `splits` runs of `per` tiles, one CTA column each; `part` holds
// 3 * splits * N floats of per-split partial results.
struct LceSplit {
  int splits, per;
};
constexpr int kLceMaxSplits = 64;
LceSplit lce_split(int N, int V, int slots);
// CTAs of the cross-entropy kernel resident at once on the current device.
int lce_slots();
// Fused linear cross-entropy backward: the vocabulary in chunks of vc rows;
// workspace after the 256-byte status region: the fp32 dH accumulator (only
// with more than one chunk), dz (N x vc) and dz^T (vc x ld_dzt), bf16.
struct LceBwdLayout {
  int vc, chunks, ld_dzt;
  size_t acc, dz, dzt, bytes;
};
LceBwdLayout lce_bwd_layout(int N, int V, int D);
cudaError_t launch_lce_bwd(int N, int V, int D, const void* hidden, const void* head, const int32_t* targets,
                           const float* lse, const float* g, void* dhidden, void* dhead, void* ws, uint32_t* status,
                           cudaStream_t st);
cudaError_t launch_lce_fwd(int N, int V, int D, const void* hidden, const void* head, const int32_t* targets,
                           float* nll, float* lse, float* target_logit, float* part, uint32_t* status,
                           cudaStream_t st);

// C (M x N, N contiguous, a multiple of 64) from A (M x K, K contiguous, boxes
// of 128 rows x 64) and B (K x N, N contiguous, boxes of 64 rows x 64) on the
// tensor cores. splits > 1 cuts the contraction into that many runs, each
// with an accumulator of its own (acc + run * M * N): kAccInit or kAccAdd
// only, joined by launch_sum_splits.
enum GemmMode : int { kStoreBf16 = 0, kAccInit = 1, kAccAdd = 2, kAccFinal = 3 };
// kInOrder: an ordinary launch. kAfter: a programmatic one that waits for the
// kernel ahead before it reads or writes memory (and before it lets a kernel
// behind it start). kBeside: a programmatic one that needs nothing of the kernel
// ahead, only of those before it, so the kernel ahead is kInOrder or kAfter.
enum GemmOrder : int { kInOrder = 0, kAfter = 1, kBeside = 2 };
struct GemmCall {
  int M, N, K;
  int mode;          // GemmMode
  const CUtensorMap* lo;  // null, or A's second term: the product of (A + lo) and B
  bool stay;         // with lo, K <= 128 and one run: a CTA keeps its columns' B
  int splits;        // <= 1: one run
  int sms;           // at most this many of the device's SMs; 0: all
  __nv_bfloat16* c;  // bf16 result (kStoreBf16: the product; kAccFinal: accumulator + product)
  float* acc;        // fp32 accumulator (kAccInit: set; kAccAdd: add; kAccFinal: read)
  uint32_t* status;
  int order;         // GemmOrder
};
cudaError_t launch_gemm(const CUtensorMap& tA, const CUtensorMap& tB, const GemmCall& gc, cudaStream_t st);
// The number of runs that makes an M x N x K product (A in `terms` terms)
// shortest on `slots` SMs; no run is empty, or longer than gemm_least_runs's.
int gemm_splits(int M, int N, int K, int slots, int terms);
// The fewest runs of at most 65,536 terms, none empty. The tensor cores cut what
// an addition of 16 products to an fp32 sum leaves over, always towards zero: a run
// loses about 2e-8 of its sum at each (8.6 million tokens in one run left dW 1.0e-2
// of its norm short), 8e-5 at this length.
int gemm_least_runs(int K);
cudaError_t launch_sum_splits(const float* acc, int splits, size_t n, __nv_bfloat16* out, cudaStream_t st);

// Token log probabilities. The vocabulary is cut into runs of whole units of
// 32 rows, one CTA column each.
constexpr int kLogpUnit = 32;
constexpr int kLogpMaxSplits = 160;
constexpr int kLogpMaxTop = 32;
int logp_max_splits(int N, int V);
struct LogpPlan {
  bool pair;  // two CTAs per product
  int splits, per, width;  // units per split and per tile of it
};
LogpPlan logp_plan(int N, int V, int D, int sms);
struct LogpFwdLayout {
  size_t part, cand, bytes;  // after the 256-byte status region
};
LogpFwdLayout logp_fwd_layout(int N, int V, int top);
cudaError_t launch_logp_fwd(int N, int V, int D, float temperature, int top, const void* hidden, const void* head,
                            const int32_t* targets, float* logp, float* lse, float* entropy, int32_t* top_ids,
                            float* top_logp, void* ws, cudaStream_t st);
struct LogpBwdLayout {
  int terms;  // of dz, bf16 each
  int vc, chunks, ld_dzt;
  int splits, splits_beside;  // runs of dH's contraction: on all SMs, and on those that dW leaves
  int splits_w;               // runs of dW's
  size_t acc, acc_w, dz, dzt, bytes;
};
LogpBwdLayout logp_bwd_layout(int N, int V, int D);
cudaError_t launch_logp_bwd(int N, int V, int D, float temperature, const void* hidden, const void* head,
                            const int32_t* targets, const float* lse, const float* entropy, const float* g_logp,
                            const float* g_entropy, void* dhidden, void* dhead, void* ws, cudaStream_t st);

// Activations in 8 bits (ckpt.cu): x (B, H, N, C) with element strides s_b,
// s_h, s_n against contiguous codes (B, H, N, C) and scales (B, H, N, ceil(C / block)).
struct CkptTensor {
  const void* x;  // save: source; load: destination
  void* codes;
  float* scales;
  int B, H, N, C;
  int64_t s_b, s_h, s_n;
};
cudaError_t launch_ckpt_save(const CkptTensor* x, int count, bool f32, int format, int block, cudaStream_t st);
cudaError_t launch_ckpt_load(const CkptTensor* x, int count, bool f32, int format, int block, cudaStream_t st);
// Start of the attention backward from 8-bit tensors: q, k and v to bf16, and
// delta and lse2 of p with the output taken from its codes.
cudaError_t launch_bwd_ckpt_prologue(const AttnParams& p, int D, const RowStrides& rs, const CkptTensor (&qkv)[3],
                                     const void* out_codes, const float* out_scales, int format, int block,
                                     cudaStream_t st);

}  // namespace pa
