// lce.cu -- fused linear cross-entropy: per-token NLL, log-sum-exp and target
// logit of z = H W^T without storing the (N, V) logits, and the backward into
// the hidden states and the head (mlx-train-perf 0.5.1 README, "The fused
// cross-entropy loss": the backward recomputes the tiles it needs instead of
// reading a stored logit matrix).
//
// Forward:
// Grid: (token tiles of 128) x (vocabulary splits). A CTA walks its split's
// vocabulary tiles of 256 rows; for each, the tcgen05 tensor cores form the
// 128 x 256 logit tile in TMEM from 64-wide K slices of H and W that TMA
// streams through a 4-stage ring (one CTA per SM), and four epilogue warps
// (one thread per token, reading its TMEM lane) fold the tile into a running
// maximum and sum of exponentials and pick up the target logit when it falls
// in the tile.
// Two TMEM accumulators let the next tile's products run while the epilogue
// reads the previous one. Each CTA writes its split's (max, sum) per token
// and, for tokens whose target lies in its split, the target logit; a merge
// kernel combines the splits.
//
// Roles: warp 0 lane 0 loads (TMA), warp 1 issues the MMAs (lane 0) and owns
// the TMEM allocation, warps 4..7 are the epilogue (warp % 4 = TMEM lane
// quarter). Every wait is bounded (sm103.cuh).
//
// Backward, over the vocabulary in chunks of Vc rows (so that nothing of size
// N x V is ever held): the same kernel, with an epilogue that turns each
// recomputed logit tile into dz = g (exp(z - lse) - [v == target]) in bf16
// and writes it twice, as dz (tokens x Vc) and dz^T (Vc x tokens); then two
// tcgen05 GEMMs, dW[chunk] = dz^T H (written once per chunk) and
// dH += dz W[chunk] (fp32 in the workspace across chunks, in chunk order, so
// the result does not depend on timing; the last chunk writes bf16 dH).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/pa.h"
#include "kernels.h"
#include "sm103.cuh"
#include "tmap.h"

namespace pa {
namespace {

// The logit tiles are 128 tokens x 256 vocabulary rows, so every product is
// an N = 256 MMA: those keep the tensor pipe at its full rate while the
// epilogue warps' arithmetic shares the issuing warp's SM sub-partition,
// where N = 128 products fall to about 84 of their 64 cycles.
constexpr int kLceStages = 4;                  // 4 x 48 KB: one CTA per SM
constexpr int kLceTile = 128;                  // tokens per CTA
constexpr int kLceVTile = 256;                 // vocabulary rows per tile
constexpr uint32_t kLceSlice = 128 * 128;      // one 128 x 64 bf16 slice of H (128-byte rows), 16 KB
constexpr uint32_t kLceSliceW = 256 * 128;     // one 256 x 64 bf16 slice of W, 32 KB
constexpr uint32_t kLceStage = kLceSlice + kLceSliceW;
constexpr int kLceThreads = 256;
constexpr uint32_t kLceTmemCols = 512;  // two 256-column fp32 accumulators

struct LceMisc {
  uint64_t full[kLceStages], empty[kLceStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t fin;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr uint32_t kLceSmem = 1024 /* misc */ + 1024 /* alignment */ + kLceStages * kLceStage;

struct LceParams {
  int N, V, D;
  int vt_per_split;  // vocabulary tiles per split
  const int32_t* targets;
  float* part_m;  // (splits, N): running maximum of the split
  float* part_s;  // (splits, N): sum of exp(z - max) over the split
  float* part_t;  // (splits, N): the target logit, written by the split holding it
  uint32_t* status;
  // backward: vocabulary tiles from vt_base on (one chunk), and dz for them
  int vt_base, vt_end;        // the chunk's vocabulary tiles: vt_base <= vt < vt_end
  const float* lse;           // (N) from the forward
  const float* g;             // (N) upstream gradient dL/dnll
  __nv_bfloat16* dz;          // (N, ld_dz): column v - vt_base * 128
  int ld_dz;
  __nv_bfloat16* dzt;         // (Vc, ld_dzt): row v - vt_base * 128, or null (no dW)
  int ld_dzt;
};

// Token tiles per group of the backward's pair order. The CTAs resident at
// once (one per SM) cover about kLceGroup token tiles of H and
// 152 / kLceGroup vocabulary tiles of W, and a group's H stays in L2 while
// the group walks every vocabulary tile of the chunk. Measured on the
// N = 8192, V = 151,936, D = 4096 backward: 22.15 ms with one token tile
// per group (vocabulary tile fastest), 21.41 / 21.18 / 21.03 / 21.22 /
// 21.74 ms with 8 / 16 / 32 / 48 / 64.
#ifndef PA_LCE_DZ_GROUP
#define PA_LCE_DZ_GROUP 32
#endif
constexpr int kLceGroup = PA_LCE_DZ_GROUP;

// BWD = false: the forward's online log-sum-exp epilogue; the CTA walks the
// vocabulary tiles of split blockIdx.y for token tile blockIdx.x. BWD =
// true: the backward's dz epilogue, which keeps nothing from tile to tile,
// so one CTA per SM takes the chunk's (token tile, vocabulary tile) pairs
// blockIdx.x, blockIdx.x + gridDim.x, ...: pairs run in groups of kLceGroup
// token tiles, token tile fastest inside a group.
template <bool BWD>
__global__ void __launch_bounds__(kLceThreads, 1)
    lce_kernel(const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmW,
               const LceParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  LceMisc& m = *reinterpret_cast<LceMisc*>(smem_raw);
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1024 + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sRing = smem_u32(ring);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int VTc = BWD ? p.vt_end - p.vt_base : 0;  // the backward chunk's vocabulary tiles
  int vt0 = 0, nt;                                  // nt >= 1 by construction of the grid
  if (BWD) {
    const int pairs = ((p.N + kLceTile - 1) / kLceTile) * VTc;
    nt = (pairs - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  } else {
    const int VT = (p.V + kLceVTile - 1) / kLceVTile;
    vt0 = blockIdx.y * p.vt_per_split;
    nt = min(vt0 + p.vt_per_split, VT) - vt0;
  }
  // token tile and vocabulary tile of this CTA's tile j (the backward's pair
  // q: group gi of token tiles g0 .. g0 + gs - 1, then its index r inside)
  const int TMc = (p.N + kLceTile - 1) / kLceTile;
  const int VTg = BWD ? VTc : 1;  // the forward never takes pairs
  const auto pair_of = [&](int j) -> int2 {
    const int q = (int)blockIdx.x + j * (int)gridDim.x;
    const int gi = q / (kLceGroup * VTg), r = q - gi * kLceGroup * VTg;
    const int g0 = gi * kLceGroup, gs = min(kLceGroup, TMc - g0);
    return make_int2(g0 + r % gs, p.vt_base + r / gs);
  };
  const auto tile_tm = [&](int j) { return BWD ? pair_of(j).x : (int)blockIdx.x; };
  const auto tile_vt = [&](int j) { return BWD ? pair_of(j).y : vt0 + j; };
  const int KS = p.D / 64;   // K slices per tile
  const Guard g{&m.abort_flag, p.status};

  if (threadIdx.x == 0) {
    m.abort_flag = 0;
    for (int s = 0; s < kLceStages; ++s) {
      mbar_init(&m.full[s], 1);
      mbar_init(&m.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&m.acc_full[b], 1);
      mbar_init(&m.acc_empty[b], 128);
    }
    mbar_init(&m.fin, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&m.tmem_base, kLceTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tmap(&tmH);
      prefetch_tmap(&tmW);
      int it = 0;
      bool ok = true;
      for (int j = 0; ok && j < nt; ++j) {
        for (int kc = 0; kc < KS; ++kc, ++it) {
          const int st = it % kLceStages;
          if (!g.wait(&m.empty[st], ((it / kLceStages) & 1) ^ 1, 40)) { ok = false; break; }
          mbar_expect_tx(&m.full[st], kLceStage);
          tma_load_2d(ring + st * kLceStage, &tmH, &m.full[st], kc * 64, tile_tm(j) * kLceTile);
          tma_load_2d(ring + st * kLceStage + kLceSlice, &tmW, &m.full[st], kc * 64, tile_vt(j) * kLceVTile);
        }
      }
      // no copy may still be landing when the CTA exits
      for (int i = (it > kLceStages ? it - kLceStages : 0); i < it; ++i)
        g.drain(&m.full[i % kLceStages], (i / kLceStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = lane == 0;
    constexpr uint32_t idZ = idesc_bf16_f32(128, 256, false, false);
    bool ok = true;
    int it = 0;
    for (int j = 0; ok && j < nt; ++j) {
      const int buf = j & 1;
      // accumulator buf is free once the epilogue has read tile j - 2 from it
      if (j >= 2 && !g.wait_warp(&m.acc_empty[buf], ((j - 2) >> 1) & 1, 41)) { ok = false; break; }
      tc_fence_after();
      for (int kc = 0; kc < KS; ++kc, ++it) {
        const int st = it % kLceStages;
        if (!g.wait_warp(&m.full[st], (it / kLceStages) & 1, 42)) { ok = false; break; }
        tc_fence_after();
        const uint64_t hd = sdesc_sw128(sRing + st * kLceStage, 16, 1024);
        const uint64_t wd = sdesc_sw128(sRing + st * kLceStage + kLceSlice, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (leader)
            umma_bf16(tmem + buf * 256, sdesc_add(hd, kk * 32), sdesc_add(wd, kk * 32), idZ,
                      (kc > 0 || kk > 0) ? 1u : 0u);
        if (leader) umma_commit(&m.empty[st]);
        __syncwarp();
      }
      if (ok && leader) umma_commit(&m.acc_full[buf]);
      __syncwarp();
    }
    if (leader) {
      umma_commit(&m.fin);  // every MMA issued has completed once this arrives
      g.drain(&m.fin, 0);
    }
    __syncwarp();
  } else if (warp >= 4 && BWD) {
    // ------------------------------------------------------------ dz epilogue
    // Thread r owns token row r of the tile: dz = g (2^(z log2e - lse log2e)
    // - [v == target]) for every vocabulary column, zero for an ignored
    // target (outside [0, V)). dz goes out in the token's row (16-byte
    // stores) and, when the head trains, in dz^T, where the 32 lanes of a
    // warp write 32 consecutive tokens of one vocabulary row.
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      const int buf = j & 1;
      const int token = tile_tm(j) * kLceTile + r;
      const bool live = token < p.N;
      const int t = live ? p.targets[token] : -1;
      const bool use = live && t >= 0 && t < p.V;
      const float gl = use ? p.g[token] : 0.f;
      const float l2 = use ? p.lse[token] * 1.4426950408889634f : 0.f;
      ok = g.wait(&m.acc_full[buf], (j >> 1) & 1, 44);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      tc_fence_after();
      const int v0 = tile_vt(j) * kLceVTile;
      const int c0v = v0 - p.vt_base * kLceVTile;  // column of v0 in the chunk
#pragma unroll 1
      for (int c0 = 0; c0 < kLceVTile; c0 += 32) {
        uint32_t a[32];
        tmem_ld32(tmem + lane_base + buf * 256 + c0, a);
        const int vc = v0 + c0;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          // columns past V (the last tile's tail) are exactly zero
          const float d0 = (use && vc + i < p.V)
                               ? gl * (ex2(fmaf(__uint_as_float(a[i]), 1.4426950408889634f, -l2)) -
                                       (vc + i == t ? 1.f : 0.f))
                               : 0.f;
          const float d1 = (use && vc + i + 1 < p.V)
                               ? gl * (ex2(fmaf(__uint_as_float(a[i + 1]), 1.4426950408889634f, -l2)) -
                                       (vc + i + 1 == t ? 1.f : 0.f))
                               : 0.f;
          w[i >> 1] = pack_bf16x2(d0, d1);
        }
        if (live) {
          // the tile's columns past V are not part of the chunk's output
          __nv_bfloat16* row = p.dz + (size_t)token * p.ld_dz + c0v + c0;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (vc + 8 * u < p.V)
              *reinterpret_cast<uint4*>(row + 8 * u) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
          if (p.dzt) {
            __nv_bfloat16* col = p.dzt + (size_t)(c0v + c0) * p.ld_dzt + token;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (vc + i < p.V)
                col[(size_t)i * p.ld_dzt] = __ushort_as_bfloat16((unsigned short)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu));
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&m.acc_empty[buf]);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int token = (int)blockIdx.x * kLceTile + r;
    const int t = token < p.N ? p.targets[token] : -1;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    float m_run = -INFINITY, s_run = 0.f, tgt = 0.f;
    bool have_t = false;
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      const int buf = j & 1;
      ok = g.wait(&m.acc_full[buf], (j >> 1) & 1, 43);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      tc_fence_after();
      const int v0 = tile_vt(j) * kLceVTile;
#pragma unroll 1
      for (int c0 = 0; c0 < kLceVTile; c0 += 32) {
        uint32_t a[32];
        tmem_ld32(tmem + lane_base + buf * 256 + c0, a);
        const int vc = v0 + c0;
        float cmax = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (vc + i < p.V) cmax = fmaxf(cmax, __uint_as_float(a[i]));
        if (cmax > -INFINITY) {
          const float m_new = fmaxf(m_run, cmax);
          float acc = 0.f;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (vc + i < p.V) acc += expf(__uint_as_float(a[i]) - m_new);
          s_run = s_run * expf(m_run - m_new) + acc;
          m_run = m_new;
        }
        if (t >= vc && t < vc + 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (t == vc + i) tgt = __uint_as_float(a[i]);
          have_t = true;
        }
      }
      tc_fence_before();
      mbar_arrive(&m.acc_empty[buf]);
    }
    if (ok && token < p.N) {
      const size_t o = (size_t)blockIdx.y * p.N + token;
      p.part_m[o] = m_run;
      p.part_s[o] = s_run;
      if (have_t) p.part_t[o] = tgt;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kLceTmemCols);
  }
}

// One thread per token: combine the splits' (max, sum) pairs and look up the
// target logit in the split that holds the target.
__global__ void __launch_bounds__(256) lce_merge_kernel(const LceParams p, int splits, float* __restrict__ nll,
                                                        float* __restrict__ lse, float* __restrict__ tgt_out) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= p.N) return;
  float M = -INFINITY;
  for (int y = 0; y < splits; ++y) M = fmaxf(M, p.part_m[(size_t)y * p.N + i]);
  float S = 0.f;
  for (int y = 0; y < splits; ++y) {
    const float my = p.part_m[(size_t)y * p.N + i];
    if (my > -INFINITY) S += p.part_s[(size_t)y * p.N + i] * expf(my - M);
  }
  const float l = M + logf(S);
  const int t = p.targets[i];
  float z = 0.f, n = 0.f;
  if (t >= 0 && t < p.V) {
    z = p.part_t[(size_t)(t / kLceVTile / p.vt_per_split) * p.N + i];
    n = l - z;
  }
  lse[i] = l;
  tgt_out[i] = z;
  nll[i] = n;
}

// ------------------------------------------------------------------ GEMM
// C (M x N) from A (M x K, K contiguous) and B (K x N, N contiguous) in
// 128 x 256 output tiles (N = 256 products, which keep their full rate beside
// the epilogue warps' arithmetic). One CTA per SM walks tiles blockIdx.x,
// blockIdx.x + gridDim.x, ... in groups of kGemmGroup row blocks (M tiles
// fastest inside a group, so a group's A panels stay in L2 while it walks
// every N tile), K in steps of 64 through a
// TMA ring (A as one 128-row x 64 box, B as four 64-row x 64 boxes, or two in
// each CTA of a pair, all 128-byte swizzled; elements past M, N or K read as
// zero; a warp each issues the copies of A and B), tcgen05
// products into two 256-column fp32 TMEM accumulators used by alternate
// tiles, so a tile's epilogue runs beside the next tile's products. The
// epilogue (one thread per output row) stores bf16, or starts / adds to /
// finishes an fp32 accumulator in global memory; each output tile belongs to
// one CTA, so no two threads touch the same element. What is only written
// (bf16, or an accumulator's start) goes through 32 KB of shared memory and
// TMA stores: rows written piecewise by their threads cost 32 separate sectors
// an instruction, which bounds a product of few K (the head's gradient of 96
// tokens, 131 MB of it, took 49 us that way and 31 us through TMA).
constexpr int kGemmN = 256;                               // output columns per tile
constexpr uint32_t kGemmA = 128 * 128;                    // 128 rows x 64 K, 16 KB
constexpr uint32_t kGemmBHalf = 64 * 128;                 // 64 K rows x 64 N columns, 8 KB
constexpr int kGemmThreads = 224;  // A's copies, products, four epilogue warps, B's copies
// PAIR: two CTAs of a cluster form one product of 256 x 256, each loading its
// own 128 rows of A and half of B's columns: 32 KB a K block instead of 48.
// TWO: A is the sum of two bf16 matrices, which take the same block of B. STAY:
// K is at most 128, a CTA takes its tiles column by column, and all of a column's
// B stays behind the ring, which only A goes through (the head's gradient of 96
// tokens in two terms: 102 us for both gradients with B in the ring, three
// stages deep, 97 us so).
template <bool PAIR, bool TWO, bool STAY>
struct GemmRing {
  static_assert(PAIR ? !TWO && !STAY : TWO || !STAY, "the others are not built");
  static constexpr int STAGES = PAIR ? 6 : STAY ? 4 : TWO ? 3 : 4;
  static constexpr int BBOXES = PAIR ? 2 : 4;  // boxes of 64 columns of B in this CTA
  static constexpr uint32_t BBLOCK = BBOXES * kGemmBHalf;
  static constexpr uint32_t B = kGemmA, LO = kGemmA + (STAY ? 0 : BBLOCK);  // in a stage; LO: A's second term
  static constexpr uint32_t STAGE = LO + (TWO ? kGemmA : 0);
  static constexpr uint32_t BYTES = STAGES * STAGE + (STAY ? 2 * BBLOCK : 0);
};
constexpr uint32_t kGemmOut = 2 * 128 * 128;  // two boxes of 128 rows x 128 bytes on their way out
constexpr uint32_t kGemmSmem = 1024 /* misc */ + 1024 /* alignment */ + GemmRing<false, false, false>::BYTES + kGemmOut;
static_assert(GemmRing<true, false, false>::BYTES == GemmRing<false, false, false>::BYTES &&
                  GemmRing<false, true, false>::BYTES == GemmRing<false, false, false>::BYTES &&
                  GemmRing<false, true, true>::BYTES == GemmRing<false, false, false>::BYTES && kGemmSmem <= 232448,
              "shared memory");

// Row blocks per group of the tile order. Measured on the N = 8192,
// V = 151,936, D = 4096 backward (38 launches a call), in one run: 20.95,
// 21.01, 20.62 and 20.99 ms with 1 (N tiles fastest), 8, 16 and 32, and
// 21.17 ms with 16 on another box, as with 1 there: the order makes no
// difference beyond the spread between runs. With N tiles fastest a launch
// of 8192 x 4096 x 8192 read 0.60 GB from DRAM against 0.19 GB of operands
// and kept the tensor pipe 78% busy.
#ifndef PA_LCE_GEMM_GROUP
#define PA_LCE_GEMM_GROUP 16
#endif
constexpr int kGemmGroup = PA_LCE_GEMM_GROUP;

struct GemmParams {
  int M, N, K;         // N a multiple of 64
  int mode;            // GemmMode
  int m_tiles;         // row blocks of 128, or of 256 in a pair
  int n_tiles;         // N tiles of kGemmN per row block
  int per_split;       // M tiles x N tiles
  int tiles;           // per_split x the runs that K is cut into
  int kb_per;          // K blocks of 64 per run
  __nv_bfloat16* c;    // bf16 result (kStoreBf16: the product; kAccFinal: accumulator + product)
  int ldc;
  float* acc;          // fp32 accumulator (kAccInit: set; kAccAdd: add; kAccFinal: read)
  int ldacc;
  uint32_t* status;
  int order;           // GemmOrder
};

struct GemmMisc {
  uint64_t full[6], empty[6];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t b_full, b_empty;  // STAY
  uint64_t fin;
  uint32_t tmem_base;
  int abort_flag;
};

// One thread's row of a box of 128 rows x 128 bytes, 128-byte swizzled: 64
// columns as bf16, or 32 as fp32.
__device__ __forceinline__ void store_box(uint32_t taddr, uint32_t out, int r, bool f32) {
  const uint32_t row = out + r * 128;
  const int x = r & 7;
  if (f32) {
    uint32_t a[32];
    tmem_ld32(taddr, a);
#pragma unroll
    for (int q = 0; q < 8; ++q) st_shared_v4(row + ((q ^ x) << 4), a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
    return;
  }
  uint32_t a[2][32];
  tmem_ld32x2(taddr, taddr + 32, a[0], a[1]);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t* e = &a[q >> 2][8 * (q & 3)];
    st_shared_v4(row + ((q ^ x) << 4), pack_bf16x2(__uint_as_float(e[0]), __uint_as_float(e[1])),
                 pack_bf16x2(__uint_as_float(e[2]), __uint_as_float(e[3])),
                 pack_bf16x2(__uint_as_float(e[4]), __uint_as_float(e[5])),
                 pack_bf16x2(__uint_as_float(e[6]), __uint_as_float(e[7])));
  }
}

template <bool PAIR, bool TWO, bool STAY>
__global__ void __launch_bounds__(kGemmThreads, 1)
    lce_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmLo,
                    const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmC,
                    const GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  GemmMisc& m = *reinterpret_cast<GemmMisc*>(smem_raw);
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1024 + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sRing = smem_u32(ring);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  using R = GemmRing<PAIR, TWO, STAY>;
  constexpr int kPer = PAIR ? 2 : 1, kRows = 128 * kPer, kGroup = kGemmGroup / kPer;
  const int cta = (int)blockIdx.x / kPer, ctas = (int)gridDim.x / kPer, rank = PAIR ? (int)blockIdx.x % 2 : 0;
  const int KB = (p.K + 63) / 64;
  // K blocks kb0 .. kb1 - 1 of tile t: its run of the contraction
  const auto tile_run = [&](int t) -> int2 {
    const int k0 = t / p.per_split * p.kb_per;
    return make_int2(k0, min(k0 + p.kb_per, KB));
  };
  // this CTA's (or pair's) tiles: t = cta + j * ctas for j < nt (>= 1: the
  // grid is never larger than the tile count)
  // STAY: t0 .. t0 + nt - 1, row blocks fastest
  const int t0 = STAY ? (int)((long long)p.tiles * cta / ctas) : cta, dt = STAY ? 1 : ctas;
  const int nt = STAY ? (int)((long long)p.tiles * (cta + 1) / ctas) - t0 : (p.tiles - cta + ctas - 1) / ctas;
  // first row (of this CTA) and column of tile t: group gi holds row blocks g0 .. g0 + gs - 1
  const auto tile_origin = [&](int t) -> int2 {
    t %= p.per_split;
    if (STAY) return make_int2(t % p.m_tiles * kRows, t / p.m_tiles * kGemmN);
    const int gi = t / (kGroup * p.n_tiles), r = t - gi * kGroup * p.n_tiles;
    const int g0 = gi * kGroup, gs = min(kGroup, p.m_tiles - g0);
    return make_int2((g0 + r % gs) * kRows + rank * 128, (r / gs) * kGemmN);
  };
  const Guard g{&m.abort_flag, p.status};

  if (threadIdx.x == 0) {
    m.abort_flag = 0;
    for (int s = 0; s < R::STAGES; ++s) {
      mbar_init(&m.full[s], 1);
      mbar_init(&m.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&m.acc_full[b], 1);
      mbar_init(&m.acc_empty[b], 128 * kPer);
    }
    mbar_init(&m.b_full, 1);
    mbar_init(&m.b_empty, 1);
    mbar_init(&m.fin, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(&m.tmem_base, 2 * kGemmN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&m.tmem_base, 2 * kGemmN);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // both CTAs' barriers are ready
  tc_fence_after();
  // What is launched programmatically behind this kernel may take the SMs that
  // it leaves, but no earlier than the kernel ahead has ended: a kBeside kernel
  // counts on what that one has written.
  if (p.order == kAfter) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = m.tmem_base;

  if (STAY && warp == 6) {
    // B of each column of tiles, once the products of the column before have read theirs
    if (lane == 0) {
      prefetch_tmap(&tmB);
      int columns = 0;
      for (int j = 0; j < nt; ++j) {
        const int n0 = tile_origin(t0 + j).y;
        if (j > 0 && n0 == tile_origin(t0 + j - 1).y) continue;
        if (!g.wait(&m.b_empty, (columns & 1) ^ 1, 49)) break;
        mbar_expect_tx(&m.b_full, KB * R::BBLOCK);
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int c = 0; c < R::BBOXES; ++c)
            tma_load_2d(ring + R::STAGES * R::STAGE + kb * R::BBLOCK + c * kGemmBHalf, &tmB, &m.b_full, n0 + 64 * c, kb * 64);
        ++columns;
      }
      if (columns > 0) g.drain(&m.b_full, (columns - 1) & 1);  // no copy may still be landing when the CTA exits
    }
    __syncwarp();
  } else if (warp == 0 || warp == 6) {
    // A's copies by warp 0, which also announces the bytes of both, B's by warp 6
    if (lane == 0) {
      const bool isA = warp == 0;
      prefetch_tmap(isA ? &tmA : &tmB);
      const uint32_t full0 = PAIR ? cluster_addr(&m.full[0], 0) : smem_u32(&m.full[0]);
      int it = 0, st = 0;
      uint32_t phase = 1;
      bool ok = true;
      for (int j = 0; ok && j < nt; ++j) {
        const int2 o = tile_origin(t0 + j * dt);
        const int m0 = o.x, n0 = o.y + 64 * rank * R::BBOXES;
        const int2 run = tile_run(t0 + j * dt);
        for (int kb = run.x; kb < run.y; ++kb, ++it) {
          if (!g.wait(&m.empty[st], phase, isA ? 45 : 49)) { ok = false; break; }
          uint8_t* sa = ring + st * R::STAGE;
          if (isA) {
            if (rank == 0) mbar_expect_tx(&m.full[st], kPer * R::STAGE);  // rank 0's barrier counts the bytes of both CTAs
            if (PAIR)
              tma_load_2d_pair(sa, &tmA, full0 + st * 8, kb * 64, m0);
            else
              tma_load_2d(sa, &tmA, &m.full[st], kb * 64, m0);
            if (TWO) tma_load_2d(sa + R::LO, &tmLo, &m.full[st], kb * 64, m0);
          } else {
#pragma unroll
            for (int c = 0; c < R::BBOXES; ++c)
              if (PAIR)
                tma_load_2d_pair(sa + R::B + c * kGemmBHalf, &tmB, full0 + st * 8, n0 + 64 * c, kb * 64);
              else
                tma_load_2d(sa + R::B + c * kGemmBHalf, &tmB, &m.full[st], n0 + 64 * c, kb * 64);
          }
          if (++st == R::STAGES) {
            st = 0;
            phase ^= 1;
          }
        }
      }
      // no copy may still be landing when the CTA exits (in a pair, no arrival of
      // the other CTA's either: each stage's last release says both)
      for (int i = (it > R::STAGES ? it - R::STAGES : 0); i < it; ++i)
        g.drain(PAIR ? &m.empty[i % R::STAGES] : &m.full[i % R::STAGES], (i / R::STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    const bool leader = lane == 0;
    constexpr uint32_t idC = idesc_bf16_f32(kRows, kGemmN, false, true);
    bool ok = true;
    int it = 0, columns = 0;
    for (int j = 0; ok && rank == 0 && j < nt; ++j) {  // rank 0 issues for both
      const int buf = j & 1;
      // accumulator buf is free once the epilogue has read tile j - 2 from it
      if (j >= 2 && !g.wait_warp(&m.acc_empty[buf], ((j - 2) >> 1) & 1, 48)) { ok = false; break; }
      if (PAIR) fence_cluster();  // half of the arrivals are the other CTA's
      tc_fence_after();
      const int2 run = tile_run(t0 + j * dt);
      if (STAY && (j == 0 || tile_origin(t0 + j).y != tile_origin(t0 + j - 1).y)) {
        if (!g.wait_warp(&m.b_full, columns & 1, 46)) { ok = false; break; }
        ++columns;
      }
      for (int kb = run.x; kb < run.y; ++kb, ++it) {
        const int st = it % R::STAGES;
        if (!g.wait_warp(&m.full[st], (it / R::STAGES) & 1, 46)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sa = sRing + st * R::STAGE;
        const uint64_t ad = sdesc_sw128(sa, 16, 1024);
        const uint64_t bd = sdesc_sw128(STAY ? sRing + R::STAGES * R::STAGE + kb * R::BBLOCK : sa + R::B, kGemmBHalf, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (leader) {
            const uint32_t add = (kb > run.x || kk > 0) ? 1u : 0u;
            if (PAIR)
              umma_bf16_pair(tmem + buf * kGemmN, sdesc_add(ad, kk * 32), sdesc_add(bd, kk * 2048), idC, add);
            else
              umma_bf16(tmem + buf * kGemmN, sdesc_add(ad, kk * 32), sdesc_add(bd, kk * 2048), idC, add);
          }
        if (TWO) {
          const uint64_t ld = sdesc_sw128(sa + R::LO, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (leader) umma_bf16(tmem + buf * kGemmN, sdesc_add(ld, kk * 32), sdesc_add(bd, kk * 2048), idC, 1u);
        }
        if (leader) PAIR ? umma_commit_pair(&m.empty[st]) : umma_commit(&m.empty[st]);
        __syncwarp();
      }
      if (ok && leader) PAIR ? umma_commit_pair(&m.acc_full[buf]) : umma_commit(&m.acc_full[buf]);
      if (STAY && ok && leader && j + 1 < nt && tile_origin(t0 + j).y != tile_origin(t0 + j + 1).y) umma_commit(&m.b_empty);
      __syncwarp();
    }
    if (leader && rank == 0) {
      PAIR ? umma_commit_pair_own(&m.fin) : umma_commit(&m.fin);  // every MMA issued has completed once this arrives
      g.drain(&m.fin, 0);
    }
    __syncwarp();
  } else {
    // warps 2..5: TMEM lane quarter warp % 4, one thread per output row
    const int quarter = warp & 3;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const bool f32 = p.mode == kAccInit, through = f32 || p.mode == kStoreBf16;
    uint8_t* out = ring + R::BYTES;
    const bool issuer = threadIdx.x == 64;
    int box = 0;
    const auto release = [&](int buf) {
      if (PAIR)
        mbar_arrive_cluster(cluster_addr(&m.acc_empty[buf], 0));
      else
        mbar_arrive(&m.acc_empty[buf]);
    };
    if (through && issuer) prefetch_tmap(&tmC);
    for (int j = 0; j < nt; ++j) {
      const int buf = j & 1;
      const bool ok = __all_sync(~0u, g.wait(&m.acc_full[buf], (j >> 1) & 1, 47));
      if (!ok) break;
      tc_fence_after();
      const int2 o = tile_origin(t0 + j * dt);
      const int m0 = o.x, n0 = o.y;
      const int row = m0 + quarter * 32 + lane;
      if (through) {
        // a box of 128 rows x 128 bytes at a time, through two buffers in turn (the
        // second CTA of a pair may lie past the last row)
        const int run = (t0 + j * dt) / p.per_split, step = f32 ? 32 : 64;
#pragma unroll 1
        for (int c0 = 0; m0 < p.M && c0 < kGemmN && n0 + c0 < p.N; c0 += step, box ^= 1) {
          if (issuer) bulk_wait_read1();  // the buffer's last copy has left it
          named_bar_sync(1, 128);
          store_box(tmem + lane_base + buf * kGemmN + c0, smem_u32(out) + box * 16384, quarter * 32 + lane, f32);
          fence_async_smem();
          named_bar_sync(1, 128);
          if (issuer) {
            tma_store_3d(&tmC, out + box * 16384, n0 + c0, m0, run);
            bulk_commit();
          }
        }
        tc_fence_before();
        release(buf);
        continue;
      }
      // each run of K has an accumulator of its own
      float* acc = p.acc + (size_t)((t0 + j * dt) / p.per_split) * p.M * p.ldacc;
#pragma unroll 1
      for (int c0 = 0; c0 < kGemmN; c0 += 32) {
        uint32_t a[32];
        tmem_ld32(tmem + lane_base + buf * kGemmN + c0, a);
        const int col = n0 + c0;
        if (row >= p.M || col >= p.N) continue;  // N is a multiple of 64: 32 columns are all in or all out
        {
          float4* ac = reinterpret_cast<float4*>(acc + (size_t)row * p.ldacc + col);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float4 v = make_float4(__uint_as_float(a[4 * q]), __uint_as_float(a[4 * q + 1]),
                                   __uint_as_float(a[4 * q + 2]), __uint_as_float(a[4 * q + 3]));
            const float4 o = ac[q];
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
            if (p.mode == kAccFinal) {
              a[4 * q] = __float_as_uint(v.x);
              a[4 * q + 1] = __float_as_uint(v.y);
              a[4 * q + 2] = __float_as_uint(v.z);
              a[4 * q + 3] = __float_as_uint(v.w);
            } else {
              ac[q] = v;
            }
          }
        }
        if (p.mode == kAccFinal) {
          uint4* cr = reinterpret_cast<uint4*>(p.c + (size_t)row * p.ldc + col);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            cr[q] = make_uint4(pack_bf16x2(__uint_as_float(a[8 * q]), __uint_as_float(a[8 * q + 1])),
                               pack_bf16x2(__uint_as_float(a[8 * q + 2]), __uint_as_float(a[8 * q + 3])),
                               pack_bf16x2(__uint_as_float(a[8 * q + 4]), __uint_as_float(a[8 * q + 5])),
                               pack_bf16x2(__uint_as_float(a[8 * q + 6]), __uint_as_float(a[8 * q + 7])));
        }
      }
      tc_fence_before();
      release(buf);
    }
    if (through && issuer) bulk_wait_all();  // the last stores have completed before the CTA exits
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // neither CTA leaves while the other's products read its shared memory
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, 2 * kGemmN);
    else
      tmem_dealloc(tmem, 2 * kGemmN);
  }
  // beside the kernel ahead of it, this one ends no earlier
  if (p.order == kBeside && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Sum of the runs' accumulators, in run order, rounded to bf16: 4 elements a thread.
__global__ void __launch_bounds__(256) sum_splits_kernel(const float4* __restrict__ acc, int splits, size_t n4,
                                                         uint2* __restrict__ out) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n4; i += (size_t)gridDim.x * blockDim.x) {
    float4 v = acc[i];
    for (int s = 1; s < splits; ++s) {
      const float4 o = acc[s * n4 + i];
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    out[i] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

}  // namespace

// Fewest K blocks of a run for which pairs are taken: below, a tile is mostly
// its epilogue, and the cluster's barriers cost more than the loads that a pair
// saves. Both gradients over V 32,003, D 2048 in us, pairs always / never / from
// 8 blocks on: 256 tokens 128 / 120 / 117, 512 tokens 185 / 192 / 185, 2,048
// tokens 471 / 491 / 471. (A in two terms, up to 128 tokens, takes no pairs.)
constexpr int kGemmPairBlocks = 8;

// Cycles of an M x N x K product cut into s runs of K, on `slots` SMs: waves x
// (K blocks + 8 blocks' worth for the pipeline's fill and the tile's epilogue);
// a block takes a pair 622 cycles (512 of products, with copies and operands in
// one shared memory) and a CTA alone its copies' 664 (48 KB at 74 bytes a cycle),
// or 1,130 with A in two terms; and, with more than one run, writing and
// reading the accumulators at 6.5 TB/s. < 0 where a run would be empty.
static double gemm_cost(int M, int N, int K, int slots, int s, bool pair, int terms) {
  const int KB = (K + 63) / 64, per = (KB + s - 1) / s;
  if ((KB + per - 1) / per != s || (pair && (terms > 1 || M <= 128 || slots < 2 || per < kGemmPairBlocks))) return -1.0;
  const long long rows = pair ? 256 : 128, at_once = pair ? slots / 2 : slots;
  const long long tiles = ((M + rows - 1) / rows) * ((N + kGemmN - 1) / kGemmN);
  const long long waves = (tiles * s + at_once - 1) / at_once;
  return (double)waves * (per * (pair ? 622.0 : terms > 1 ? 1130.0 : 664.0) + 8 * 512.0) + (s > 1 ? (double)s * M * N * 8 / 6.5e6 * 1900 : 0.0);
}

int gemm_least_runs(int K) {
  const int KB = (K + 63) / 64;
  int runs = (KB + 1023) / 1024;
  for (;;) {  // runs of equal length may be fewer than asked for
    const int per = (KB + runs - 1) / runs, used = (KB + per - 1) / per;
    if (used == runs) return runs;
    runs = used;
  }
}

int gemm_splits(int M, int N, int K, int slots, int terms) {
  const int least = gemm_least_runs(K);
  int best = least;
  double best_cost = -1;
  for (int s = least; s <= 64 && s <= (K + 63) / 64; ++s)
    for (const bool pair : {false, true}) {
      const double cost = gemm_cost(M, N, K, slots, s, pair, terms);
      if (cost >= 0 && (best_cost < 0 || cost < best_cost)) {
        best_cost = cost;
        best = s;
      }
    }
  return best;
}

cudaError_t launch_gemm(const CUtensorMap& tA, const CUtensorMap& tB, const GemmCall& gc, cudaStream_t st) {
  const int KB = (gc.K + 63) / 64, planes = gc.splits > 1 ? gc.splits : 1, kb_per = (KB + planes - 1) / planes;
  // A short K (a vocabulary's last chunk) may fill fewer runs: the others' tiles
  // are left out, which leaves their accumulators as they are.
  const int splits = (KB + kb_per - 1) / kb_per;
  if (splits != planes && gc.mode != kAccAdd) return cudaErrorInvalidValue;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (gc.sms > 0 && gc.sms < sms) sms = gc.sms;
  const int terms = gc.lo ? 2 : 1;
  const double one = gemm_cost(gc.M, gc.N, gc.K, sms, splits, false, terms);
  const double two = gemm_cost(gc.M, gc.N, gc.K, sms, splits, true, terms);
  const bool pair = two >= 0 && two < one;
  if (gc.stay && (!gc.lo || KB > 2 || planes > 1)) return cudaErrorInvalidValue;
  const auto kfn = pair      ? lce_gemm_kernel<true, false, false>
                   : gc.stay ? lce_gemm_kernel<false, true, true>
                   : gc.lo   ? lce_gemm_kernel<false, true, false>
                             : lce_gemm_kernel<false, false, false>;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
  if (e != cudaSuccess) return e;
  const long long rows = pair ? 256 : 128, mt = (gc.M + rows - 1) / rows, ntl = (gc.N + kGemmN - 1) / kGemmN;
  if (mt * ntl * splits > (1ll << 30)) return cudaErrorInvalidValue;
  GemmParams q{};
  q.M = gc.M;
  q.N = gc.N;
  q.K = gc.K;
  q.mode = gc.mode;
  q.m_tiles = (int)mt;
  q.n_tiles = (int)ntl;
  q.per_split = (int)(mt * ntl);
  q.tiles = q.per_split * splits;
  q.kb_per = kb_per;
  q.c = gc.c;
  q.ldc = gc.N;
  q.acc = gc.acc;
  q.ldacc = gc.N;
  q.status = gc.status;
  q.order = gc.order;
  CUtensorMap tC;
  if (gc.mode == kAccInit) {
    if (!tmap_3d_sw128(&tC, gc.acc, true, gc.N, gc.M, splits)) return cudaErrorInvalidValue;
  } else if (!tmap_3d_sw128(&tC, gc.mode == kAccAdd ? static_cast<void*>(gc.acc) : gc.c, gc.mode == kAccAdd, gc.N, gc.M, 1)) {
    return cudaErrorInvalidValue;  // (only read by the modes that store through it)
  }
  const int at_once = pair ? sms / 2 : sms, grid = q.tiles < at_once ? q.tiles : at_once;
  if (grid < 1) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid * (pair ? 2 : 1));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kGemmSmem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2] = {cluster_pair(), programmatic_launch()};
  cfg.attrs = pair ? attrs : attrs + 1;
  cfg.numAttrs = (pair ? 1 : 0) + (gc.order == kInOrder ? 0 : 1);
  return cudaLaunchKernelEx(&cfg, kfn, tA, gc.lo ? *gc.lo : tA, tB, tC, q);
}

cudaError_t launch_sum_splits(const float* acc, int splits, size_t n, __nv_bfloat16* out, cudaStream_t st) {
  const size_t n4 = n / 4, blocks = (n4 + 255) / 256;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks < 4096 ? blocks : 4096));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr = programmatic_launch();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sum_splits_kernel, reinterpret_cast<const float4*>(acc), splits, n4,
                            reinterpret_cast<uint2*>(out));
}

// The vocabulary split of the (token tile x split) grid: the one that makes
// waves x (tiles per CTA + 1) smallest for `slots` resident CTAs, i.e. the
// shortest run once the last wave's idle SMs and each CTA's pipeline fill (about
// one tile) are counted. At most kLceMaxSplits splits (the workspace's partial
// sums are sized for that).
LceSplit lce_split(int N, int V, int slots) {
  const int TT = (N + kLceTile - 1) / kLceTile, VT = (V + kLceVTile - 1) / kLceVTile;
  if (slots < 1) slots = 1;
  LceSplit best{1, VT};
  long long best_cost = -1;
  for (int s = 1; s <= VT && s <= kLceMaxSplits; ++s) {
    const int per = (VT + s - 1) / s, used = (VT + per - 1) / per;
    const long long ctas = (long long)TT * used, waves = (ctas + slots - 1) / slots;
    const long long cost = waves * (per + 1);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = LceSplit{used, per};
    }
  }
  return best;
}

int lce_slots() {
  // one resident CTA per SM: 4 x 48 KB stages and all 512 TMEM columns
  static_assert(kLceSmem <= 232448, "shared memory");
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms <= 0)
    sms = 148;
  return sms;
}

cudaError_t launch_lce_fwd(int N, int V, int D, const void* hidden, const void* head, const int32_t* targets,
                           float* nll, float* lse, float* target_logit, float* part, uint32_t* status,
                           cudaStream_t st) {
  const LceSplit sp = lce_split(N, V, lce_slots());
  CUtensorMap tH, tW;
  if (!tmap_bf16_2d_sw128(&tH, hidden, D, N, kLceTile) || !tmap_bf16_2d_sw128(&tW, head, D, V, kLceVTile))
    return cudaErrorInvalidValue;
  LceParams p{};
  p.N = N;
  p.V = V;
  p.D = D;
  p.vt_per_split = sp.per;
  p.targets = targets;
  p.part_m = part;
  p.part_s = part + (size_t)sp.splits * N;
  p.part_t = part + (size_t)2 * sp.splits * N;
  p.status = status;
  cudaError_t e = cudaFuncSetAttribute(lce_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLceSmem);
  if (e != cudaSuccess) return e;
  dim3 grid((N + kLceTile - 1) / kLceTile, sp.splits);
  lce_kernel<false><<<grid, kLceThreads, kLceSmem, st>>>(tH, tW, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  lce_merge_kernel<<<(N + 255) / 256, 256, 0, st>>>(p, sp.splits, nll, lse, target_logit);
  return cudaGetLastError();
}

}  // namespace pa

namespace pa {

int lce_bwd_chunk(int N, int V) {
  // dz and dz^T of one chunk together take 4 N Vc bytes: at most 512 MiB
  // (chunks are whole vocabulary tiles)
  long long vc = ((1ll << 27) / (N > 0 ? N : 1)) / kLceVTile * kLceVTile;
  const long long vmax = (long long)(V + kLceVTile - 1) / kLceVTile * kLceVTile;
  if (vc > 8192) vc = 8192;
  if (vc > vmax) vc = vmax;
  if (vc < kLceVTile) vc = kLceVTile;
  return (int)vc;
}

LceBwdLayout lce_bwd_layout(int N, int V, int D) {
  LceBwdLayout L;
  L.vc = lce_bwd_chunk(N, V);
  L.chunks = (V + L.vc - 1) / L.vc;
  L.ld_dzt = (N + 63) / 64 * 64;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  L.acc = 256;
  L.dz = L.acc + (L.chunks > 1 ? up((size_t)N * D * 4) : 0);
  L.dzt = L.dz + up((size_t)N * L.vc * 2);
  L.bytes = L.dzt + up((size_t)L.vc * L.ld_dzt * 2);
  return L;
}

cudaError_t launch_lce_bwd(int N, int V, int D, const void* hidden, const void* head, const int32_t* targets,
                           const float* lse, const float* g, void* dhidden, void* dhead, void* ws, uint32_t* status,
                           cudaStream_t st) {
  const LceBwdLayout L = lce_bwd_layout(N, V, D);
  uint8_t* w = static_cast<uint8_t*>(ws);
  __nv_bfloat16* dz = reinterpret_cast<__nv_bfloat16*>(w + L.dz);
  __nv_bfloat16* dzt = reinterpret_cast<__nv_bfloat16*>(w + L.dzt);
  float* acc = reinterpret_cast<float*>(w + L.acc);
  CUtensorMap tH, tW, tHb;
  if (!tmap_bf16_2d_sw128(&tH, hidden, D, N, kLceTile) || !tmap_bf16_2d_sw128(&tW, head, D, V, kLceVTile) ||
      !tmap_bf16_2d_sw128(&tHb, hidden, D, N, 64))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(lce_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLceSmem);
  if (e != cudaSuccess) return e;
  for (int c = 0; c < L.chunks; ++c) {
    const int cv0 = c * L.vc, kc = (V - cv0 < L.vc) ? V - cv0 : L.vc;  // the chunk's vocabulary rows
    // dz (and dz^T) of the chunk: one CTA per SM over its (token tile,
    // vocabulary tile) pairs
    LceParams p{};
    p.N = N;
    p.V = V;
    p.D = D;
    p.vt_per_split = 0;
    p.targets = targets;
    p.status = status;
    p.vt_base = cv0 / kLceVTile;
    p.vt_end = (cv0 + kc + kLceVTile - 1) / kLceVTile;
    p.lse = lse;
    p.g = g;
    p.dz = dz;
    p.ld_dz = L.vc;
    p.dzt = dhead ? dzt : nullptr;
    p.ld_dzt = L.ld_dzt;
    const int pairs = ((N + kLceTile - 1) / kLceTile) * (p.vt_end - p.vt_base);
    lce_kernel<true><<<pairs < lce_slots() ? pairs : lce_slots(), kLceThreads, kLceSmem, st>>>(tH, tW, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // dW rows of the chunk = dz^T H (tokens are the contraction)
    if (dhead) {
      CUtensorMap tA;
      if (!tmap_bf16_2d_sw128_pitch(&tA, dzt, N, kc, L.ld_dzt, 128)) return cudaErrorInvalidValue;
      GemmCall gp{};
      gp.M = kc;
      gp.N = D;
      gp.K = N;
      gp.mode = kStoreBf16;
      gp.c = static_cast<__nv_bfloat16*>(dhead) + (size_t)cv0 * D;
      gp.status = status;
      if ((e = launch_gemm(tA, tHb, gp, st)) != cudaSuccess) return e;
    }
    // dH += dz W[chunk] (the chunk's vocabulary rows are the contraction)
    CUtensorMap tA, tB;
    if (!tmap_bf16_2d_sw128_pitch(&tA, dz, kc, N, L.vc, 128) ||
        !tmap_bf16_2d_sw128(&tB, static_cast<const __nv_bfloat16*>(head) + (size_t)cv0 * D, D, kc, 64))
      return cudaErrorInvalidValue;
    GemmCall gp{};
    gp.M = N;
    gp.N = D;
    gp.K = kc;
    gp.mode = L.chunks == 1 ? kStoreBf16 : c == 0 ? kAccInit : c == L.chunks - 1 ? kAccFinal : kAccAdd;
    gp.c = static_cast<__nv_bfloat16*>(dhidden);
    gp.acc = acc;
    gp.status = status;
    if ((e = launch_gemm(tA, tB, gp, st)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pa
