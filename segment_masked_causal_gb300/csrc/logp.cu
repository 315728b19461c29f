// logp.cu -- log probabilities of given tokens with entropy and the most
// likely alternatives, and the gradient of the first two, straight from the
// hidden states and the head: z = H W^T / T without storing the (N, V) logits.
//
//   lse_i  = ln sum_v exp(z_iv)          logp_i = z_i,t(i) - lse_i
//   H_i    = lse_i - sum_v p_iv z_iv     p = exp(z - lse)
//   dz_iv  = (g_i ([v = t(i)] - p_iv) - e_i p_iv (ln p_iv + H_i)) / T
//
// for L = sum_i g_i logp_i + e_i H_i. The backward forms the logits again
// (as the fused cross-entropy beside it does, mlx-train-perf 0.5.1 README,
// "The fused cross-entropy loss"), writes dz of a vocabulary chunk in bf16
// and multiplies it out with the GEMM of lce.cu.
//
// Forward: one pass over the vocabulary. With x the unscaled logits, m their
// running maximum and t = (x - m) log2 e / T, a row keeps S = sum 2^t and
// A = sum 2^t t, so that lse = m / T + ln 2 log2 S and H = ln 2 (log2 S - A / S):
// A is a sum of terms that are all <= 0 and vanish at both ends, so nothing
// cancels in it. A maximum larger by -d (in t's units) turns (S, A) into
// (S 2^d, (A + d S) 2^d).
//   The difference is taken before the scaling, so that t is 0 at the maximum,
// nowhere above, and off by its own rounding only, however large the logits: those
// of a masked vocabulary row may be the type's lowest value, whose product with
// log2 e / T rounds by 1e30. It costs an addition for two columns: 777 tokens over
// V 50,257, D 1024 60.9 -> 61.7 us, and 73.2 -> 76.9 us where the epilogue is all
// there is (4,096 tokens, V 32,003, D 64). 2^d is 0 from d = -150 on, so d is cut
// at kFar, and d S stays finite.
//   Both sums carry what their additions lose: with one likely token S is near 1,
// and of a hundred thousand others at 1e-9, which add 1e-4 in all, 32 columns
// together are less than half a step of it (8,192 tokens over V 151,936 were 4e-5
// off, now 9e-7; no time that could be measured).
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

constexpr int kTok = 128;                  // tokens per CTA
constexpr int kUnit = kLogpUnit;           // vocabulary rows of one unit: what splits are counted in
constexpr int kTileUnits = 8;              // units per logit tile: 256 columns
constexpr uint32_t kSliceH = kTok * 128;   // 128 x 64 bf16, 16 KB
constexpr int kThreads = 256;
// Eight epilogue warps, two a token quarter: the last tile's epilogue stands
// behind its products (1,000 tokens over V 151,936, D 512: 564 us with four
// warps, 547 with eight; 4,096 over V 32,003, D 64: 331 and 327).
constexpr int kDzThreads = 384;
constexpr uint32_t kTmemCols = 512;  // two 256-column fp32 accumulators
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kFar = -30000.f;  // 2^t and 2^t t are 0 here

// The ring of K slices: one CTA per SM. PAIR: two CTAs form one product of 256
// tokens x 256 vocabulary rows, each holding its own 128 tokens and half of the
// vocabulary rows. A tile of 128 x 256 alone takes 48 KB a K slice into an SM
// for 512 cycles of products; with every SM copying, the L2 gives each about 77
// bytes a cycle (620 cycles), in a shared memory that the operands are read
// from as well. The pair takes 32 KB.
template <bool PAIR>
struct Ring {
  static constexpr int STAGES = PAIR ? 6 : 4;
  static constexpr uint32_t UNIT = (PAIR ? kUnit / 2 : kUnit) * 128;  // this CTA's rows of a unit
  static constexpr uint32_t STAGE = kSliceH + kTileUnits * UNIT;
  static constexpr uint32_t BYTES = STAGES * STAGE;
};
constexpr uint32_t kSmem = 1024 /* misc */ + 1024 /* alignment */ + Ring<false>::BYTES;
// Behind the ring, with alternatives: 32 candidates of each epilogue thread.
constexpr int kCands = 32;
constexpr uint32_t kSmemTop = kSmem + kCands * 128 * sizeof(float2);
static_assert(Ring<true>::BYTES == Ring<false>::BYTES && kSmemTop <= 232448, "shared memory");

struct Misc {
  uint64_t full[6], empty[6];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t fin;
  uint32_t tmem_base;
  int abort_flag;
};

// The boxes of a launch: `wide` units of W (or half of that many rows a CTA in
// a pair) in tmW, `rest` in tmR for the shorter last tile of a split, and
// `rows` tokens of H, `reps` times.
struct Boxes {
  int wide, rest, rows, reps;
};

struct FwdParams {
  int N, V, D, top;
  int units_per_split, splits;
  Boxes boxes;  // reps 1, 2 or 4: how often the token tile's rows are repeated (see logp_fwd_kernel)
  float sl2, inv_t;  // log2(e) / temperature, 1 / temperature
  const int32_t* targets;
  float4* part;    // (splits, N) {m, S, A, the target's raw logit}
  float2* cand;    // (N, splits, top) {raw logit, vocabulary row or -1}, largest first
  uint32_t* status;
};

struct BwdParams {
  int N, V, D;
  int v_base, v_end;   // the chunk's vocabulary rows
  int tile_units;      // units of 32 rows per logit tile
  Boxes boxes;
  int first;           // 1: this launch starts the call (clears the status word)
  float sl2, inv_t;
  const int32_t* targets;
  const float* lse;
  const float* entropy;    // read where g_entropy is given
  const float* g_logp;
  const float* g_entropy;  // may be null
  __nv_bfloat16* dz;       // (terms, N, ld_dz)
  int ld_dz;
  __nv_bfloat16* dzt;      // (terms, ld_dz, ld_dzt), or null (frozen head)
  int ld_dzt;
  uint32_t* status;
};

// One logit tile: 128 tokens from tile row tm, `units` x 32 vocabulary rows
// from unit u.
struct Tile {
  int tm, u, units;
};

// Token tiles per group of the backward's order, token tile fastest: a
// group's H stays in L2 while it walks the chunk's vocabulary tiles (the
// cross-entropy backward measured 22.2 ms without groups, 21.0 with 32).
constexpr int kGroup = 32;

// The largest of the W values from x[W s] on; NaN is passed over.
template <int W>
__device__ __forceinline__ float max_of(const uint32_t (&x)[32], int s) {
  const auto f = [&](int i) { return __uint_as_float(x[W * s + i]); };
  if (W == 2) return fmaxf(f(0), f(1));
  if (W == 4) return fmax3(f(0), f(1), fmaxf(f(2), f(3 % W)));
  return fmaxf(fmax3(f(0), f(1), f(2 % W)), fmax3(fmax3(f(3 % W), f(4 % W), f(5 % W)), f(6 % W), f(7 % W)));
}

// Which of the eight values from a[8 s] on are above `least`, as bits.
__device__ __forceinline__ uint32_t over8(const uint32_t (&a)[32], int s, float least) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m |= __uint_as_float(a[8 * s + i]) > least ? 1u << i : 0u;
  return m;
}

// Two words to shared memory where `on` is not 0, without a branch.
__device__ __forceinline__ void st_shared_if(uint32_t on, uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p st.shared.v2.b32 [%1], {%2, %3};\n\t}" ::"r"(on), "r"(addr),
               "r"(x), "r"(y)
               : "memory");
}

// Barriers and TMEM. In a pair the full and acc_empty barriers of rank 0 serve
// both CTAs; the others are each CTA's own. `readers`: epilogue threads of a CTA.
template <bool PAIR>
__device__ __forceinline__ void setup(Misc& m, int readers) {
  if (threadIdx.x == 0) {
    m.abort_flag = 0;
    for (int s = 0; s < Ring<PAIR>::STAGES; ++s) {
      mbar_init(&m.full[s], 1);
      mbar_init(&m.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&m.acc_full[b], 1);
      mbar_init(&m.acc_empty[b], PAIR ? 2 * readers : readers);
    }
    mbar_init(&m.fin, 1);
    fence_mbar_init();
  }
  if ((threadIdx.x >> 5) == 1) {
    if (PAIR) {
      tmem_alloc_pair(&m.tmem_base, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&m.tmem_base, kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // both CTAs' barriers are ready
  tc_fence_after();
}

template <bool PAIR>
__device__ __forceinline__ void teardown(uint32_t tmem) {
  tc_fence_before();
  __syncthreads();
  // neither CTA of a pair leaves while the other's products read its shared memory
  if (PAIR) cluster_sync();
  if ((threadIdx.x >> 5) == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, kTmemCols);
    else
      tmem_dealloc(tmem, kTmemCols);
  }
}

// 64-wide K slices of H and W through the ring, each as one box, W's by lane 0
// of warp 0 and H's by lane 0 of warp 2: one round of waiting, announcing and
// issuing takes a thread about 320 cycles and each further copy 60, which is
// near the 512 cycles of a slice's products. A copy itself costs its rows, past
// the tensor's end or not, so a tile's tokens are brought in only up to the
// last one (eight-row swizzle atoms; the product's other rows come from
// whatever the ring holds and are nobody's). The tokens of a tile that repeats
// them come `reps` times, 128 / reps rows apart. In a pair each CTA loads its
// own tokens and its half of the tile's vocabulary rows, the first half in rank
// 0, and rank 0's barrier counts the bytes of both.
template <bool PAIR, bool TOKENS, class TileOf>
__device__ __forceinline__ void load_tiles(Misc& m, const Guard& g, uint8_t* ring, const CUtensorMap* tmH,
                                           const CUtensorMap* tmW, const CUtensorMap* tmR, int nt, int KS,
                                           const Boxes bx, TileOf tile_of) {
  using R = Ring<PAIR>;
  if (TOKENS) {
    prefetch_tmap(tmH);
  } else {
    prefetch_tmap(tmW);
    prefetch_tmap(tmR);
  }
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const uint32_t full0 = PAIR ? cluster_addr(&m.full[0], 0) : smem_u32(&m.full[0]);
  const int rep_rows = kTok / bx.reps;
  int st = 0, it = 0;
  uint32_t phase = 1;
  bool ok = true;
  for (int j = 0; ok && j < nt; ++j) {
    const Tile t = tile_of(j);
    const int w0 = t.u * kUnit + (PAIR ? (int)rank * t.units * (kUnit / 2) : 0);  // first vocabulary row here
    // a box may hold more units than the tile (at the vocabulary's end): they are not used
    const bool rest = t.units <= bx.rest;
    const CUtensorMap* tm = rest ? tmR : tmW;
    const uint32_t bytes = (PAIR ? 2 : 1) * (bx.reps * bx.rows * 128 + (rest ? bx.rest : bx.wide) * R::UNIT);
    for (int kc = 0; kc < KS; ++kc, ++it) {
      if (!g.wait(&m.empty[st], phase, TOKENS ? 55 : 50)) { ok = false; break; }
      uint8_t* sh = ring + st * R::STAGE;
      const uint32_t full = full0 + st * 8;
      if (TOKENS) {
        if (PAIR)
          tma_load_2d_pair(sh, tmH, full, kc * 64, t.tm * kTok);
        else
          for (int r = 0; r < bx.reps; ++r)
            tma_load_2d(sh + r * rep_rows * 128, tmH, &m.full[st], kc * 64, t.tm * rep_rows);
      } else {
        if (rank == 0) mbar_expect_tx(&m.full[st], bytes);
        if (PAIR)
          tma_load_2d_pair(sh + kSliceH, tm, full, kc * 64, w0);
        else
          tma_load_2d(sh + kSliceH, tm, &m.full[st], kc * 64, w0);
      }
      if (++st == R::STAGES) {
        st = 0;
        phase ^= 1;
      }
    }
  }
  // No copy may still be landing when the CTA exits, and in a pair no arrival
  // of the other CTA's: there each stage's last release says both.
  for (int i = (it > R::STAGES ? it - R::STAGES : 0); i < it; ++i)
    g.drain(PAIR ? &m.empty[i % R::STAGES] : &m.full[i % R::STAGES], (i / R::STAGES) & 1);
}

// Warp 1 (of rank 0 in a pair): the tile's products into accumulator j mod 2.
// The whole warp runs the loop and the waits; lane 0 issues.
template <bool PAIR, class TileOf>
__device__ __forceinline__ void multiply_tiles(Misc& m, const Guard& g, uint32_t sRing, uint32_t tmem, int nt, int KS,
                                               TileOf tile_of) {
  using R = Ring<PAIR>;
  if (PAIR && cluster_rank() != 0) return;
  const bool leader = (threadIdx.x & 31) == 0;
  bool ok = true;
  int it = 0;
  for (int j = 0; ok && j < nt; ++j) {
    const int buf = j & 1;
    const uint32_t id = idesc_bf16_f32(PAIR ? 256 : 128, tile_of(j).units * kUnit, false, false);
    if (j >= 2 && !g.wait_warp(&m.acc_empty[buf], ((j - 2) >> 1) & 1, 51)) { ok = false; break; }
    if (PAIR) fence_cluster();  // half of the arrivals are the other CTA's
    tc_fence_after();
    for (int kc = 0; kc < KS; ++kc, ++it) {
      const int st = it % R::STAGES;
      if (!g.wait_warp(&m.full[st], (it / R::STAGES) & 1, 52)) { ok = false; break; }
      tc_fence_after();
      const uint64_t hd = sdesc_sw128(sRing + st * R::STAGE, 16, 1024);
      const uint64_t wd = sdesc_sw128(sRing + st * R::STAGE + kSliceH, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        if (leader) {
          const uint32_t add = (kc > 0 || kk > 0) ? 1u : 0u;
          if (PAIR)
            umma_bf16_pair(tmem + buf * 256, sdesc_add(hd, kk * 32), sdesc_add(wd, kk * 32), id, add);
          else
            umma_bf16(tmem + buf * 256, sdesc_add(hd, kk * 32), sdesc_add(wd, kk * 32), id, add);
        }
      if (leader) PAIR ? umma_commit_pair(&m.empty[st]) : umma_commit(&m.empty[st]);
      __syncwarp();
    }
    if (ok && leader) PAIR ? umma_commit_pair(&m.acc_full[buf]) : umma_commit(&m.acc_full[buf]);
    __syncwarp();
  }
  if (leader) {
    PAIR ? umma_commit_pair_own(&m.fin) : umma_commit(&m.fin);  // every MMA issued has completed once this arrives
    g.drain(&m.fin, 0);
  }
  __syncwarp();
}

// An epilogue thread has read its share of accumulator `buf`.
template <bool PAIR>
__device__ __forceinline__ void release_acc(Misc& m, int buf) {
  tc_fence_before();
  if (PAIR)
    mbar_arrive_cluster(cluster_addr(&m.acc_empty[buf], 0));
  else
    mbar_arrive(&m.acc_empty[buf]);
}

// Put (v, id) into a list that runs from the largest down, behind every entry
// that is not smaller: with ids coming in increasing order, equal values keep
// the lower id first. v = -inf leaves the list as it is.
template <int KM>
__device__ __forceinline__ void insert(float (&z)[KM], int (&id)[KM], float v, int vid) {
#pragma unroll
  for (int p = KM - 1; p > 0; --p) {
    id[p] = v > z[p - 1] ? id[p - 1] : (v > z[p] ? vid : id[p]);
    z[p] = fmaxf(z[p], fminf(z[p - 1], v));
  }
  id[0] = v > z[0] ? vid : id[0];
  z[0] = fmaxf(z[0], v);
}

// What the epilogue warps leave for each other where they share tokens.
struct Joint {
  float4 sums[4][32];              // [quarter][lane] {m, S, A, the target's raw logit}
  float2 top[4][kLogpMaxTop][32];  // [quarter][slot][lane] {raw logit, vocabulary row}
};
static_assert(sizeof(Joint) <= Ring<false>::BYTES, "fits the ring");

// sum * f + x into sum, and what the product and the addition have rounded off
// into lost (Knuth, "The Art of Computer Programming" 2, 4.2.2: the error of an
// addition is itself a float). The intrinsics keep them from being fused.
__device__ __forceinline__ void add_kept(float& sum, float& lost, float f, float x) {
  const float p = __fmul_rn(sum, f), s = __fadd_rn(p, x), b = __fsub_rn(s, p);
  const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(s, b)), __fsub_rn(x, b));
  lost = fmaf(lost, f, __fadd_rn(fmaf(sum, f, -p), e));
  sum = s;
}

// d of a sum kept under the maximum `was` when that becomes m (0 before there is one).
__device__ __forceinline__ float shift_of(float was, float m, float sl2) {
  return was > -INFINITY ? fmaxf((was - m) * sl2, kFar) : 0.f;
}

// (m, S, A) of two disjoint sets of columns as that of both.
__device__ __forceinline__ void join(float4& x, const float4& y, float sl2) {
  const float m = fmaxf(x.x, y.x);
  const float dx = shift_of(x.x, m, sl2), dy = shift_of(y.x, m, sl2);
  const float sx = ex2(dx), sy = ex2(dy);
  x.z = fmaf(fmaf(dx, x.y, x.z), sx, fmaf(dy, y.y, y.z) * sy);
  x.y = fmaf(x.y, sx, y.y * sy);
  x.x = m;
  x.w += y.w;  // 0 where the target lies in other columns
}

// The split's results of one token whose columns the warps quarter,
// quarter + groups, ... have taken: the sums joined, the lists merged (among
// equal logits the lower row first).
template <int KL>
__device__ __forceinline__ void write_joint(const FwdParams& p, const Joint& j, int quarter, int lane, int groups,
                                            int token, bool lists) {
  float4 x = j.sums[quarter][lane];
  for (int r = 1; r < p.boxes.reps; ++r) join(x, j.sums[quarter + r * groups][lane], p.sl2);
  p.part[(size_t)blockIdx.y * p.N + token] = x;
  if (!lists) return;
  const int first = KL - p.top;  // slots before it hold no candidates
  float2 head[4];
  int pos[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    pos[r] = first;
    head[r] = r < p.boxes.reps ? j.top[quarter + r * groups][first][lane] : make_float2(-INFINITY, __int_as_float(-1));
  }
  float2* out = p.cand + ((size_t)token * p.splits + blockIdx.y) * p.top;
  for (int k = 0; k < p.top; ++k) {
    int best = 0;
    float2 b = head[0];
#pragma unroll
    for (int r = 1; r < 4; ++r)
      if (head[r].x > b.x || (head[r].x == b.x && (unsigned)__float_as_int(head[r].y) < (unsigned)__float_as_int(b.y))) {
        b = head[r];
        best = r;
      }
    out[k] = b;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r == best && ++pos[r] < KL)
        head[r] = j.top[quarter + r * groups][pos[r]][lane];
      else if (r == best)
        head[r] = make_float2(-INFINITY, __int_as_float(-1));
  }
}

// The same for values alone.
template <int KM>
__device__ __forceinline__ void insert_value(float (&z)[KM], float v) {
#pragma unroll
  for (int p = KM - 1; p > 0; --p) z[p] = fmaxf(z[p], fminf(z[p - 1], v));
  z[0] = fmaxf(z[0], v);
}

// The largest float below x (-inf stays).
__device__ __forceinline__ float below(float x) {
  const int b = __float_as_int(x);
  return x == 0.f ? -1.4e-45f : __int_as_float(x > 0.f ? b - 1 : x > -INFINITY ? b + 1 : b);
}

// 32 columns of this thread's TMEM lane from vocabulary row vc on, those past V as -inf.
__device__ __forceinline__ void load_chunk(uint32_t taddr, int vc, int V, uint32_t (&a)[32]) {
  tmem_ld32(taddr, a);
  if (vc + 32 > V) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (vc + i >= V) a[i] = __float_as_uint(-INFINITY);
  }
}

// Forward. CTA (token tile blockIdx.x, split blockIdx.y) walks its split's
// units in tiles of up to eight; the epilogue warps hold one token per thread. The
// alternatives are kept in registers, KM slots of which the first KM - top are
// filled with +inf, so that the smallest kept value is always in the last
// slot: a 32-column chunk (then each eight of it) in which no lane's maximum
// beats it is done with one vote. Otherwise each lane notes its columns that do
// in a buffer of 32, and only when some lane's would overflow do all lanes put
// theirs into their lists, side by side. A row gets a new alternative ever more rarely (in
// column n with probability top / n), but one of a warp's 32 rows nearly
// always does: inserting column by column, for the one or two lanes that want
// it, took 777 tokens with 8 alternatives over V 50,257, D 1024 from 71 to
// 144 us; with the buffers it was 103 us. Most of a list's insertions come from
// the first columns, so the first tile is read twice: the top-th largest of
// its groups' maxima (two, four or eight columns each) is a value that `top`
// columns reach, and only columns that reach it are taken: 99 us then, 89 us with
// the loaders and plans that came after (and 17 tokens with 20 of them over V
// 151,936, D 4096 205 us instead of 211).
//
// A TMEM lane is read by one warp of the four alone, so with few tokens most
// epilogue warps would have none. For N <= 64 (32) the tile holds the tokens'
// rows twice (four times) instead of rows past N: the product costs the same,
// and each warp takes every second (fourth) 32-column chunk of the tokens,
// whose results the CTA joins through shared memory at the end. 17 tokens with
// 20 alternatives at V 151,936, D 4096 took 217 us without and 206 us with it
// (before the buffers).
template <int KM, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    logp_fwd_kernel(const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmR, const FwdParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Misc& m = *reinterpret_cast<Misc*>(smem_raw);
  uint8_t* ring =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1024 + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int U = (p.V + kUnit - 1) / kUnit;
  const int u0 = (int)blockIdx.y * p.units_per_split, u1 = min(u0 + p.units_per_split, U);
  const int width = p.boxes.wide, nt = (u1 - u0 + width - 1) / width;  // >= 1 by construction of the grid
  const int KS = p.D / 64;
  const Guard g{&m.abort_flag, p.status};
  const auto tile_of = [&](int j) {
    const int u = u0 + j * width;
    return Tile{(int)blockIdx.x, u, min(width, u1 - u)};
  };
  // The status word starts at 0: no wait can give up within 2 s of the launch.
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0u;
  setup<PAIR>(m, kThreads - 128);
  // the merge may take its place on the SMs; it waits for this kernel's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = m.tmem_base;

  if (warp == 0) {
    if (lane == 0) load_tiles<PAIR, false>(m, g, ring, &tmH, &tmW, &tmR, nt, KS, p.boxes, tile_of);
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) load_tiles<PAIR, true>(m, g, ring, &tmH, &tmW, &tmR, nt, KS, p.boxes, tile_of);
    __syncwarp();
  } else if (warp == 1) {
    multiply_tiles<PAIR>(m, g, smem_u32(ring), tmem, nt, KS, tile_of);
  } else if (warp >= 4) {
    const int quarter = warp & 3;
    const int groups = 4 / p.boxes.reps, share = quarter / groups;  // this warp's share of the columns
    const int row0 = (int)blockIdx.x * (kTok / p.boxes.reps) + (quarter % groups) * 32, token = row0 + lane;
    const bool live = token < p.N, any = row0 < p.N;
    const int t = live ? p.targets[token] : -1;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    constexpr int KL = KM > 0 ? KM : 1;
    float tz[KL];
    int ti[KL];
    const auto clear_list = [&]() {
#pragma unroll
      for (int k = 0; k < KL; ++k) {
        tz[k] = k < KM - p.top ? INFINITY : -INFINITY;
        ti[k] = -1;
      }
    };
    clear_list();
    float least = -INFINITY;  // no alternative is this small or smaller
    float2* mine = reinterpret_cast<float2*>(ring + Ring<PAIR>::BYTES) + quarter * 32 + lane;  // entry e at 128 e
    const uint32_t mine_at = smem_u32(mine);
    uint32_t held = 0;
    const auto insert_held = [&]() {  // in column order, so that equal values keep the lower row first
      const uint32_t most = __reduce_max_sync(~0u, held);
      float2 next = mine[0];
      for (uint32_t e = 0; e < most; ++e) {
        const float2 x = next;
        next = mine[128 * min(e + 1, kCands - 1u)];
        insert<KL>(tz, ti, e < held ? x.x : -INFINITY, __float_as_int(x.y));
      }
      held = 0;
      least = fmaxf(least, tz[KL - 1]);
    };
    float m_run = -INFINITY, s_run = 0.f, a_run = 0.f, s_lost = 0.f, a_lost = 0.f, tgt = 0.f;
    const uint64_t sl2 = f2(p.sl2, p.sl2);
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      const int buf = j & 1;
      ok = __all_sync(~0u, g.wait(&m.acc_full[buf], (j >> 1) & 1, 53));
      if (!ok) break;
      tc_fence_after();
      const Tile tl = tile_of(j);
      if (KM > 0 && j == 0 && any) {
#pragma unroll 1
        for (int c = share; c < tl.units; c += p.boxes.reps) {
          uint32_t a[32];
          load_chunk(tmem + lane_base + buf * 256 + c * 32, (tl.u + c) * kUnit, p.V, a);
          if (KM == 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) insert_value<KL>(tz, fmaxf(max_of<8>(a, q), -INFINITY));  // NaN as -inf
          } else if (p.boxes.reps == 1) {
#pragma unroll
            for (int q = 0; q < 8; ++q) insert_value<KL>(tz, fmaxf(max_of<4>(a, q), -INFINITY));
          } else {
#pragma unroll
            for (int q = 0; q < 16; ++q) insert_value<KL>(tz, fmaxf(max_of<2>(a, q), -INFINITY));
          }
        }
        least = below(tz[KL - 1]);
        clear_list();
      }
      if (any) {
#pragma unroll 1
        for (int c = share; c < tl.units; c += p.boxes.reps) {
          uint32_t a[32];
          const int vc = (tl.u + c) * kUnit;
          load_chunk(tmem + lane_base + buf * 256 + c * 32, vc, p.V, a);
          float m8[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) m8[q] = max_of<8>(a, q);
          const float cmax = fmaxf(fmax3(m8[0], m8[1], m8[2]), m8[3]);
          // a row with nothing but -inf so far: the shift is 0, and S and A stay 0
          const float m_new = fmaxf(m_run, cmax);
          const float shift = m_new > -INFINITY ? m_new : 0.f;
          const uint64_t off = f2(-shift, -shift);
          uint64_t s2 = 0ull, a2 = 0ull;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 x = f2_split(mul2(add2(f2(__uint_as_float(a[i]), __uint_as_float(a[i + 1])), off), sl2));
            const uint64_t e = f2(ex2(x.x), ex2(x.y));
            s2 = add2(s2, e);
            // 2^t t -> 0 as t -> -inf: a finite factor keeps 0 * inf out
            a2 = fma2(e, f2(fmaxf(x.x, kFar), fmaxf(x.y, kFar)), a2);
          }
          const float2 ss = f2_split(s2), aa = f2_split(a2);
          const float d = shift_of(m_run, shift, p.sl2), sc = ex2(d);
          a_run = fmaf(d, s_run, a_run);
          a_lost = fmaf(d, s_lost, a_lost);
          add_kept(a_run, a_lost, sc, aa.x + aa.y);
          add_kept(s_run, s_lost, sc, ss.x + ss.y);
          m_run = m_new;
          if (t >= vc && t < vc + 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (t == vc + i) tgt = __uint_as_float(a[i]);
          }
          if (KM > 0) {
            if (__any_sync(~0u, live && cmax > least)) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (!__any_sync(~0u, live && m8[q] > least)) continue;
                uint32_t want = over8(a, q, live ? least : INFINITY);
                if (__any_sync(~0u, held + __popc(want) > kCands)) {
                  insert_held();
                  want = over8(a, q, live ? least : INFINITY);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint32_t bit = (want >> i) & 1u;
                  st_shared_if(bit, mine_at + held * (128 * sizeof(float2)), a[8 * q + i], vc + 8 * q + i);
                  held += bit;
                }
              }
            }
          }
        }
      }
      release_acc<PAIR>(m, buf);
    }
    s_run += s_lost;
    a_run += a_lost;
    if (KM > 0) insert_held();
    if (!PAIR && p.boxes.reps > 1) {
      // every product has completed and every copy been read: the ring is free
      Joint* joint = reinterpret_cast<Joint*>(ring);
      joint->sums[quarter][lane] = make_float4(m_run, s_run, a_run, tgt);
      if (KM > 0) {
#pragma unroll
        for (int k = 0; k < KL; ++k) joint->top[quarter][k][lane] = make_float2(tz[k], __int_as_float(ti[k]));
      }
      named_bar_sync(1, 128);  // warps 4..7, whether their waits ended well or not
      if (ok && live && share == 0) write_joint<KL>(p, *joint, quarter, lane, groups, token, KM > 0);
    } else if (ok && live) {
      p.part[(size_t)blockIdx.y * p.N + token] = make_float4(m_run, s_run, a_run, tgt);
      if (KM > 0) {
        const size_t o = ((size_t)token * p.splits + blockIdx.y) * p.top;
#pragma unroll
        for (int k = 0; k < KL; ++k) {
          const int at = k - (KM - p.top);
          if (at >= 0) p.cand[o + at] = make_float2(tz[k], __int_as_float(ti[k]));
        }
      }
    }
  }
  teardown<PAIR>(tmem);
}

// Bits of a float in an unsigned order, both zeros alike; > 0 for every number.
__device__ __forceinline__ uint32_t ordered(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The splits' results of a token: their (m, S, A) in a fixed tree, then `top`
// rounds that each take the largest head of the splits' lists (lowest row first
// among equals), staged in shared memory. One warp per token and eight tokens a
// block, or, where tokens are few, a block per token (WPT = 8): reading the
// lists is what takes the time, 3,000 entries for 20 alternatives of 149
// splits, and eight warps have eight times the loads in flight. Each lane of
// the token's first warp owns the splits lane, lane + 32, ....
// 6.2 us for a token's five alternatives of 143 splits, 10.2 us for 17 tokens'
// 20 of 149 (8.3 and 12.9 with the loads in three steps and heads in shared memory).
constexpr int kListsPerLane = (kLogpMaxSplits + 31) / 32;
template <int WPT>
__global__ void __launch_bounds__(256) logp_merge_kernel(const FwdParams p, float* __restrict__ logp,
                                                         float* __restrict__ lse, float* __restrict__ entropy,
                                                         int32_t* __restrict__ top_ids, float* __restrict__ top_logp) {
  extern __shared__ float2 lists[];  // per token: splits x top {logit, row}
  const int lane = threadIdx.x & 31, tokens = (blockDim.x >> 5) / WPT, slot = (threadIdx.x >> 5) / WPT;
  const int token = blockIdx.x * tokens + slot;
  const int n = p.splits * p.top;
  float2* mine = lists + (size_t)slot * n;
  const bool first = (threadIdx.x >> 5) % WPT == 0 && token < p.N;
  const int t = first ? p.targets[token] : -1;  // an input: read before the forward has ended
  const bool scored = t >= 0 && t < p.V;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // everything that is read goes out at once
  const float zt = scored ? p.part[(size_t)(t / kUnit / p.units_per_split) * p.N + token].w : 0.f;
  float4 q[kListsPerLane];
#pragma unroll
  for (int l = 0; l < kListsPerLane; ++l) {
    const int s = lane + 32 * l;
    q[l] = first && s < p.splits ? p.part[(size_t)s * p.N + token] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
  }
  if (token < p.N) {
    const float2* from = p.cand + (size_t)token * n;
#pragma unroll 8
    for (int i = threadIdx.x % (32 * WPT); i < n; i += 32 * WPT) mine[i] = from[i];
  }
  if (WPT > 1)
    __syncthreads();
  else
    __syncwarp();
  if (!first) return;
  float M = -INFINITY;
#pragma unroll
  for (int l = 0; l < kListsPerLane; ++l) M = fmaxf(M, q[l].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
  float S = 0.f, A = 0.f;
#pragma unroll
  for (int l = 0; l < kListsPerLane; ++l) {
    const float d = shift_of(q[l].x, M, p.sl2), sc = exp2f(d);
    S = fmaf(q[l].y, sc, S);
    A = fmaf(fmaf(d, q[l].y, q[l].z), sc, A);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    S += __shfl_xor_sync(~0u, S, o);
    A += __shfl_xor_sync(~0u, A, o);
  }
  // From the logit and not from lse: a likely token's log probability is a
  // small difference, which lse would have rounded off.
  const float l2 = log2f(S), ls = fmaf(M, p.inv_t, kLn2 * l2);
  const auto log_p = [&](float z) { return kLn2 * fmaf(z - M, p.sl2, -l2); };
  if (lane == 0) {
    const float h = kLn2 * (l2 - A / S);
    logp[token] = scored ? log_p(zt) : 0.f;
    lse[token] = ls;
    entropy[token] = h < 0.f ? 0.f : h;  // rounding below the least entropy there is; NaN stays
  }
  if (p.top == 0) return;
  // Each list's head and the entry behind it are kept in registers, so that a
  // round is two warp reductions; lane k keeps the outcome of round k.
  uint32_t key[kListsPerLane], row[kListsPerLane], next_key[kListsPerLane], next_row[kListsPerLane];
  int at[kListsPerLane];  // entry after next
  const auto fetch = [&](int l, int e, uint32_t& k, uint32_t& r) {  // key 0: the list is at its end
    const int s = lane + 32 * l;
    k = 0;
    r = 0xFFFFFFFFu;
    if (s >= p.splits || e >= p.top) return;
    const float2 x = mine[s * p.top + e];
    r = (uint32_t)__float_as_int(x.y);
    if (__float_as_int(x.y) >= 0) k = ordered(x.x);
  };
#pragma unroll
  for (int l = 0; l < kListsPerLane; ++l) {
    fetch(l, 0, key[l], row[l]);
    fetch(l, 1, next_key[l], next_row[l]);
    at[l] = 2;
  }
  uint32_t my_key = 0, my_row = 0;
  for (int k = 0; k < p.top; ++k) {
    uint32_t best = key[0], best_row = row[0];
    int bl = 0;
#pragma unroll
    for (int l = 1; l < kListsPerLane; ++l)
      if (key[l] > best) {  // the lower split of a lane's equal heads holds the lower rows
        best = key[l];
        best_row = row[l];
        bl = l;
      }
    const uint32_t most = __reduce_max_sync(~0u, best);
    if (most == 0) break;  // fewer logits above -inf than asked for
    const uint32_t low = __reduce_min_sync(~0u, best == most ? best_row : 0xFFFFFFFFu);
    if (lane == k) {
      my_key = most;
      my_row = low;
    }
    if (best == most && best_row == low) {  // one lane: rows differ
#pragma unroll
      for (int l = 0; l < kListsPerLane; ++l)
        if (l == bl) {
          key[l] = next_key[l];
          row[l] = next_row[l];
          fetch(l, at[l]++, next_key[l], next_row[l]);
        }
    }
    __syncwarp();
  }
  if (lane < p.top) {
    const float z = __uint_as_float(my_key & 0x80000000u ? my_key ^ 0x80000000u : ~my_key);
    top_ids[(size_t)token * p.top + lane] = my_key ? (int32_t)my_row : -1;
    top_logp[(size_t)token * p.top + lane] = my_key ? log_p(z) : -INFINITY;
  }
}

// min(x, 0); NaN stays.
__device__ __forceinline__ float not_above_0(float x) {
  float r;
  asm("min.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
  return r;
}

// Backward, one chunk of the vocabulary: one CTA per SM over the chunk's
// (token tile, vocabulary tile) pairs; the vocabulary tiles have eight units,
// or fewer where that makes the longest CTA shorter (few tokens). Each
// recomputed logit becomes
//   dz = p (cA + cB log2 p) + [v = t] g / T,
//   cA = -(g + e H) / T,  cB = -e ln 2 / T,
// exactly 0 in rows without a gradient and in columns past V. p is cut at 1: from
// logits of 2^24 on the roundings of z and lse alone could make it anything up to
// infinity, and with one such token the whole head's gradient. dz is rounded to
// bf16, the operand type of the two products that follow (at most 2^-8 of the
// value, as in the cross-entropy's backward; sums stay in fp32).
// That and the results' own rounding, 1.66e-3 of the norm each, make 2.35e-3. But
// the gradients of a few tokens hang on the few values at their targets, whose
// roundings do not average out: 3.5e-3 for one token, 2.6e-3 for 96. So up to
// 128 tokens, where the products wait for the head more than for the tensor pipe,
// dz is the sum of two bf16 terms (2^-16 of the value): the results' rounding
// alone is left, for 97 us instead of 84 (both gradients of 96 tokens over V
// 32,003, D 2048).
template <bool PAIR, int TERMS>
__global__ void __launch_bounds__(kDzThreads, 1)
    logp_dz_kernel(const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmW,
                   const BwdParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Misc& m = *reinterpret_cast<Misc*>(smem_raw);
  uint8_t* ring =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1024 + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // token tiles are counted in rows of 256 in a pair
  constexpr int kPer = PAIR ? 2 : 1;
  const int cta = (int)blockIdx.x / kPer, ctas = (int)gridDim.x / kPer, rank = PAIR ? (int)blockIdx.x % 2 : 0;
  const int TM = (p.N + kPer * kTok - 1) / (kPer * kTok), units = (p.v_end - p.v_base + kUnit - 1) / kUnit;
  const int VT = (units + p.tile_units - 1) / p.tile_units;
  const int nt = (TM * VT - cta + ctas - 1) / ctas;
  const int KS = p.D / 64;
  const Guard g{&m.abort_flag, p.status};
  const auto tile_of = [&](int j) {
    constexpr int kG = kGroup / kPer;
    const int q = cta + j * ctas;
    const int gi = q / (kG * VT), r = q - gi * kG * VT;
    const int g0 = gi * kG, gs = min(kG, TM - g0);
    const int u = r / gs * p.tile_units;
    return Tile{(g0 + r % gs) * kPer + rank, p.v_base / kUnit + u, min(p.tile_units, units - u)};
  };
  if (p.first && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;  // no wait can give up within 2 s
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  setup<PAIR>(m, kDzThreads - 128);
  if (!p.first) asm volatile("griddepcontrol.wait;" ::: "memory");  // the last chunk's products have read dz
  const uint32_t tmem = m.tmem_base;

  if (warp == 0) {
    if (lane == 0) load_tiles<PAIR, false>(m, g, ring, &tmH, &tmW, &tmW, nt, KS, p.boxes, tile_of);
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) load_tiles<PAIR, true>(m, g, ring, &tmH, &tmW, &tmW, nt, KS, p.boxes, tile_of);
    __syncwarp();
  } else if (warp == 1) {
    multiply_tiles<PAIR>(m, g, smem_u32(ring), tmem, nt, KS, tile_of);
  } else if (warp >= 4) {
    const int quarter = warp & 3;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    for (int j = 0; j < nt; ++j) {
      const int buf = j & 1;
      const Tile tl = tile_of(j);
      const int token = tl.tm * kTok + quarter * 32 + lane;
      const bool live = token < p.N;
      const int t = live ? p.targets[token] : -1;
      const float gl = live && t >= 0 && t < p.V ? p.g_logp[token] : 0.f;
      const float ge = live && p.g_entropy ? p.g_entropy[token] : 0.f;
      const bool use = gl != 0.f || ge != 0.f;
      const float cA = -p.inv_t * (ge != 0.f ? fmaf(ge, p.entropy[token], gl) : gl), cB = -p.inv_t * ge * kLn2;
      const float one = p.inv_t * gl, l2 = use ? p.lse[token] * kLog2e : 0.f;
      if (!__all_sync(~0u, g.wait(&m.acc_full[buf], (j >> 1) & 1, 54))) break;
      tc_fence_after();
      const int v0 = tl.u * kUnit, c0v = v0 - p.v_base;  // column of v0 in the chunk
#pragma unroll 1
      for (int c0 = (warp >> 2) % 2 * 32; c0 < tl.units * kUnit; c0 += 64) {  // every second unit
        uint32_t a[32];
        tmem_ld32(tmem + lane_base + buf * 256 + c0, a);
        const int vc = v0 + c0;
        float d[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float x = not_above_0(fmaf(__uint_as_float(a[i]), p.sl2, -l2));
          d[i] = ex2(x) * fmaf(cB, fmaxf(x, kFar), cA);
        }
        if (t >= vc && t < vc + 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (t == vc + i) d[i] += one;
        }
        if (!use || vc + 32 > p.V) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!use || vc + i >= p.V) d[i] = 0.f;
        }
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            w[i] = pack_bf16x2(d[2 * i], d[2 * i + 1]);
            if (term + 1 < TERMS) {  // what is left for the next term
              d[2 * i] -= __uint_as_float(w[i] << 16);
              d[2 * i + 1] -= __uint_as_float(w[i] & 0xFFFF0000u);
            }
          }
          if (!live) continue;
          __nv_bfloat16* row = p.dz + ((size_t)term * p.N + token) * p.ld_dz + c0v + c0;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (vc + 8 * u < p.V)
              *reinterpret_cast<uint4*>(row + 8 * u) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
          if (!p.dzt) continue;
          __nv_bfloat16* colp = p.dzt + ((size_t)term * p.ld_dz + c0v + c0) * p.ld_dzt + token;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (vc + i < p.V)
              colp[(size_t)i * p.ld_dzt] =
                  __ushort_as_bfloat16((unsigned short)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu));
        }
      }
      release_acc<PAIR>(m, buf);
    }
  }
  teardown<PAIR>(tmem);
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms <= 0)
    sms = 152;
  return sms;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Rows of a token tile that a launch brings in.
static int token_rows(int N) { return N < kTok ? (N + 7) / 8 * 8 : kTok; }
// How often a forward tile repeats its tokens.
static int token_reps(int N) { return N <= 32 ? 4 : N <= 64 ? 2 : 1; }

// Most splits of the vocabulary: each at least one unit, and no more CTAs in
// all than about sixteen a SM.
int logp_max_splits(int N, int V) {
  const int TM = (N + kTok - 1) / kTok, U = (V + kUnit - 1) / kUnit;
  int s = 2432 / TM;
  if (s > kLogpMaxSplits) s = kLogpMaxSplits;
  if (s > U) s = U;
  return s < 1 ? 1 : s;
}

// Cycles that a K slice of a tile of `units` takes a CTA (or a pair), as
// measured: a round of waiting for a stage, announcing and issuing its copies,
// 360; the products, 64 a unit and 110 for the shared memory that copies and
// operands share (622 for 256 columns: a pair's 82% of the tensor pipe); the
// copies, 74 bytes a cycle with every SM copying; and the head's rows out of
// DRAM, 23 bytes a cycle and SM, shared by the `sharing` token tiles that read
// them at about the same time.
static long long slice_cycles(int units, bool pair, int token_bytes, int sharing) {
  const int head_bytes = units * (int)(pair ? Ring<true>::UNIT : Ring<false>::UNIT);
  long long c = 360;
  for (const long long x :
       {64ll * units + 110, (long long)(token_bytes + head_bytes) / 74, (long long)head_bytes / (23ll * sharing)})
    if (x > c) c = x;
  return c;
}

// The split of the vocabulary over `slots` CTAs (or pairs) at once that takes
// the fewest cycles, tiles of a split about equal: waves x (the tiles' slices +
// 12,000 and 400 a slice for a CTA's start, the pipeline's fill, the last
// epilogue and the exit: 8,192 tokens over V 151,936, D 4096 took 5.60 ms in
// three waves and 5.73 ms in eight that fill the SMs a little better).
static LogpPlan best_plan(int N, int V, int D, int slots, bool pair, long long* cost_out) {
  const int rows = pair ? 2 * kTok : kTok, TM = (N + rows - 1) / rows, U = (V + kUnit - 1) / kUnit;
  const int token_bytes = token_rows(N) * 128 * token_reps(N);
  LogpPlan best{pair, 1, U, kTileUnits};
  long long best_cost = -1;
  for (int s = 1, most = logp_max_splits(N, V); s <= most; ++s) {
    const int per = (U + s - 1) / s, used = (U + per - 1) / per;
    const int tiles = (per + kTileUnits - 1) / kTileUnits, width = (per + tiles - 1) / tiles;
    const long long slices = (tiles - 1) * slice_cycles(width, pair, token_bytes, TM) +
                             slice_cycles(per - (tiles - 1) * width, pair, token_bytes, TM);
    const long long waves = ((long long)TM * used + slots - 1) / slots, cost = waves * ((slices + 400) * (D / 64) + 12000);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = LogpPlan{pair, used, per, width};
    }
  }
  *cost_out = best_cost;
  return best;
}

// Pairs of CTAs where that is faster; tokens then come in rows of 256, so 777
// of them are 1,024 rows instead of 896.
LogpPlan logp_plan(int N, int V, int D, int sms) {
  long long single = 0, paired = 0;
  const LogpPlan a = best_plan(N, V, D, sms, false, &single);
  if (N <= kTok || sms < 2) return a;
  const LogpPlan b = best_plan(N, V, D, sms / 2, true, &paired);
  return paired < single ? b : a;
}

LogpFwdLayout logp_fwd_layout(int N, int V, int top) {
  const size_t rows = (size_t)logp_max_splits(N, V) * N;
  LogpFwdLayout L;
  L.part = 256;
  L.cand = L.part + up256(rows * sizeof(float4));
  L.bytes = L.cand + up256(rows * top * sizeof(float2));
  return L;
}

cudaError_t launch_logp_fwd(int N, int V, int D, float temperature, int top, const void* hidden, const void* head,
                            const int32_t* targets, float* logp, float* lse, float* entropy, int32_t* top_ids,
                            float* top_logp, void* ws, cudaStream_t st) {
  const LogpPlan sp = logp_plan(N, V, D, sm_count());
  const LogpFwdLayout L = logp_fwd_layout(N, V, top);
  CUtensorMap tH, tW, tR;
  const int cut = sp.pair ? 2 : 1, rest = sp.per % sp.width;
  const Boxes bx{sp.width, rest, token_rows(N), token_reps(N)};
  if (!tmap_bf16_2d_sw128(&tH, hidden, D, N, bx.rows) || !tmap_bf16_2d_sw128(&tW, head, D, V, sp.width * kUnit / cut) ||
      !tmap_bf16_2d_sw128(&tR, head, D, V, (rest ? rest : sp.width) * kUnit / cut))
    return cudaErrorInvalidValue;
  uint8_t* w = static_cast<uint8_t*>(ws);
  FwdParams p{};
  p.boxes = bx;
  p.N = N;
  p.V = V;
  p.D = D;
  p.top = top;
  p.units_per_split = sp.per;
  p.splits = sp.splits;
  p.sl2 = kLog2e / temperature;
  p.inv_t = 1.f / temperature;
  p.targets = targets;
  p.part = reinterpret_cast<float4*>(w + L.part);
  p.cand = reinterpret_cast<float2*>(w + L.cand);
  p.status = reinterpret_cast<uint32_t*>(w);
  // lists of the next multiple of eight slots: inserting costs five instructions a slot
  const auto kfn = top == 0    ? (sp.pair ? logp_fwd_kernel<0, true> : logp_fwd_kernel<0, false>)
                   : top <= 8  ? (sp.pair ? logp_fwd_kernel<8, true> : logp_fwd_kernel<8, false>)
                   : top <= 16 ? (sp.pair ? logp_fwd_kernel<16, true> : logp_fwd_kernel<16, false>)
                   : top <= 24 ? (sp.pair ? logp_fwd_kernel<24, true> : logp_fwd_kernel<24, false>)
                               : (sp.pair ? logp_fwd_kernel<kLogpMaxTop, true> : logp_fwd_kernel<kLogpMaxTop, false>);
  const uint32_t smem = top == 0 ? kSmem : kSmemTop;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sp.pair ? (N + 2 * kTok - 1) / (2 * kTok) * 2 : (N + kTok - 1) / kTok, sp.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr = cluster_pair();
    cfg.attrs = &attr;
    cfg.numAttrs = sp.pair ? 1 : 0;
    if ((e = cudaLaunchKernelEx(&cfg, kfn, tH, tW, tR, p)) != cudaSuccess) return e;
  }
  // a block per token while that fills less than two rounds of the SMs; else
  // as many tokens a block as 40 KB of lists hold, 8 at most
  const size_t lists = (size_t)sp.splits * top * sizeof(float2);
  const bool few = top > 0 && N <= 304;
  int warps = 8;
  if (!few)
    while (warps > 1 && warps * lists > 40960) --warps;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(few ? N : (N + warps - 1) / warps);
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = few ? lists : warps * lists;
  cfg.stream = st;
  cudaLaunchAttribute attr = programmatic_launch();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? logp_merge_kernel<8> : logp_merge_kernel<1>, p, logp, lse, entropy, top_ids,
                            top_logp);
}

// Units per vocabulary tile of the dz kernel: the fewest cycles for the CTA (or
// pair) with the most tiles, 1,500 a tile beside its slices.
static int dz_tile_units(int N, int rows, int D, int slots, bool pair, long long* cost_out) {
  const int units = (rows + kUnit - 1) / kUnit, TM = (N + (pair ? 2 : 1) * kTok - 1) / ((pair ? 2 : 1) * kTok);
  int best = kTileUnits;
  long long best_cost = -1;
  for (int u = kTileUnits; u >= 4; --u) {
    const long long tiles = (long long)TM * ((units + u - 1) / u);
    const long long cost = (tiles + slots - 1) / slots * (slice_cycles(u, pair, token_rows(N) * 128, TM) * (D / 64) + 1500);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = u;
    }
  }
  *cost_out = best_cost;
  return best;
}

// SMs for dH where it runs beside dW from the start. With one token tile dW
// only writes the head's gradient and dH only reads the head: one after the
// other they leave DRAM idle at their ends and in the turn between them. Both
// gradients of 96 tokens with dz in one term, in turn / side by side: V 32,003,
// D 2048 94 / 84 us; V 8,192, D 4096 63 / 58 us. From two token tiles on the
// products take their time on the tensor pipe, and halves of the SMs fit fewer
// tile counts (192 tokens, V 32,003, D 2048 103 / 137 us). With two terms, dH on
// 64, 72 or 80 of 152 SMs, 1 and 96 tokens: V 32,003, D 2048 89 and 98, 85 and
// 98, 90 and 103 us; V 151,936, D 4096 702 and 730, 654 and 714, 666 and 763 us.
static int beside_sms(int sms) { return sms / 2 / 8 * 8; }

LogpBwdLayout logp_bwd_layout(int N, int V, int D) {
  LogpBwdLayout L;
  // dz of one chunk takes at most 128 MiB (about what L2 holds), and dz^T, whose
  // rows are padded to whole runs of 64 tokens, at most 256; in whole vocabulary
  // tiles, of which there is one at least (so both are more past 262,144 tokens).
  const long long vmax = (long long)(V + 255) / 256 * 256;
  L.terms = N <= kTok ? 2 : 1;
  L.ld_dzt = (N + 63) / 64 * 64;
  long long vc = (1ll << 26) / (L.terms * (long long)N);
  if (vc > (1ll << 27) / (L.terms * (long long)L.ld_dzt)) vc = (1ll << 27) / (L.terms * (long long)L.ld_dzt);
  vc = vc / 256 * 256;
  if (vc > vmax) vc = vmax;
  if (vc < 256) vc = 256;
  L.vc = (int)vc;
  L.chunks = (V + L.vc - 1) / L.vc;
  const int K = L.vc < V ? L.vc : V;
  L.splits = gemm_splits(N, D, K, 152, L.terms);
  L.splits_beside = N <= kTok ? gemm_splits(N, D, K, beside_sms(152), L.terms) : L.splits;
  const int most = L.splits > L.splits_beside ? L.splits : L.splits_beside;
  L.splits_w = gemm_least_runs(N);
  L.acc = 256;
  L.acc_w = L.acc + (L.chunks > 1 || most > 1 ? up256((size_t)most * N * D * 4) : 0);
  L.dz = L.acc_w + (L.splits_w > 1 ? up256((size_t)L.splits_w * K * D * 4) : 0);
  L.dzt = L.dz + up256((size_t)L.terms * N * L.vc * 2);
  L.bytes = L.dzt + up256((size_t)L.terms * L.vc * L.ld_dzt * 2);
  return L;
}

cudaError_t launch_logp_bwd(int N, int V, int D, float temperature, const void* hidden, const void* head,
                            const int32_t* targets, const float* lse, const float* entropy, const float* g_logp,
                            const float* g_entropy, void* dhidden, void* dhead, void* ws, cudaStream_t st) {
  const LogpBwdLayout L = logp_bwd_layout(N, V, D);
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint32_t* status = reinterpret_cast<uint32_t*>(w);
  __nv_bfloat16* dz = reinterpret_cast<__nv_bfloat16*>(w + L.dz);
  __nv_bfloat16* dzt = reinterpret_cast<__nv_bfloat16*>(w + L.dzt);
  float* acc = reinterpret_cast<float*>(w + L.acc);
  const int sms = sm_count(), TM1 = (N + kTok - 1) / kTok, TM2 = (N + 2 * kTok - 1) / (2 * kTok);
  // dW and dH side by side, each on its part of the SMs
  const int apart = dhead && N <= kTok ? beside_sms(sms) : 0, splits = apart ? L.splits_beside : L.splits;
  const int first_rows = V < L.vc ? V : L.vc;
  long long single = 0, paired = 0;
  dz_tile_units(N, first_rows, D, sms, false, &single);
  if (N > kTok && sms >= 2) dz_tile_units(N, first_rows, D, sms / 2, true, &paired);
  const bool pair = paired > 0 && paired < single;
  const int TM = pair ? TM2 : TM1, slots = pair ? sms / 2 : sms;
  CUtensorMap tH, tHb;
  if (!tmap_bf16_2d_sw128(&tH, hidden, D, N, token_rows(N)) || !tmap_bf16_2d_sw128(&tHb, hidden, D, N, 64))
    return cudaErrorInvalidValue;
  const auto kfn = L.terms > 1 ? logp_dz_kernel<false, 2> : pair ? logp_dz_kernel<true, 1> : logp_dz_kernel<false, 1>;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attrs[2] = {cluster_pair(), programmatic_launch()};
  // Each kernel but the first is launched programmatically behind the one
  // ahead: dz after the products of the chunk before, dW after dz, dH beside dW.
  for (int c = 0; c < L.chunks; ++c) {
    const int cv0 = c * L.vc, kc = V - cv0 < L.vc ? V - cv0 : L.vc;  // the chunk's vocabulary rows
    BwdParams p{};
    p.N = N;
    p.V = V;
    p.D = D;
    p.v_base = cv0;
    p.v_end = cv0 + kc;
    long long cost = 0;
    p.tile_units = dz_tile_units(N, kc, D, slots, pair, &cost);
    p.boxes = Boxes{p.tile_units, 0, token_rows(N), 1};
    CUtensorMap tW;
    if (!tmap_bf16_2d_sw128(&tW, head, D, V, p.tile_units * kUnit / (pair ? 2 : 1))) return cudaErrorInvalidValue;
    p.first = c == 0;
    p.sl2 = kLog2e / temperature;
    p.inv_t = 1.f / temperature;
    p.targets = targets;
    p.lse = lse;
    p.entropy = entropy;
    p.g_logp = g_logp;
    p.g_entropy = g_entropy;
    p.dz = dz;
    p.ld_dz = L.vc;
    p.dzt = dhead ? dzt : nullptr;
    p.ld_dzt = L.ld_dzt;
    p.status = status;
    const int units = (kc + kUnit - 1) / kUnit;
    const long long pairs = (long long)TM * ((units + p.tile_units - 1) / p.tile_units);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((pairs < slots ? (int)pairs : slots) * (pair ? 2 : 1));
    cfg.blockDim = dim3(kDzThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = pair ? attrs : attrs + 1;
    cfg.numAttrs = (pair ? 1 : 0) + (c == 0 ? 0 : 1);
    if ((e = cudaLaunchKernelEx(&cfg, kfn, tH, tW, p)) != cudaSuccess) return e;
    // dW rows of the chunk = dz^T H (the tokens are the contraction)
    if (dhead) {
      CUtensorMap tA, tLo;
      if (!tmap_bf16_2d_sw128_pitch(&tA, dzt, N, kc, L.ld_dzt, 128) ||
          (L.terms > 1 && !tmap_bf16_2d_sw128_pitch(&tLo, dzt + (size_t)L.vc * L.ld_dzt, N, kc, L.ld_dzt, 128)))
        return cudaErrorInvalidValue;
      GemmCall gc{};
      gc.lo = L.terms > 1 ? &tLo : nullptr;
      gc.stay = L.terms > 1;
      gc.M = kc;
      gc.N = D;
      gc.K = N;
      gc.mode = L.splits_w > 1 ? kAccInit : kStoreBf16;
      gc.splits = L.splits_w;
      gc.c = static_cast<__nv_bfloat16*>(dhead) + (size_t)cv0 * D;
      gc.acc = reinterpret_cast<float*>(w + L.acc_w);
      gc.status = status;
      gc.order = kAfter;
      gc.sms = apart ? sms - apart : 0;
      if ((e = launch_gemm(tA, tHb, gc, st)) != cudaSuccess) return e;
    }
    // dH += dz W[chunk] (the chunk's vocabulary rows are the contraction),
    // the contraction cut into `splits` runs with an accumulator each
    CUtensorMap tA, tLo, tB;
    if (!tmap_bf16_2d_sw128_pitch(&tA, dz, kc, N, L.vc, 128) ||
        (L.terms > 1 && !tmap_bf16_2d_sw128_pitch(&tLo, dz + (size_t)N * L.vc, kc, N, L.vc, 128)) ||
        !tmap_bf16_2d_sw128(&tB, static_cast<const __nv_bfloat16*>(head) + (size_t)cv0 * D, D, kc, 64))
      return cudaErrorInvalidValue;
    GemmCall gc{};
    gc.lo = L.terms > 1 ? &tLo : nullptr;
    gc.M = N;
    gc.N = D;
    gc.K = kc;
    gc.splits = splits;
    gc.sms = apart;
    if (splits > 1)
      gc.mode = c == 0 ? kAccInit : kAccAdd;
    else
      gc.mode = L.chunks == 1 ? kStoreBf16 : c == 0 ? kAccInit : c == L.chunks - 1 ? kAccFinal : kAccAdd;
    gc.c = static_cast<__nv_bfloat16*>(dhidden);
    gc.acc = acc;
    gc.status = status;
    gc.order = dhead ? kBeside : kAfter;
    if ((e = launch_gemm(tA, tB, gc, st)) != cudaSuccess) return e;
    // behind dH, which ends no earlier than dW
    if (dhead && L.splits_w > 1 &&
        (e = launch_sum_splits(reinterpret_cast<float*>(w + L.acc_w), L.splits_w, (size_t)kc * D,
                               static_cast<__nv_bfloat16*>(dhead) + (size_t)cv0 * D, st)) != cudaSuccess)
      return e;
  }
  if (splits > 1) return launch_sum_splits(acc, splits, (size_t)N * D, static_cast<__nv_bfloat16*>(dhidden), st);
  return cudaSuccess;
}

}  // namespace pa
