// paged.cu -- attention of a step's new tokens over a paged cache, for sm_103a.
//
// Rows. A tile has the TQ = 128 / G new tokens (rounded down) of one sequence times
// the G query heads of one kv head: row r is token r / G, head r % G, which is the
// order in which one TMA box {64, G, TQ} brings q. So keys and values are read once
// for all heads that share them, a single token fills G rows, and a long chunk
// fills 128. An item is (sequence, tile, kv head); a visit is 128 of its keys.
//
// Work. What there is to do is known on the device only (a step's lengths change
// while it is replayed from a graph), and it is dealt out evenly: every item has
// a cost (its keys and a fixed part), the costs of a step lie one behind the other on a
// line, and CTA c of P takes the line from W c / P to W (c + 1) / P. A CTA finds its
// ends by a scan over the sequences and a search in one of them, and walks the items
// between. An item that an end cuts leaves partial results (maximum, sums, O
// unnormalised) in the workspace, at most two a CTA; a second kernel joins them. So
// one long context spreads over all SMs as evenly as many short ones.
//
// Visits. As in fwd.cu: S = Q K^T into one of two TMEM buffers, softmax in two
// warpgroups that take the visits in turn (one thread a row), P from TMEM, O += P V in
// TMEM, lazy rescaling. The pipeline runs on from item to item: the next item's K and V are
// loaded, and its S formed, while the last one's O is written. Pages arrive by TMA, one
// box per page and 64 columns, a lane each, the page numbers loaded a visit ahead. Rows
// past a sequence's tokens and pages that are not there are masked in S; their rows of
// V are set to zero in shared memory before the product, because 0 * NaN is NaN.
//
// Warp roles: 0 Q and K producer, 1 V producer, 2 S issuer and TMEM owner, 3 PV
// issuer, 4..7 and 8..11 the softmax groups.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "sm103.cuh"
#include "softmax.cuh"
#include "tmap.h"

namespace pa {
namespace {

constexpr int kCtas = 160;       // at most; the workspace's layout has room for as many
constexpr int kThreads = 384;
// Cost of an item besides its keys, in keys: what Q's load, the pipeline's turn and the
// epilogue take.
constexpr int kItemCost = 256;
constexpr int kLeastVisits = 2;  // of a part of an item
constexpr int kLeastCost = 512;  // of a CTA

template <int D>
struct Layout {
  static constexpr int DL = D == 64 ? 64 : 128;  // columns of a tile in shared memory
  static constexpr int NC = DL / 64;             // 64-column chunks
  static constexpr int NSK = 3, NSV = 2;
  static constexpr uint32_t CHUNK = 128 * 128;
  static constexpr uint32_t TB = NC * CHUNK;
  static constexpr uint32_t OFF_K = TB, OFF_V = OFF_K + NSK * TB;
  static constexpr uint32_t MISC = 8192;
  static constexpr uint32_t SMEM = OFF_V + NSV * TB + MISC + 1024;
  static constexpr uint32_t TM_O = 0, TM_S = 128, TM_P = 384, TMEM_COLS = 512;
};

// A place on the line of work: before visit kt of item (s, i, h), of nkt visits.
struct Bound {
  int s, i, h, kt, nkt;
};

struct Misc {
  uint64_t q_full, q_free, k_full[3], k_empty[3], v_full[2], v_empty[2];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], mh_full[2][4], sums_full, o_free, fin_s, fin_pv;
  uint32_t tmem_base;
  int abort_flag;
  Bound ends[2];
  long long scan[kThreads / 32];
  float mh[2][128];          // [visit parity][row]: row maximum in use after the visit
  float sums[2][2][2][128];  // [item parity][group][l, lr][row]
};

// Partial results of a CTA: slot 0 of the item that its run begins inside of, slot 1 of
// the one that it ends inside of. O as float4 of row r, columns 4c .. 4c + 3 at [c][r].
struct Partial {
  float m[128], l[128], lr[128];
};
__host__ __device__ constexpr size_t partial_bytes(int D) { return sizeof(Partial) + (size_t)128 * D * 4; }
constexpr size_t kOffRecords = 256, kOffPartials = kOffRecords + kCtas * sizeof(int4);

// What a CTA left: the item that it began and did not end, if any (s, i, h, else s = -1),
// and what its run begins with.
enum Head : int { kWhole = 0, kGoesOn = 1, kEnds = 2, kEmpty = 3 };

struct FwdArgs {
  PagedArgs p;
  int TQ, page_shift;
  __nv_bfloat16* out;
  float* lse;
  uint8_t* ws;
};

__device__ __forceinline__ int tiles_of(const FwdArgs& a, int ql) { return (ql + a.TQ - 1) / a.TQ; }
// Visits of tile i of a sequence's tiles: the keys that its last token sees.
__device__ __forceinline__ int visits_of(const FwdArgs& a, const SeqRows& r, int i) {
  const int ql = r.b - r.a, e = min(r.base() + min(ql, (i + 1) * a.TQ), a.p.width * a.p.page);
  return e <= kTile ? 1 : (e + kTile - 1) / kTile;
}
// Costs of a sequence's items of one kv head: tile i's and all before it.
struct Costs {
  long long A;
  int ql, n, TQ;
  __device__ __forceinline__ Costs(const FwdArgs& a, const SeqRows& r) {
    ql = r.b - r.a;
    n = tiles_of(a, ql);
    TQ = a.TQ;
    A = (long long)min(max(r.base(), 0), a.p.width * a.p.page) + kItemCost;
  }
  __device__ __forceinline__ long long before(int i) const { return A * i + (long long)TQ * i * (i + 1) / 2; }
  __device__ __forceinline__ long long of(int i) const { return A + (i == n - 1 ? ql : TQ * (i + 1)); }
  __device__ __forceinline__ long long all() const { return n ? before(n - 1) + of(n - 1) : 0; }
};

// Where `x` of sequence s's cost lies. A cut that would leave fewer than kLeastVisits on
// one of its sides moves to the item's end on that side.
__device__ Bound place(const FwdArgs& a, int s, long long x) {
  const SeqRows r = seq_rows(a.p, s);
  const Costs c(a, r);
  const int H = a.p.Hkv;
  int i = 0;
  for (int hi = c.n; hi - i > 1;) {
    const int mid = i + (hi - i) / 2;
    if (c.before(mid) * H <= x)
      i = mid;
    else
      hi = mid;
  }
  x -= c.before(i) * H;
  const long long of = c.of(i);
  Bound b;
  b.s = s;
  b.i = i;
  b.h = (int)min(x / of, (long long)H - 1);
  b.nkt = visits_of(a, r, i);
  b.kt = (int)min((x - b.h * of) * b.nkt / of, (long long)b.nkt - 1);
  if (b.kt < kLeastVisits)
    b.kt = 0;
  else if (b.nkt - b.kt < kLeastVisits)
    b.kt = b.nkt;
  return b;
}

// Both ends of this CTA's run, by all threads.
__device__ void find_ends(const FwdArgs& a, Misc& m) {
  const int S = a.p.S, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long total = 0, x[2] = {0, 0};
  for (int pass = 0; pass < 2; ++pass) {  // the sum, then the places in it
    long long run = 0;
    for (int s0 = 0; s0 < S; s0 += kThreads) {
      const int s = s0 + tid;
      long long mine = 0;
      if (s < S) mine = Costs(a, seq_rows(a.p, s)).all() * a.p.Hkv;
      long long v = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
      }
      if (lane == 31) m.scan[warp] = v;
      __syncthreads();
      long long before = run;
      for (int w = 0; w < kThreads / 32; ++w) {
        const long long u = m.scan[w];
        if (w < warp) before += u;
        run += u;
      }
      v += before;  // inclusive
      if (S <= kThreads) {  // everything is here already: no second pass over memory
        total = run;
        pass = 1;
      }
      if (pass == 1) {
        if (s0 == 0) {
          const long long P = max(1ll, min((long long)gridDim.x, total / kLeastCost)), per = total / P, rest = total % P;
          for (int e = 0; e < 2; ++e) {
            const long long c = min((long long)blockIdx.x + e, P);
            x[e] = per * c + rest * c / P;
          }
        }
        for (int e = 0; e < 2; ++e)
          if (mine > 0 && x[e] >= v - mine && x[e] < v) m.ends[e] = place(a, s, x[e] - (v - mine));
      }
      __syncthreads();
    }
    total = run;
  }
}

// The parts of items in a CTA's run, in order.
struct Walk {
  const FwdArgs& a;
  Bound at, end;
  SeqRows r;
  int n;         // tiles of the sequence
  int kt0, kt1;  // visits of this part
  __device__ __forceinline__ Walk(const FwdArgs& a_, const Misc& m) : a(a_), at(m.ends[0]), end(m.ends[1]) {
    r.a = r.b = r.kv = n = 0;
    if (at.s < a.p.S) load();
    kt0 = kt1 = 0;
    first = true;
  }
  // To the next part; false when there is none.
  __device__ __forceinline__ bool next() {
    for (;;) {
      if (!first) step();
      if (at.s >= a.p.S || (at.s == end.s && at.i == end.i && at.h == end.h && end.kt == 0) || past()) return false;
      kt0 = first ? at.kt : 0;
      first = false;
      at.nkt = visits_of(a, r, at.i);
      const bool last = at.s == end.s && at.i == end.i && at.h == end.h;
      kt1 = last ? end.kt : at.nkt;
      if (last) end.s = -1;  // nothing behind this one
      if (kt0 < kt1) return true;
    }
  }
  __device__ __forceinline__ int nkt() const { return at.nkt; }
  __device__ __forceinline__ int row0() const { return r.a + at.i * a.TQ; }                      // the tile's first row of q
  __device__ __forceinline__ int tokens() const { return min(a.TQ, r.b - r.a - at.i * a.TQ); }  // and its tokens
  __device__ __forceinline__ int first_seen() const { return r.base() + at.i * a.TQ + 1; }      // keys that its first one sees
  __device__ __forceinline__ int cap() const { return min(r.kv, a.p.width * a.p.page); }        // keys in the cache

 private:
  bool first;
  __device__ __forceinline__ bool past() const { return end.s < 0; }
  __device__ __forceinline__ void load() {
    r = seq_rows(a.p, at.s);
    n = tiles_of(a, r.b - r.a);
  }
  __device__ __forceinline__ void step() {
    if (++at.h < a.p.Hkv) return;
    at.h = 0;
    if (++at.i < n) return;
    at.i = 0;
    for (++at.s; at.s < a.p.S; ++at.s) {
      load();
      if (n > 0) return;
    }
  }
};

// A lane's page of visit kt: its number, or -1 (not there, or past the sequence's keys).
__device__ __forceinline__ int page_of(const FwdArgs& a, int s, int kt, int cap, int lane, int per) {
  const int key = kt * kTile + lane * a.p.page;
  if (lane >= per || key >= cap) return -1;
  const int id = __ldg(a.p.page_table + (int64_t)s * a.p.width + (key >> a.page_shift));
  return id >= 0 && id < a.p.pages ? id : -1;
}
// Pages of visit kt within the sequence's keys that are not in the cache, a bit each.
__device__ __forceinline__ uint32_t missing(const FwdArgs& a, int id, int kt, int cap, int lane, int per) {
  return __ballot_sync(~0u, lane < per && kt * kTile + lane * a.p.page < cap && id < 0);
}

// Keys k0 .. k0+31 that a row with `seen` keys does not see, and those of missing
// pages (bits of 16 keys: the low one for the first 16), out of its scores.
__device__ __forceinline__ void hide32(uint32_t (&x)[32], int k0, int seen, uint32_t bad) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    x[c] = (k0 + c < seen && !((c < 16 ? bad : bad >> 1) & 1)) ? x[c] : __float_as_uint(-INFINITY);
}
// The missing pages' bits as bits of 16 keys each.
__device__ __forceinline__ uint32_t by16(uint32_t bad, int page_shift) {
  uint32_t r = 0;
  for (int e = 0; e < 8; ++e) r |= ((bad >> ((e * 16) >> page_shift)) & 1u) << e;
  return r;
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2, int c3) {
  tma_load_bhnd(dst, m, bar, c0, c1, c2, c3);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ FwdArgs a) {
  using L = Layout<D>;
  constexpr int NSK = L::NSK, NSV = L::NSV, NC = L::NC;
  static_assert(sizeof(Misc) <= L::MISC, "misc region");
  static_assert(L::SMEM <= 232448, "shared memory");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Misc& m = *reinterpret_cast<Misc*>(smem_raw);
  uint8_t* base =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + sizeof(Misc) + 1023) & ~uintptr_t(1023));
  uint8_t *bK = base + L::OFF_K, *bV = base + L::OFF_V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* status = reinterpret_cast<uint32_t*>(a.ws);
  const Guard g{&m.abort_flag, status};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) *status = 0;
    m.abort_flag = 0;
    mbar_init(&m.q_full, 1);
    mbar_init(&m.q_free, 1);
    for (int s = 0; s < NSK; ++s) {
      mbar_init(&m.k_full[s], 1);
      mbar_init(&m.k_empty[s], 1);
    }
    for (int s = 0; s < NSV; ++s) {
      mbar_init(&m.v_full[s], 1);
      mbar_init(&m.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&m.s_full[s], 1);
      mbar_init(&m.s_free[s], 4);  // the four warps of the group that owns the visit
      mbar_init(&m.p_full[s], 4);
      mbar_init(&m.pv_done[s], 1);
      for (int q = 0; q < 4; ++q) mbar_init(&m.mh_full[s][q], 1);
    }
    mbar_init(&m.sums_full, 8);
    mbar_init(&m.o_free, 8);
    mbar_init(&m.fin_s, 1);
    mbar_init(&m.fin_pv, 1);
    fence_mbar_init();
    m.ends[0] = m.ends[1] = Bound{a.p.S, 0, 0, 0, 0};
  }
  if (warp == 2) {
    tmem_alloc(&m.tmem_base, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem_base;
  find_ends(a, m);

  const int per = a.p.page >= kTile ? 1 : kTile / a.p.page;  // pages of a visit
  const int box = min(a.p.page, kTile);                      // and the rows of one
  Walk w(a, m);
  if (warp == 0) {
    // ------------------------------------------------------ Q and K producer
    if (lane == 0) {  // what the second kernel has to know
      const Bound b = m.ends[0], e = m.ends[1];
      const bool same = b.s == e.s && b.i == e.i && b.h == e.h;
      const bool inside = b.kt > 0 && b.kt < b.nkt;
      int4 rec = make_int4(-1, 0, 0, kWhole);
      if (inside) rec.w = !same ? kEnds : e.kt == b.kt ? kEmpty : e.kt == e.nkt ? kEnds : kGoesOn;
      if (e.kt > 0 && e.kt < e.nkt && !(same && b.kt > 0)) rec = make_int4(e.s, e.i, e.h, rec.w);
      reinterpret_cast<int4*>(a.ws + kOffRecords)[blockIdx.x] = rec;
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
    }
    __syncwarp();
    const int pl = lane % per, ch = lane / per;
    const int mine = ch < NC ? pl : per;  // this lane's page of a visit
    int vc = 0, items = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int cap = w.cap();
      int id = page_of(a, w.at.s, w.kt0, cap, mine, per);
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++vc) {
        const int now = id, sk = vc % NSK;
        if (kt + 1 < w.kt1) id = page_of(a, w.at.s, kt + 1, cap, mine, per);
        const uint32_t boxes = __popc(__ballot_sync(~0u, now >= 0));
        if (!g.wait_warp(&m.k_empty[sk], ((vc / NSK) & 1) ^ 1, 1)) { ok = false; break; }
        if (lane == 0) mbar_expect_tx(&m.k_full[sk], boxes * box * 128);
        __syncwarp();
        if (now >= 0)
          tma_load_4d(bK + sk * L::TB + ch * L::CHUNK + pl * box * 128, &tmK, &m.k_full[sk], ch * 64,
                      (kt * kTile) & (a.p.page - 1) & ~(kTile - 1), w.at.h, now);
        if (kt == w.kt0) {  // Q once the last item's S products have read theirs
          if (items > 0 && !g.wait_warp(&m.q_free, (items - 1) & 1, 2)) { ok = false; break; }
          if (lane == 0) {
            mbar_expect_tx(&m.q_full, NC * a.TQ * a.p.G * 128);
            for (int c = 0; c < NC; ++c)
              tma_load_4d(base + c * L::CHUNK, &tmQ, &m.q_full, c * 64, 0, w.row0(), w.at.h);
          }
          __syncwarp();
          ++items;
        }
      }
    }
    if (lane == 0) {  // no copy may still be landing when the CTA exits
      if (items > 0) g.drain(&m.q_full, (items - 1) & 1);
      for (int i = (vc > NSK ? vc - NSK : 0); i < vc; ++i) g.drain(&m.k_full[i % NSK], (i / NSK) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ V producer
    if (lane == 0) prefetch_tmap(&tmV);
    const int pl = lane % per, ch = lane / per;
    const int mine = ch < NC ? pl : per;
    int vc = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int cap = w.cap();
      int id = page_of(a, w.at.s, w.kt0, cap, mine, per);
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++vc) {
        const int now = id, sv = vc % NSV;
        if (kt + 1 < w.kt1) id = page_of(a, w.at.s, kt + 1, cap, mine, per);
        const uint32_t boxes = __popc(__ballot_sync(~0u, now >= 0));
        if (!g.wait_warp(&m.v_empty[sv], ((vc / NSV) & 1) ^ 1, 3)) { ok = false; break; }
        if (lane == 0) mbar_expect_tx(&m.v_full[sv], boxes * box * 128);
        __syncwarp();
        if (now >= 0)
          tma_load_4d(bV + sv * L::TB + ch * L::CHUNK + pl * box * 128, &tmV, &m.v_full[sv], ch * 64,
                      (kt * kTile) & (a.p.page - 1) & ~(kTile - 1), w.at.h, now);
      }
    }
    if (lane == 0)
      for (int i = (vc > NSV ? vc - NSV : 0); i < vc; ++i) g.drain(&m.v_full[i % NSV], (i / NSV) & 1);
    __syncwarp();
  } else if (warp == 2) {
    // -------------------------------------------------------------- S issuer
    const bool leader = lane == 0;
    constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false);
    const uint64_t qd = sdesc_sw128(smem_u32(base), 16, 1024);
    int vc = 0, items = 0;
    bool ok = true;
    while (ok && w.next()) {
      if (!g.wait_warp(&m.q_full, items & 1, 4)) { ok = false; break; }
      ++items;
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++vc) {
        const int sb = vc & 1, sk = vc % NSK;
        if (vc >= 2 && !g.wait_warp(&m.s_free[sb], ((vc - 2) >> 1) & 1, 5)) { ok = false; break; }
        if (!g.wait_warp(&m.k_full[sk], (vc / NSK) & 1, 6)) { ok = false; break; }
        tc_fence_after();
        const uint64_t kd = sdesc_sw128(smem_u32(bK + sk * L::TB), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ko = (kk >> 2) * L::CHUNK + (kk & 3) * 32;
          if (leader) umma_bf16(tmem + L::TM_S + sb * 128, sdesc_add(qd, ko), sdesc_add(kd, ko), idS, kk > 0 ? 1u : 0u);
        }
        if (leader) {
          umma_commit(&m.s_full[sb]);
          umma_commit(&m.k_empty[sk]);
          if (kt + 1 == w.kt1) umma_commit(&m.q_free);
        }
        __syncwarp();
      }
    }
    if (leader) {
      umma_commit(&m.fin_s);
      g.drain(&m.fin_s, 0);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------- PV issuer
    const bool leader = lane == 0;
    constexpr uint32_t idO = idesc_bf16_f32(128, D, false, true);
    int vc = 0, items = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int cap = w.cap();
      int id = page_of(a, w.at.s, w.kt0, cap, lane, per);
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++vc) {
        const int now = id, sb = vc & 1, sv = vc % NSV;
        if (kt + 1 < w.kt1) id = page_of(a, w.at.s, kt + 1, cap, lane, per);
        const uint32_t bad = missing(a, now, kt, cap, lane, per);
        if (!g.wait_warp(&m.v_full[sv], (vc / NSV) & 1, 7)) { ok = false; break; }
        const int there = cap - kt * kTile;  // rows of this visit that hold keys
        if (bad || there < kTile) {
          // zeros where there are none: eight lanes a row of 128 bytes
          for (int r = lane >> 3; r < kTile; r += 4)
            if (r >= there || (bad >> (r >> a.page_shift)) & 1)
              for (int c = 0; c < NC; ++c)
                st_shared_v4(smem_u32(bV + sv * L::TB + c * L::CHUNK + r * 128 + (lane & 7) * 16), 0, 0, 0, 0);
          fence_async_smem();
          __syncwarp();
        }
        if (kt == w.kt0) {  // O is free once the last item's has been read
          if (items > 0 && !g.wait_warp(&m.o_free, (items - 1) & 1, 8)) { ok = false; break; }
          ++items;
        }
        if (!g.wait_warp(&m.p_full[sb], (vc >> 1) & 1, 9)) { ok = false; break; }
        tc_fence_after();
        const uint64_t vd = sdesc_sw128(smem_u32(bV + sv * L::TB), L::CHUNK, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (leader)
            umma_bf16_ta(tmem + L::TM_O, tmem + L::TM_P + sb * 64 + kk * 8, sdesc_add(vd, kk * 2048), idO,
                         (kt > w.kt0 || kk > 0) ? 1u : 0u);
        if (leader) {
          umma_commit(&m.pv_done[sb]);
          umma_commit(&m.v_empty[sv]);
        }
        __syncwarp();
      }
    }
    if (leader) {
      umma_commit(&m.fin_pv);
      g.drain(&m.fin_pv, 0);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    const int grp = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int tok = r / a.p.G, gh = r - tok * a.p.G;
    const int warp_tok = (quarter * 32) / a.p.G;  // the token of the warp's first row
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_base + L::TM_O;
    const float sl2 = a.p.scale_log2;
    int vc = 0, items = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int cap = w.cap(), first_seen = min(w.first_seen(), cap), nt = w.tokens();
      const int seen = min(w.first_seen() + tok, cap);
      const bool active = warp_tok < nt;  // some row of this warp is a token's
      float m_w = -INFINITY;              // the maximum this group's sums are taken against
      uint64_t l2 = 0ull, lr2 = 0ull;     // exact and bf16-rounded weight sums
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++vc) {
        if ((vc & 1) != grp) continue;
        const int id = page_of(a, w.at.s, kt, cap, lane, per);
        ok = g.wait_warp(&m.s_full[grp], (vc >> 1) & 1, 10);
        if (!ok) break;
        if (!active) {  // in step with the others, nothing to do
          warp_arrive(&m.s_free[grp], lane);
          warp_arrive(&m.mh_full[grp][quarter], lane);
          if (vc >= 2 && !(ok = g.wait_warp(&m.pv_done[grp], ((vc - 2) >> 1) & 1, 11))) break;
          warp_arrive(&m.p_full[grp], lane);
          continue;
        }
        tc_fence_after();
        uint32_t x0[32], x1[32], x2[32], x3[32];
        tmem_ld128(tmem + lane_base + L::TM_S + grp * 128, x0, x1, x2, x3);
        tc_fence_before();
        warp_arrive(&m.s_free[grp], lane);
        const uint32_t bad = missing(a, id, kt, cap, lane, per);
        const bool masked = bad || (kt + 1) * kTile > first_seen;
        if (masked) {
          const uint32_t b16 = by16(bad, a.page_shift);
          const int k0 = kt * kTile;
          hide32(x0, k0, seen, b16);
          hide32(x1, k0 + 32, seen, b16 >> 2);
          hide32(x2, k0 + 64, seen, b16 >> 4);
          hide32(x3, k0 + 96, seen, b16 >> 6);
        }
        const float ms = fmax3(fmaxf(max32(x0), max32(x1)), max32(x2), max32(x3)) * sl2;
        float m_prev = -INFINITY;
        if (kt > w.kt0) {  // the maximum in use after the previous visit, from the other group
          ok = g.wait_warp(&m.mh_full[grp ^ 1][quarter], ((vc - 1) >> 1) & 1, 12);
          if (!ok) break;
          m_prev = m.mh[grp ^ 1][r];
        }
        const bool rescale = __any_sync(~0u, ms > m_prev + 8.f);
        const float m_new = rescale ? fmaxf(m_prev, ms) : m_prev;
        m.mh[grp][r] = m_new;
        warp_arrive(&m.mh_full[grp][quarter], lane);
        if (m_w != m_new) {
          const float f = (m_w == -INFINITY) ? 0.f : ex2(m_w - m_new);
          l2 = mul2(l2, f2(f, f));
          lr2 = mul2(lr2, f2(f, f));
          m_w = m_new;
        }
        const float moff = (m_new == -INFINITY) ? 0.f : m_new;
        const uint64_t sc = f2(sl2, sl2), off = f2(-moff, -moff);
        const uint32_t tP = tmem + lane_base + L::TM_P + grp * 64;
        if (vc >= 2) {
          ok = g.wait_warp(&m.pv_done[grp], ((vc - 2) >> 1) & 1, 13);
          if (!ok) break;
          tc_fence_after();
        }
        uint64_t t2 = 0ull, tr2 = 0ull;
        // O's normaliser takes the rounded weights where a row may have few keys, see fwd.cu
        if (masked) {
          exp_store32<true>(x0, sc, off, tP, t2, tr2);
          exp_store32<true>(x1, sc, off, tP + 16, t2, tr2);
          exp_store32<true>(x2, sc, off, tP + 32, t2, tr2);
          exp_store32<true>(x3, sc, off, tP + 48, t2, tr2);
        } else {
          exp_store32<false>(x0, sc, off, tP, t2, tr2);
          exp_store32<false>(x1, sc, off, tP + 16, t2, tr2);
          exp_store32<false>(x2, sc, off, tP + 32, t2, tr2);
          exp_store32<false>(x3, sc, off, tP + 48, t2, tr2);
          tr2 = t2;
        }
        l2 = add2(l2, t2);
        lr2 = add2(lr2, tr2);
        if (rescale && kt > w.kt0) {  // O holds earlier visits: rescale it once their PV is done
          const float alpha = (m_prev == -INFINITY) ? 0.f : ex2(m_prev - m_new);
          ok = g.wait_warp(&m.pv_done[grp ^ 1], ((vc - 1) >> 1) & 1, 14);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(tO + c0, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
            tmem_st32(tO + c0, v);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&m.p_full[grp], lane);
      }
      if (!ok) break;
      // -------------------------------------------------------------- epilogue
      // The final maximum is the one the last visit's group handed on; both groups take
      // their sums to it, add them up and write half of O each.
      const int last = vc - 1, ip = items & 1;
      ok = g.wait_warp(&m.mh_full[last & 1][quarter], (last >> 1) & 1, 15);
      if (!ok) break;
      const float m_fin = active ? m.mh[last & 1][r] : -INFINITY;
      const float f = (m_w == m_fin) ? 1.f : (m_w == -INFINITY ? 0.f : ex2(m_w - m_fin));
      const float2 lp = f2_split(l2), lrp = f2_split(lr2);
      m.sums[ip][grp][0][r] = (lp.x + lp.y) * f;
      m.sums[ip][grp][1][r] = (lrp.x + lrp.y) * f;
      warp_arrive(&m.sums_full, lane);
      ok = g.wait_warp(&m.sums_full, items & 1, 16) && g.wait_warp(&m.pv_done[last & 1], (last >> 1) & 1, 17);
      if (!ok) break;
      ++items;
      tc_fence_after();
      // both groups add the two groups' sums in the same order
      const float lt = m.sums[ip][0][0][r] + m.sums[ip][1][0][r], lrt = m.sums[ip][0][1][r] + m.sums[ip][1][1][r];
      const bool whole = w.kt0 == 0 && w.kt1 == w.nkt();
      const bool mine = tok < nt;
      const int c_lo = grp * (L::DL / 2), c_hi = min(c_lo + L::DL / 2, D);
      if (active) {
        const float inv = lrt > 0.f ? 1.f / lrt : 0.f;
        const int64_t row = w.row0() + tok;
        const int head = w.at.h * a.p.G + gh;
        __nv_bfloat16* po = a.out + row * a.p.o_t + (int64_t)head * a.p.o_h;
        uint8_t* slot = a.ws + kOffPartials + ((size_t)blockIdx.x * 2 + (w.kt0 == 0 ? 1 : 0)) * partial_bytes(D);
        float4* part = reinterpret_cast<float4*>(slot + sizeof(Partial));
#pragma unroll 1
        for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(tO + c0, v);
          if (mine && whole) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4 y;
              y.x = pack_bf16x2(__uint_as_float(v[q * 8 + 0]) * inv, __uint_as_float(v[q * 8 + 1]) * inv);
              y.y = pack_bf16x2(__uint_as_float(v[q * 8 + 2]) * inv, __uint_as_float(v[q * 8 + 3]) * inv);
              y.z = pack_bf16x2(__uint_as_float(v[q * 8 + 4]) * inv, __uint_as_float(v[q * 8 + 5]) * inv);
              y.w = pack_bf16x2(__uint_as_float(v[q * 8 + 6]) * inv, __uint_as_float(v[q * 8 + 7]) * inv);
              *reinterpret_cast<uint4*>(po + c0 + q * 8) = y;
            }
          } else if (mine) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              part[(size_t)(c0 / 4 + q) * 128 + r] =
                  make_float4(__uint_as_float(v[q * 4]), __uint_as_float(v[q * 4 + 1]), __uint_as_float(v[q * 4 + 2]),
                              __uint_as_float(v[q * 4 + 3]));
          }
          __syncwarp();
        }
        if (mine && grp == 0) {
          if (whole) {
            a.lse[row * a.p.Hq + head] = m_fin * 0.6931471805599453f + logf(lt);
          } else {
            Partial& pt = *reinterpret_cast<Partial*>(slot);
            pt.m[r] = m_fin;
            pt.l[r] = lt;
            pt.lr[r] = lrt;
          }
        }
      }
      tc_fence_before();
      warp_arrive(&m.o_free, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// Joins the parts of the item that CTA blockIdx.x began and did not end.
template <int D>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ FwdArgs a) {
  __shared__ int heads[kCtas];
  __shared__ int slots[kCtas];
  __shared__ int count;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4* recs = reinterpret_cast<const int4*>(a.ws + kOffRecords);
  const int4 rec = recs[blockIdx.x];
  if (rec.x < 0) return;
  const int P = gridDim.x;
  for (int c = blockIdx.x + 1 + threadIdx.x; c < P; c += 256) heads[c] = recs[c].w;
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    slots[n++] = blockIdx.x * 2 + 1;
    for (int c = blockIdx.x + 1; c < P; ++c) {
      if (heads[c] != kEmpty) slots[n++] = c * 2;
      if (heads[c] != kGoesOn && heads[c] != kEmpty) break;
    }
    count = n;
  }
  __syncthreads();
  const SeqRows r = seq_rows(a.p, rec.x);
  const int row0 = r.a + rec.y * a.TQ, nt = min(a.TQ, r.b - row0), rows = nt * a.p.G, n = count;
  const uint8_t* parts = a.ws + kOffPartials;
  for (int e = blockIdx.y * 256 + threadIdx.x; e < rows * (D / 4); e += gridDim.y * 256) {
    const int c = e / rows, row = e - c * rows;
    float M = -INFINITY;
    for (int k = 0; k < n; ++k) M = fmaxf(M, reinterpret_cast<const Partial*>(parts + slots[k] * partial_bytes(D))->m[row]);
    float l = 0.f, lr = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < n; ++k) {
      const Partial& pt = *reinterpret_cast<const Partial*>(parts + slots[k] * partial_bytes(D));
      const float4 v = reinterpret_cast<const float4*>(&pt + 1)[(size_t)c * 128 + row];
      const float w = pt.m[row] == -INFINITY ? 0.f : ex2(pt.m[row] - M);
      l = fmaf(pt.l[row], w, l);
      lr = fmaf(pt.lr[row], w, lr);
      o.x = fmaf(v.x, w, o.x);
      o.y = fmaf(v.y, w, o.y);
      o.z = fmaf(v.z, w, o.z);
      o.w = fmaf(v.w, w, o.w);
    }
    const float inv = lr > 0.f ? 1.f / lr : 0.f;
    const int tok = row / a.p.G, head = rec.z * a.p.G + (row - tok * a.p.G);
    const int64_t at = row0 + tok;
    *reinterpret_cast<uint2*>(a.out + at * a.p.o_t + (int64_t)head * a.p.o_h + c * 4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (c == 0) a.lse[at * a.p.Hq + head] = M * 0.6931471805599453f + logf(l);
  }
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms <= 0)
    sms = 152;
  return sms;
}

template <int D>
cudaError_t launch_d(const FwdArgs& a, const void* q, const void* k_pages, const void* v_pages, cudaStream_t st) {
  using L = Layout<D>;
  const PagedArgs& p = a.p;
  CUtensorMap tq, tk, tv;
  const uint64_t qd[4] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)p.T, (uint64_t)p.Hkv};
  const int64_t qs[3] = {p.q_h, p.q_t, p.Hkv > 1 ? p.G * p.q_h : D};
  const uint32_t qbox[2] = {(uint32_t)p.G, (uint32_t)a.TQ};
  const uint64_t kd[4] = {(uint64_t)D, (uint64_t)p.page, (uint64_t)p.Hkv, (uint64_t)p.pages};
  const int64_t ks[3] = {p.p_n, p.p_h, p.p_p};
  const uint32_t kbox[2] = {(uint32_t)std::min(p.page, kTile), 1};
  if (!tmap_bf16_4d_sw128(&tq, q, qd, qs, qbox) || !tmap_bf16_4d_sw128(&tk, k_pages, kd, ks, kbox) ||
      !tmap_bf16_4d_sw128(&tv, v_pages, kd, ks, kbox))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(paged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(sm_count(), kCtas);
  paged_kernel<D><<<ctas, kThreads, L::SMEM, st>>>(tq, tk, tv, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, 4);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr = programmatic_launch();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, a);
}

}  // namespace

size_t paged_ws_bytes(int D) { return kOffPartials + 2 * kCtas * partial_bytes(D); }

cudaError_t launch_paged_fwd(const PagedArgs& p, const void* q, const void* k_pages, const void* v_pages, void* out, float* lse,
                             void* ws, cudaStream_t st) {
  FwdArgs a{};
  a.p = p;
  a.TQ = kTile / p.G;
  while ((1 << a.page_shift) < p.page) ++a.page_shift;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.ws = static_cast<uint8_t*>(ws);
  if (p.D == 64) return launch_d<64>(a, q, k_pages, v_pages, st);
  if (p.D == 96) return launch_d<96>(a, q, k_pages, v_pages, st);
  return launch_d<128>(a, q, k_pages, v_pages, st);
}

}  // namespace pa
