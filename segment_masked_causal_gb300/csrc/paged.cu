// paged.cu -- attention of a step's new tokens over a paged cache, for sm_103a.
//
// Rows. A tile is floor(128 / G) new tokens of one sequence times the G query heads of
// one kv head: row r is token r / G, head r % G, which is the order in which one TMA box
// {64, G, tokens} brings q. So keys and values are read once for all heads that share
// them, a single token fills G rows and a long chunk 128. An item is (sequence, two
// neighbouring tiles or what is left of them, kv head); a visit is 128 of its keys.
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
// Visits. Two streams, each with an S buffer and an O accumulator in TMEM and a softmax
// warpgroup, one thread a row: S = Q K^T, P = 2^(S log2e scale - m) as bf16 over S, O += P V
// with P from TMEM. While one stream is in its softmax, the tensor cores work for the
// other. An item of two tiles gives each stream a tile, and both take every visit (K and
// V are read from shared memory for 256 rows); an item of one tile has its visits dealt out to
// the streams in turn, whose sums and O are joined at its end, or, with few visits, goes whole to
// one of them. No stream ever waits for the other's maximum, and O is rescaled, lazily, between a
// stream's own products. P is rounded to bf16 because the matrix instruction takes its second
// product's two operands in one type and V is bf16; the sums below it are of the weights before that. So out is
// 2.0e-3 to 2.4e-3 of its norm off, of which its own rounding is 1.7e-3.
//
// Few rows. A TMEM lane belongs to one warp of four, so where an item has at most eight
// rows the tile holds them four times and each of a group's warps takes 32 of a visit's
// 128 keys (its P has zeros for the others); the four parts of a row are joined
// at the item's end as well (256 requests of 300 keys: 102 -> 82 us; 64 of up to 16,000: 89 -> 86). With
// more rows that join costs more than it saves (33 x 5 tokens: 41 us with up to 32 rows, 38 without).
//
// The pipeline runs on from item to item: the next item's Q, K and V are loaded while the
// last one's O is written. Pages arrive by TMA, one box per page and 64 columns, a lane
// each, the page numbers loaded a visit ahead. Rows past a sequence's tokens and pages
// that are not there are masked in S, and the second product leaves out the steps of 16
// keys without any; what is left of the last one's rows of V is set to zero.
//
// What bounds it. Tokens of one each: DRAM (64 requests of 4,000 keys, heads 32 on 8 of 128: 163 us,
// 0.95 of the copy bandwidth), below some 50 MB of keys the start of the pipeline, the last
// epilogue and the join (one token of 100 keys 8.8 us). Long chunks: the chain of a stream (S, softmax,
// PV and their hand-overs, 3,200 to 3,700 cycles a visit of both against 2,048 of tensor work; 8,192
// tokens of one prompt: 439 us, 0.64 of the matrix peak). One S buffer for both streams with P beside it takes PV
// out of that chain, but each S then waits for the other stream to load the last one (a chunk of 2,001
// beside 47 single tokens: 10 to 20% longer).
//
// Warp roles: 0 Q and K producer, 1 V producer, 2 S issuer and TMEM owner, 3 PV
// issuer, 4..7 and 8..11 the softmax groups of streams 0 and 1.
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

constexpr int kCtas = 160;  // at most; the workspace's layout has room for as many
constexpr int kThreads = 384;
// Cost of an item besides its keys, in keys: what Q's load, the pipeline's turn and the
// epilogue take; and of a key for two tiles. No more than a fit to the times of steps of several
// kinds: a chunk of 2,001 tokens beside 47 single ones takes 102 us
// with these, 111 with 448 and 1.4 for pairs, 103 with 900 and 2.2, 104 with 384 for single
// tiles; with 192 there 64 requests of up to 16,000 keys take 84.8 us instead of 83.5, and with 256
// 33 x 5 tokens 29.9 instead of 27.1.
constexpr int kItemCost = 320, kPairItemCost = 640;
constexpr float kPairCost = 1.8f;
// Visits of a part of an item: fewer are not worth a join (some 3 us, and the part's way through
// memory), which is not launched at all where the table holds less than two parts. Against three,
// over a table of 32,768 tokens: chunks of 1,500 tokens 25.0 -> 22.1 us, one token of 700 keys 14.5 -> 12.7, but
// 8 chunks of 512 42.7 -> 45.9 and a chunk of 2,001 beside 47 tokens 99 -> 102; without the join, over tables that
// just hold them, the first two take 19.9 and 11.8.
constexpr int kLeastVisits = 4;
constexpr int kLeastCost = 512;  // of a CTA; with 768 one token of 100 keys takes 10.6 us instead of 8.8
// Visits of an item of few rows that one stream takes alone, so that its epilogue runs beside the
// next item's visits (256 requests of 300 keys: 75.6 -> 71.9 us; with five visits 64
// requests of up to 16,000 keys lose 1%). More rows have longer visits, and take turns from two on
// (33 x 5 tokens: 30.6 us with three alone, 30.0 with one).
constexpr int kAlone = 3;
constexpr int kFew = 8;           // rows of an item that the tile holds four times, see above
constexpr int kStage = 2560;      // bytes of a softmax warp's staging buffer

template <int D>
struct Layout {
  static constexpr int DL = D == 64 ? 64 : 128;  // columns of a tile in shared memory
  static constexpr int NC = DL / 64;             // 64-column chunks
  static constexpr int NS = D == 64 ? 4 : 2;     // stages of K, and of V
  static constexpr uint32_t CHUNK = 128 * 128;
  static constexpr uint32_t TB = NC * CHUNK;
  static constexpr uint32_t OFF_K = 2 * TB, OFF_V = OFF_K + NS * TB, OFF_STAGE = OFF_V + NS * TB;
  static constexpr uint32_t MISC = 4096;
  static constexpr uint32_t SMEM = OFF_STAGE + 8 * kStage + MISC + 1024;
  // TMEM: the streams' O, P and S. Heads of 64 leave room for P beside S, so that the next S is
  // formed during the second product (64 requests of 8,000 keys: 182 -> 174 us); else P lies over
  // the first half of its S.
  static constexpr bool OWN_P = D == 64;
  static constexpr uint32_t TM_O = 0, LD_O = OWN_P ? 64 : 128, TM_S = 256, TM_P = OWN_P ? 128 : TM_S, LD_P = OWN_P ? 64 : 128,
                            TMEM_COLS = 512;
};

// A place on the line of work: before visit kt of item (s, i, h), of nkt visits.
struct alignas(16) Bound {
  int s, i, h, kt;
  int nkt;
  SeqRows r;
};

// A part of an item, as the K producer hands it to the other warps; nt 0 ends the run.
struct alignas(16) Item {
  int row0, nt, h;    // first row of q, tokens, kv head
  int s;              // sequence
  int kt0, kt1, nkt;  // visits of the part, and of the item
  int cap, seen0;     // keys in the cache; keys that the first token sees
  int turns, stream;  // visit vc goes to stream (vc & turns) | stream (a pair's visits to 0 and 1)
};
static_assert(sizeof(Item) == 48, "three vectors, see next_item");
constexpr int kItems = 4;

struct Misc {
  uint64_t q_full[2], q_free[2], k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], o_free[2], sums[2], group[2], fin_s, fin_pv;
  uint64_t item_full[kItems], item_free[kItems];
  uint32_t tmem_base;
  int abort_flag;
  Bound ends[2];
  Item items[kItems];
  uint32_t k_bad[4], v_bad[4], s_bad[2];  // missing pages of the visit in a stage, or in a stream's S
  float stat[2][2][128];                  // [stream][maximum, sum][row]
};

// Partial results of a CTA: slot 0 of the item that its run begins inside of, slot 1 of
// the one that it ends inside of. O as float4 of row r, columns 4c .. 4c + 3 at [c][r].
struct Partial {
  float m[256], l[256];
};
__host__ __device__ constexpr size_t partial_bytes(int D) { return sizeof(Partial) + (size_t)256 * D * 4; }
constexpr size_t kOffRecords = 256, kOffPartials = kOffRecords + kCtas * sizeof(int4);

// What a CTA left: the item that it began and did not end, if any (first row of q, rows of the
// tile, else 0, kv head), and what its run begins with.
enum Head : int { kWhole = 0, kGoesOn = 1, kEnds = 2, kEmpty = 3 };

struct FwdArgs {
  PagedArgs p;
  int TQ;   // tokens of a tile; an item has two of them
  int TQf;  // tokens of one that has few rows
  int page_shift;
  int g_inv;  // ceil(2^16 / G)
  int ctas;
  int least_cost;    // of a CTA, in units
  float cost_scale;  // units a key: a power of two
  __nv_bfloat16* out;
  float* lse;
  uint8_t* ws;
};

// r / G, exact for a row of an item (r < 256, G <= 128) without a division's forty instructions.
__device__ __forceinline__ int by_group(const FwdArgs& a, int r) { return (r * a.g_inv) >> 16; }
__host__ __device__ __forceinline__ int items_of(const FwdArgs& a, int ql) {
  const int n = 2 * a.TQ;
  return ql <= n ? (ql > 0) : (ql + n - 1) / n;
}
// Visits of item i of a sequence: the keys that its last token sees.
__device__ __forceinline__ int visits_of(const FwdArgs& a, const SeqRows& r, int i) {
  const int ql = r.b - r.a, e = min(r.base() + min(ql, (i + 1) * 2 * a.TQ), a.p.width * a.p.page);
  return e <= kTile ? 1 : (e + kTile - 1) / kTile;
}
// Costs of a sequence's items of one kv head, in keys: item i's and all before it. They are
// fp32, since they only have to be the same wherever they are computed (so each product that is added to
// something is an fmaf, and none is left to the compiler), and never to fall as i rises.
struct Costs {
  float A, per, w;
  int ql, n;
  __host__ __device__ __forceinline__ Costs(const FwdArgs& a, const SeqRows& r) {
    ql = r.b - r.a;
    n = items_of(a, ql);
    per = (float)(2 * a.TQ);
    // a sequence of more than a tile is taken as made of pairs of them
    w = ql > a.TQ ? kPairCost : 1.f;
    per *= w;
    A = fmaf(w, (float)min(max(r.base(), 0), a.p.width * a.p.page), (float)(ql > a.TQ ? kPairItemCost : kItemCost));
  }
  __host__ __device__ __forceinline__ float mean(int i) const { return fmaf(0.5f * per, (float)(i + 1), A); }
  __host__ __device__ __forceinline__ float before(int i) const { return mean(i) * (float)i; }
  __host__ __device__ __forceinline__ float of(int i) const {
    return i == n - 1 ? fmaf(w, (float)ql, A) : fmaf(per, (float)(i + 1), A);
  }
  // of the whole sequence and all kv heads, in units of 2^shift keys
  __host__ __device__ __forceinline__ float units(const FwdArgs& a) const {
    return fmaf(mean(n - 1), (float)(n - 1), of(n - 1)) * (float)a.p.Hkv * a.cost_scale;
  }
  // the same in whole ones: the sum over a step fits 32 bits (see sized)
  __device__ __forceinline__ uint32_t scaled(const FwdArgs& a) const { return n ? max(1u, __float2uint_rd(units(a))) : 0u; }
};

// Where `units` of sequence s's cost lie: a function of them that never falls as they rise,
// so that the end of one run is the start of the next. A cut that would leave fewer visits than
// a join is worth on one of its sides moves to the item's end on that side.
__device__ __forceinline__ Bound place(const FwdArgs& a, int s, const SeqRows& r, uint32_t units) {
  const Costs c(a, r);
  const float H = (float)a.p.Hkv, x = __fdividef((float)units, a.cost_scale * H);  // of one kv head's line
  int i = 0;
  for (int hi = c.n; hi - i > 1;) {
    const int mid = i + (hi - i) / 2;
    if (c.before(mid) <= x)
      i = mid;
    else
      hi = mid;
  }
  // the heads of an item one behind the other
  const float part = fmaxf(__fdividef((x - c.before(i)) * H, c.of(i)), 0.f);
  Bound b;
  b.s = s;
  b.i = i;
  b.h = min((int)part, a.p.Hkv - 1);
  b.r = r;
  b.nkt = visits_of(a, r, i);
  b.kt = min((int)((part - (float)b.h) * (float)b.nkt), b.nkt - 1);
  if (b.kt < kLeastVisits)
    b.kt = 0;
  else if (b.nkt - b.kt < kLeastVisits)
    b.kt = b.nkt;
  return b;
}

// Both ends of this CTA's run. Every thread adds up the costs of its share of the sequences
// (neighbours); warp 0 finds the thread's share that an end lies in, then the sequence in it and
// the place, a lane for each end. sums: room for a number a thread.
__device__ __forceinline__ void find_ends(const FwdArgs& a, Bound (&ends)[2], uint32_t* sums) {
  const int S = a.p.S, tid = threadIdx.x, lane = tid & 31, share = (S + kThreads - 1) / kThreads;
  uint32_t mine = 0;
  SeqRows r{0, 0, 0};
#pragma unroll 1
  for (int k = 0; k < share; ++k)
    if (tid * share + k < S) {
      r = seq_rows(a.p, tid * share + k);
      mine += Costs(a, r).scaled(a);
    }
  if (S > 32) {
    sums[tid] = mine;
    __syncthreads();
  }
  if (tid >= 32) return;
  // a lane's part of the sums, and what lies before it
  const int per = S > 32 ? kThreads / 32 : 1;
  if (S > 32) {
    mine = 0;
#pragma unroll 4
    for (int k = 0; k < per; ++k) mine += sums[lane * per + k];
  }
  uint32_t v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  const uint32_t total = __shfl_sync(~0u, v, 31);
  // A run's share of the total, the same numbers in every CTA: as a fraction in 2^-32, which times
  // c < P stays below one for any rounding of it.
  const uint32_t P = max(1u, min(gridDim.x, __float2uint_rd(__fdividef((float)total, (float)a.least_cost))));
  const uint32_t share32 = __float2uint_rd(__fdividef(4294967040.f, (float)P));
  const uint32_t c = blockIdx.x + (lane & 1);
  const uint32_t x = c >= P ? total : __umulhi(total, c * share32);  // lane 0's end, and lane 1's
  const uint32_t x0 = __shfl_sync(~0u, x, 0), x1 = __shfl_sync(~0u, x, 1);
  const uint32_t hit0 = __ballot_sync(~0u, x0 >= v - mine && x0 < v), hit1 = __ballot_sync(~0u, x1 >= v - mine && x1 < v);
  const uint32_t hit = lane ? hit1 : hit0;
  const int from = hit ? __ffs(hit) - 1 : 0;
  int at = hit ? from : S;
  uint32_t left = x - __shfl_sync(~0u, v - mine, from);
  SeqRows t{__shfl_sync(~0u, r.a, from), __shfl_sync(~0u, r.b, from), __shfl_sync(~0u, r.kv, from)};
  if (lane < 2) {
    if (at < S && S > 32) {
      // The thread's share, then the sequence in it. Both are there, for the numbers are those that
      // were added up; the loops end all the same if somebody changes the arrays meanwhile.
      int k = at * per;
      while (k < kThreads - 1 && left >= sums[k]) left -= sums[k++];
      for (at = min(k * share, S - 1);; ++at) {
        t = seq_rows(a.p, at);
        const uint32_t cost = Costs(a, t).scaled(a);
        if (left < cost || at == S - 1) break;
        left -= cost;
      }
    }
    ends[lane] = at < S ? place(a, at, t, left) : Bound{S, 0, 0, 0, 0, SeqRows{0, 0, 0}};
  }
  __syncwarp();
}

// The parts of items in a CTA's run, in order. A whole warp takes it, and passes sequences without
// new tokens 128 at a time: one at a time they are 0.1 us each, and a step's slots may be few of very many in
// use (two tokens in 256 slots: 32 -> 10 us; in 2^24 slots 1.7 s, close to the 2 s after which waits give up).
struct Walk {
  const FwdArgs& a;
  SeqRows r;
  int s, i, h;   // the item
  int n;         // items of the sequence and kv head
  int kt0, kt1;  // visits of this part
  int nkt;       // and of the item
  __device__ __forceinline__ Walk(const FwdArgs& a_, const Misc& m) : a(a_) {
    const Bound b = m.ends[0], e = m.ends[1];
    s = b.s, i = b.i, h = b.h, kt0 = b.kt, r = b.r;
    es = e.s, ei = e.i, eh = e.h, ek = e.kt;
    n = items_of(a, r.b - r.a);
    kt1 = nkt = 0;
    first = true;
  }
  // To the next part; false when there is none.
  __device__ __forceinline__ bool next() {
    for (;;) {
      if (!first) {
        step();
        kt0 = 0;
      }
      first = false;
      const bool last = s == es && i == ei && h == eh;
      if (s >= a.p.S || es < 0 || (last && ek == 0)) return false;
      nkt = visits_of(a, r, i);
      kt1 = last ? ek : nkt;
      if (last) es = -1;  // nothing behind this one
      if (kt0 < kt1) return true;
    }
  }
  __device__ __forceinline__ Item item() const {
    const int t0 = i * 2 * a.TQ;
    return Item{r.a + t0, min(2 * a.TQ, r.b - r.a - t0), h, s, kt0, kt1, nkt, min(r.kv, a.p.width * a.p.page),
                r.base() + t0 + 1, 0, 0};
  }

 private:
  bool first;
  int es, ei, eh, ek;  // the run's end
  __device__ __forceinline__ void step() {
    if (++h < a.p.Hkv) return;
    h = 0;
    if (++i < n) return;
    i = 0;
    if (++s < a.p.S && enter()) return;
    for (++s; s < a.p.S; s += 128) {
      uint32_t some[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = s + k * 32 + (int)(threadIdx.x & 31);
        SeqRows t{0, 0, 0};
        if (x < a.p.S) t = seq_rows(a.p, x);
        some[k] = __ballot_sync(~0u, t.b > t.a);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (some[k]) {
          s += k * 32 + __ffs(some[k]) - 1;
          enter();
          return;
        }
    }
  }
  __device__ __forceinline__ bool enter() {  // sequence s; whether it has items
    r = seq_rows(a.p, s);
    n = items_of(a, r.b - r.a);
    return n > 0;
  }
};

// A lane's page of visit kt as the table has it; -1 past the sequence's keys. What it
// returns is looked at a visit later, so that nobody stands and waits for it.
__device__ __forceinline__ int page_of(const FwdArgs& a, int s, int kt, int cap, int lane, int per) {
  const int key = kt * kTile + lane * a.p.page;
  int id = -1;
  if (lane < per && key < cap) id = __ldg(a.p.page_table + (int64_t)s * a.p.width + (key >> a.page_shift));
  return id;
}
// A producer's lanes: lane l brings chunk l / per of page l % per of a visit.
static_assert(kTile == 128, "the shifts below");
struct PageLanes {
  int per, box, page, chunk, lane;
  __device__ __forceinline__ PageLanes(const FwdArgs& a, int lane_, int NC) {
    const int shift = max(7 - a.page_shift, 0);
    per = 1 << shift;
    box = min(a.p.page, kTile);
    page = lane_ & (per - 1);
    chunk = lane_ >> shift;
    lane = chunk < NC ? page : per;
  }
};

// Bits of the 32 keys from k0 on (of visit kt, its keys k0 + ...) that a row with `seen`
// keys sees and whose pages are there.
__device__ __forceinline__ uint32_t seen32(int seen, int k0, int in_visit, uint32_t bad, int page_shift) {
  const int n = seen - k0;
  uint32_t m = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
  if (bad) {
    if ((bad >> (in_visit >> page_shift)) & 1) m &= 0xFFFF0000u;
    if ((bad >> ((in_visit + 16) >> page_shift)) & 1) m &= 0x0000FFFFu;
  }
  return m;
}
__device__ __forceinline__ void hide32(uint32_t (&x)[32], uint32_t m) {
#pragma unroll
  for (int c = 0; c < 32; ++c) x[c] = (m >> c) & 1 ? x[c] : __float_as_uint(-INFINITY);
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void warp_arrive2(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(bar);
    mbar_arrive(bar);
  }
}
__device__ __forceinline__ float weight(float m, float M) { return m == -INFINITY ? 0.f : ex2(m - M); }

// A softmax thread's running state: the maximum in use and the weights' sums.
struct Running {
  float m;
  uint64_t l2;  // two partial sums
};
// Takes the running maximum on for scores whose largest (scaled) is ms; returns what O, if it
// holds anything, has to be multiplied with where `rescale` comes out true (for the whole warp).
// Only `mine` rows have a say: what the others hold may be left over from anything.
__device__ __forceinline__ float advance(Running& u, float ms, bool mine, bool& rescale) {
  rescale = __any_sync(~0u, mine && ms > u.m + 8.f);
  float f = 1.f;
  if (rescale) {
    const float m_new = fmaxf(u.m, ms);
    f = u.m == m_new ? 1.f : weight(u.m, m_new);
    u.l2 = mul2(u.l2, f2(f, f));
    u.m = m_new;
  }
  return f;
}
template <int D>
__device__ __forceinline__ void scale_o(uint32_t tO, float f) {
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 16) {  // few at a time: the scores stay in registers beside them
    uint32_t v[16];
    tmem_ld16(tO + c0, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
    tmem_st16(tO + c0, v);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmF,
                 const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const __grid_constant__ FwdArgs a) {
  using L = Layout<D>;
  constexpr int NS = L::NS, NC = L::NC;
  static_assert(sizeof(Misc) <= L::MISC, "misc region");
  static_assert(L::SMEM <= 232448, "shared memory");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Misc& m = *reinterpret_cast<Misc*>(smem_raw);
  uint8_t* base =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + sizeof(Misc) + 1023) & ~uintptr_t(1023));
  uint8_t *bK = base + L::OFF_K, *bV = base + L::OFF_V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Guard g{&m.abort_flag, reinterpret_cast<uint32_t*>(a.ws)};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    m.abort_flag = 0;
#pragma unroll 1
    for (int s = 0; s < NS; ++s) {
      mbar_init(&m.k_full[s], 1);
      mbar_init(&m.k_empty[s], 1);
      mbar_init(&m.v_full[s], 1);
      mbar_init(&m.v_empty[s], 1);
    }
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      mbar_init(&m.q_full[s], 1);
      mbar_init(&m.q_free[s], 1);
      mbar_init(&m.s_full[s], 2);  // the S issuer itself, and its products
      mbar_init(&m.s_free[s], 4);  // the four warps of the stream's group
      mbar_init(&m.p_full[s], 4);
      mbar_init(&m.pv_done[s], 1);
      mbar_init(&m.o_free[s], 8);  // both groups' warps, or those of one group twice
      mbar_init(&m.sums[s], 4);
      mbar_init(&m.group[s], 4);
    }
#pragma unroll 1
    for (int s = 0; s < kItems; ++s) {
      mbar_init(&m.item_full[s], 1);
      mbar_init(&m.item_free[s], kThreads / 32 - 1);
    }
    mbar_init(&m.fin_s, 1);
    mbar_init(&m.fin_pv, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    prefetch_tmap(&tmF);
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 2) {
    tmem_alloc(&m.tmem_base, L::TMEM_COLS);
    tmem_relinquish();
  }
  // Up to here nothing that the kernels ahead write was looked at.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0 && blockIdx.x == 0) *g.status = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem_base;
  find_ends(a, m.ends, reinterpret_cast<uint32_t*>(base + L::OFF_STAGE));

  // All roles count alike: ic the items, vc the visits (K and V stages, and the stream of a visit where an item
  // of one tile takes turns, see Item), qt the Q buffer of the next item of one tile.
  int ic = 0, vc = 0;
  bool ok = true;
  const auto next_item = [&](Item& it) {
    const int slot = ic % kItems;
    ok = g.wait_warp(&m.item_full[slot], (ic / kItems) & 1, 18);
    if (!ok) return false;
    const int4* from = reinterpret_cast<const int4*>(&m.items[slot]);
    int4* to = reinterpret_cast<int4*>(&it);
#pragma unroll
    for (int k = 0; k < 3; ++k) to[k] = from[k];
    warp_arrive(&m.item_free[slot], lane);
    ++ic;
    return it.nt > 0;
  };
  const auto is_pair = [&](const Item& it) { return it.nt > a.TQ; };
  const auto is_few = [&](const Item& it) { return it.nt * a.p.G <= kFew; };
  if (warp == 0) {
    // ------------------------------------------------------ Q and K producer
    if (lane == 0) {  // what the second kernel has to know
      const Bound &b = m.ends[0], &e = m.ends[1];
      const bool same = b.s == e.s && b.i == e.i && b.h == e.h;
      int4 rec = make_int4(0, 0, 0, kWhole);
      if (b.kt > 0 && b.kt < b.nkt) rec.w = !same ? kEnds : e.kt == b.kt ? kEmpty : e.kt == e.nkt ? kEnds : kGoesOn;
      if (e.kt > 0 && e.kt < e.nkt && !(same && b.kt > 0)) {
        const int t0 = e.i * 2 * a.TQ;
        rec = make_int4(e.r.a + t0, min(2 * a.TQ, e.r.b - e.r.a - t0) * a.p.G, e.h, rec.w);
      }
      reinterpret_cast<int4*>(a.ws + kOffRecords)[blockIdx.x] = rec;
    }
    __syncwarp();
    const PageLanes pl(a, lane, NC);
    Walk w(a, m);
    int turn = 0;                // the stream of the next item that one takes alone
    uint32_t used = 0, odd = 0;  // bits of the Q buffers: whether they were used, the parity of that
    int qt = 0;
    for (bool more = true; ok && more;) {
      more = w.next();
      Item it = more ? w.item() : Item{};
      if (!is_pair(it)) {
        it.turns = it.kt1 - it.kt0 > (is_few(it) ? kAlone : 1);
        if (!it.turns) it.stream = turn, turn ^= 1;
      }
      const int slot = ic % kItems;
      if (ic >= kItems && !(ok = g.wait_warp(&m.item_free[slot], (ic / kItems - 1) & 1, 19))) break;
      if (lane == 0) {
        m.items[slot] = it;
        mbar_arrive(&m.item_full[slot]);
      }
      __syncwarp();
      ++ic;
      if (!more) break;
      const bool pair = is_pair(it), few = is_few(it);
      int id = page_of(a, it.s, it.kt0, it.cap, pl.lane, pl.per);
      // Q goes ahead of the item's first K where two buffers take turns, and behind it where
      // both wait for the last item's products.
      const int visits = it.kt1 - it.kt0, q_at = pair ? 1 : 0;
#pragma unroll 1
      for (int v = 0; ok && v < max(visits, q_at + 1); ++v) {
        if (v == q_at) {
#pragma unroll 1
          for (int t = 0; ok && t <= q_at; ++t) {
            const int b = pair ? t : qt;
            if ((used >> b) & 1 && !(ok = g.wait_warp(&m.q_free[b], ((odd >> b) & 1) ^ 1, 2))) break;
            if (lane == 0) mbar_expect_tx(&m.q_full[b], NC * a.p.G * 128 * (few ? 4 * a.TQf : a.TQ));
            __syncwarp();
            const int c = lane >> 2, q = lane & 3;  // a lane a box
            if (c < NC && (few || q == 0))
              tma_load_bhnd(base + b * L::TB + c * L::CHUNK + q * 32 * 128, few ? &tmF : &tmQ, &m.q_full[b], c * 64, 0,
                            it.row0 + t * a.TQ, it.h);
            used |= 1u << b;
            odd ^= 1u << b;
          }
          if (!pair) qt ^= 1;
          if (!ok) break;
        }
        if (v >= visits) break;
        const int kt = it.kt0 + v, now = id, sk = vc % NS;
        if (v + 1 < visits) id = page_of(a, it.s, kt + 1, it.cap, pl.lane, pl.per);
        const bool there = (uint32_t)now < (uint32_t)a.p.pages;
        const uint32_t boxes = __ballot_sync(~0u, there);
        const uint32_t bad = __ballot_sync(~0u, lane < pl.per && kt * kTile + lane * a.p.page < it.cap && !there);
        if (!(ok = g.wait_warp(&m.k_empty[sk], ((vc / NS) & 1) ^ 1, 1))) break;
        if (lane == 0) {
          m.k_bad[sk] = bad;
          mbar_expect_tx(&m.k_full[sk], __popc(boxes) * pl.box * 128);
        }
        __syncwarp();
        if (there)
          tma_load_bhnd(bK + sk * L::TB + pl.chunk * L::CHUNK + pl.page * pl.box * 128, &tmK, &m.k_full[sk], pl.chunk * 64,
                        (kt * kTile) & (a.p.page - 1) & ~(kTile - 1), it.h, now);
        ++vc;
      }
    }
    if (lane == 0) {  // no copy may still be landing when the CTA exits
      for (int b = 0; b < 2; ++b)
        if ((used >> b) & 1) g.drain(&m.q_full[b], ((odd >> b) & 1) ^ 1);
      for (int i = (vc > NS ? vc - NS : 0); i < vc; ++i) g.drain(&m.k_full[i % NS], (i / NS) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ V producer
    const PageLanes pl(a, lane, NC);
    Item it;
    while (ok && next_item(it)) {
      int id = page_of(a, it.s, it.kt0, it.cap, pl.lane, pl.per);
      for (int kt = it.kt0; kt < it.kt1; ++kt, ++vc) {
        const int now = id, sv = vc % NS;
        if (kt + 1 < it.kt1) id = page_of(a, it.s, kt + 1, it.cap, pl.lane, pl.per);
        const bool there = (uint32_t)now < (uint32_t)a.p.pages;
        const uint32_t boxes = __ballot_sync(~0u, there);
        const uint32_t bad = __ballot_sync(~0u, lane < pl.per && kt * kTile + lane * a.p.page < it.cap && !there);
        if (!(ok = g.wait_warp(&m.v_empty[sv], ((vc / NS) & 1) ^ 1, 3))) break;
        if (lane == 0) {
          m.v_bad[sv] = bad;
          mbar_expect_tx(&m.v_full[sv], __popc(boxes) * pl.box * 128);
        }
        __syncwarp();
        if (there)
          tma_load_bhnd(bV + sv * L::TB + pl.chunk * L::CHUNK + pl.page * pl.box * 128, &tmV, &m.v_full[sv], pl.chunk * 64,
                        (kt * kTile) & (a.p.page - 1) & ~(kTile - 1), it.h, now);
      }
    }
    if (lane == 0)
      for (int i = (vc > NS ? vc - NS : 0); i < vc; ++i) g.drain(&m.v_full[i % NS], (i / NS) & 1);
    __syncwarp();
  } else if (warp == 2) {
    // -------------------------------------------------------------- S issuer
    const bool leader = lane == 0;
    constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false);
    const uint64_t qd = sdesc_sw128(smem_u32(base), 16, 1024);
    // bits of the streams: whether they had a visit, the parity of their visits; of the Q buffers' uses
    uint32_t had = 0, odd = 0, q_odd = 0;
    int qt = 0;
    Item it;
    while (ok && next_item(it)) {
      const bool pair = is_pair(it);
#pragma unroll 1
      for (int t = 0; ok && t < (pair ? 2 : 1); ++t) {
        const int b = pair ? t : qt;
        ok = g.wait_warp(&m.q_full[b], (q_odd >> b) & 1, 4);
        q_odd ^= 1u << b;
      }
      for (int kt = it.kt0; ok && kt < it.kt1; ++kt, ++vc) {
        const int sk = vc % NS;
        if (!(ok = g.wait_warp(&m.k_full[sk], (vc / NS) & 1, 6))) break;
        const uint32_t bad = m.k_bad[sk];
        const uint64_t kd = sdesc_sw128(smem_u32(bK + sk * L::TB), 16, 1024);
        const int lo = (vc & it.turns) | it.stream, hi = lo + pair;
#pragma unroll 1
        for (int gs = lo; gs <= hi; ++gs) {
          // the stream's last S has been read, and its P, where that lies over S
          if ((had >> gs) & 1 && !(ok = g.wait_warp(L::OWN_P ? &m.s_free[gs] : &m.pv_done[gs], ((odd >> gs) & 1) ^ 1, 5))) break;
          had |= 1u << gs;
          odd ^= 1u << gs;
          tc_fence_after();
          if (leader) {
            const uint64_t qb = sdesc_add(qd, (pair ? gs : qt) * L::TB);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t ko = (kk >> 2) * L::CHUNK + (kk & 3) * 32;
              umma_bf16(tmem + L::TM_S + gs * 128, sdesc_add(qb, ko), sdesc_add(kd, ko), idS, kk > 0 ? 1u : 0u);
            }
            m.s_bad[gs] = bad;
            mbar_arrive(&m.s_full[gs]);
            umma_commit(&m.s_full[gs]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) {
          umma_commit(&m.k_empty[sk]);
          if (kt + 1 == it.kt1) {
            if (pair || qt == 0) umma_commit(&m.q_free[0]);
            if (pair || qt == 1) umma_commit(&m.q_free[1]);
          }
        }
        __syncwarp();
      }
      if (!pair) qt ^= 1;
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
    // bits of the streams: the parity of their visits, whether O held an item, the parity of those
    uint32_t odd = 0, held = 0, held_odd = 0;
    Item it;
    while (ok && next_item(it)) {
      const bool pair = is_pair(it);
      uint32_t fresh = 3;
      for (int kt = it.kt0; kt < it.kt1; ++kt, ++vc) {
        const int sv = vc % NS;
        if (!(ok = g.wait_warp(&m.v_full[sv], (vc / NS) & 1, 7))) break;
        // The product takes the steps of 16 keys that hold some. Rows past the last key in its
        // step are set to zero (0 * NaN is NaN); a visit without any key takes one step of zeros.
        const int there = it.cap - kt * kTile;
        uint32_t steps = there >= kTile ? 0xFFu : there <= 0 ? 0u : (1u << ((there + 15) >> 4)) - 1u;
        const uint32_t bad = m.v_bad[sv];
        if (bad) {
#pragma unroll 1
          for (int kk = 0; kk < 8; ++kk)
            if ((bad >> ((kk * 16) >> a.page_shift)) & 1) steps &= ~(1u << kk);
        }
        if (there < kTile || steps == 0) {
          const int r0 = steps == 0 ? 0 : there, r1 = steps == 0 ? 16 : (there + 15) & ~15;
          for (int e = r0 * 128 + lane * 16; e < r1 * 128; e += 512)
            for (int c = 0; c < NC; ++c) st_shared_v4(smem_u32(bV + sv * L::TB + c * L::CHUNK + e), 0, 0, 0, 0);
          fence_async_smem();
          __syncwarp();
          if (steps == 0) steps = 1;
        }
        const uint64_t vd = sdesc_sw128(smem_u32(bV + sv * L::TB), L::CHUNK, 1024);
        const int lo = (vc & it.turns) | it.stream, hi = lo + pair;
#pragma unroll 1
        for (int gs = lo; gs <= hi; ++gs) {
          const uint32_t bit = 1u << gs;
          if (fresh & bit) {  // O is free once its last item's has been read
            if (held & bit && !(ok = g.wait_warp(&m.o_free[gs], ((held_odd >> gs) & 1) ^ 1, 8))) break;
            held |= bit;
            held_odd ^= bit;
          }
          const uint32_t tO = tmem + L::TM_O + gs * L::LD_O, tP = tmem + L::TM_P + gs * L::LD_P;
          const bool add = !(fresh & bit);
          if (!(ok = g.wait_warp(&m.p_full[gs], (odd >> gs) & 1, 9))) break;
          tc_fence_after();
          if (leader) {
            if (steps == 0xFFu) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                umma_bf16_ta(tO, tP + kk * 8, sdesc_add(vd, kk * 2048), idO, (add || kk > 0) ? 1u : 0u);
            } else {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                if ((steps >> kk) & 1)
                  umma_bf16_ta(tO, tP + kk * 8, sdesc_add(vd, kk * 2048), idO, (add || (steps & ((1u << kk) - 1u))) ? 1u : 0u);
            }
          }
          odd ^= bit;
          fresh &= ~bit;
          if (leader) umma_commit(&m.pv_done[gs]);
          __syncwarp();
        }
        if (!ok) break;
        if (leader) umma_commit(&m.v_empty[sv]);
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
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_base + L::TM_O, tS = tmem + lane_base + L::TM_S + grp * 128,
                   tP = tmem + lane_base + L::TM_P + grp * L::LD_P;
    const float sl2 = a.p.scale_log2;
    const uint64_t sc = f2(sl2, sl2);
    // Parities, in one register since the scores leave few: of this stream's visits (and whether it had
    // any), of its group's barrier, of the two groups', of all visits; above them the items' number.
    constexpr uint32_t NV = 1, HAD = 2, GP = 4, EX = 8, VC = 16, IC = 32;
    uint32_t ph = 0;
    // The item stays in its place until the epilogue has read it again, for its numbers would take
    // registers from the scores in between.
    for (; ok; ph += IC) {
      const int ring = ph / IC % kItems;
      if (!(ok = g.wait_warp(&m.item_full[ring], ph / (IC * kItems) & 1, 18))) break;
      const Item& at = m.items[ring];
      if (at.nt == 0) break;
      const bool few = is_few(at);
      int first_seen, seen, kt, kt1, step;
      bool mine_row, active;
      {
        const Item it = at;
        const bool pair = is_pair(it);
        const int t0 = pair ? grp * a.TQ : 0;  // this stream's first token of the item
        const int rl = few ? lane : r, tok = t0 + by_group(a, rl);
        mine_row = t0 * a.p.G + rl < it.nt * a.p.G && rl < a.TQ * a.p.G;
        first_seen = min(it.seen0 + t0, it.cap);  // keys that the first one sees
        seen = min(it.seen0 + tok, it.cap);
        active = few || t0 + by_group(a, quarter * 32) < it.nt;  // some row of this warp is a token's
        step = 1 + it.turns;
        kt = it.kt0;
        if (it.turns)
          kt += (int)(ph / VC & 1) != grp;
        else if (!pair && it.stream != grp)
          kt = it.kt1;
        kt1 = it.kt1;
        ph ^= (it.kt1 - it.kt0) & 1 ? VC : 0;
      }
      Running u{-INFINITY, 0ull};
      const bool part = kt < kt1;  // this stream has visits of the item
      bool any = false;
      for (; kt < kt1; kt += step, ph = (ph ^ NV) | HAD) {
        if (!(ok = g.wait_warp(&m.s_full[grp], ph & NV, 10))) break;
        if (!active) {  // in step with the others, nothing to do
          if (L::OWN_P) {
            warp_arrive(&m.s_free[grp], lane);
            if ((ph & HAD) && !(ok = g.wait_warp(&m.pv_done[grp], ~ph & NV, 20))) break;
          }
          warp_arrive(&m.p_full[grp], lane);
          continue;
        }
        tc_fence_after();
        const uint32_t bad = m.s_bad[grp];
        const bool masked = bad || (kt + 1) * kTile > first_seen;
        const int k0 = kt * kTile;
        bool rescale;
        uint64_t t2 = 0ull, none = 0ull;
        float f;
        if (few) {
          uint32_t x[32];
          tmem_ld32(tS + quarter * 32, x);
          if (L::OWN_P) {
            tc_fence_before();
            warp_arrive(&m.s_free[grp], lane);
          }
          if (masked) hide32(x, seen32(seen, k0 + quarter * 32, quarter * 32, bad, a.page_shift));
          f = advance(u, max32(x) * sl2, mine_row, rescale);
          if (L::OWN_P && (ph & HAD)) {  // the last P has been read
            if (!(ok = g.wait_warp(&m.pv_done[grp], ~ph & NV, 20))) break;
            tc_fence_after();
          }
          if (rescale && any) scale_o<D>(tO + grp * L::LD_O, f);
          const float moff = (u.m == -INFINITY) ? 0.f : u.m;
          exp_store32<false>(x, sc, f2(-moff, -moff), tP + quarter * 16, t2, none);
          const uint32_t zero[16] = {};
#pragma unroll
          for (int q = 1; q < 4; ++q) tmem_st16_nowait(tP + ((quarter + q) & 3) * 16, zero);
        } else {
          // Twice through the scores, 64 at a time: maximum, then weights. Held all at once and unrolled
          // they take every register and half of the loop's code, and its time hangs on how the
          // compiler lays the rest out (a chunk of 4,096 of 8,192 tokens 320 to 367 us from one build to
          // the next, now 330 to 337; 33 x 5 tokens 30.2 -> 28.5, a chunk beside 47 tokens 106 -> 102).
          float ms = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 128; c += 64) {
            uint32_t x0[32], x1[32];
            tmem_ld32x2(tS + c, tS + c + 32, x0, x1);
            if (masked) {
              hide32(x0, seen32(seen, k0 + c, c, bad, a.page_shift));
              hide32(x1, seen32(seen, k0 + c + 32, c + 32, bad, a.page_shift));
            }
            ms = fmax3(ms, max32(x0), max32(x1));
          }
          f = advance(u, ms * sl2, mine_row, rescale);
          if (L::OWN_P && (ph & HAD)) {
            if (!(ok = g.wait_warp(&m.pv_done[grp], ~ph & NV, 20))) break;
            tc_fence_after();
          }
          // the stream's last product has ended (its S was formed after it, or see above), so O stands still
          if (rescale && any) scale_o<D>(tO + grp * L::LD_O, f);
          const float moff = (u.m == -INFINITY) ? 0.f : u.m;
          const uint64_t off = f2(-moff, -moff);
#pragma unroll 1
          for (int c = 0; c < 128; c += 64) {
            uint32_t x0[32], x1[32];
            tmem_ld32x2(tS + c, tS + c + 32, x0, x1);
            if (L::OWN_P && c == 64) {
              tc_fence_before();
              warp_arrive(&m.s_free[grp], lane);
            }
            if (masked) {
              hide32(x0, seen32(seen, k0 + c, c, bad, a.page_shift));
              hide32(x1, seen32(seen, k0 + c + 32, c + 32, bad, a.page_shift));
            }
            exp_store32<false>(x0, sc, off, tP + c / 2, t2, none);
            exp_store32<false>(x1, sc, off, tP + c / 2 + 16, t2, none);
          }
        }
        u.l2 = add2(u.l2, t2);
        any = true;
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&m.p_full[grp], lane);
      }
      if (!ok) break;
      // -------------------------------------------------------------- epilogue
      if (!part) {  // the other stream's item alone
        warp_arrive(&m.item_free[ring], lane);
        continue;
      }
      const Item it = at;
      const bool pair = is_pair(it);
      const int t0 = pair ? grp * a.TQ : 0, rl = few ? lane : r, tok = t0 + by_group(a, rl);
      const int rows = it.nt * a.p.G, row = t0 * a.p.G + rl;  // the item's rows, and this thread's
      warp_arrive(&m.item_free[ring], lane);
      const bool halves = it.turns;  // two streams' O to be joined, half of the columns each
      const bool whole = it.kt1 - it.kt0 == it.nkt;
      const int c_lo = halves ? grp * (L::DL / 2) : 0, c_hi = halves ? min(c_lo + L::DL / 2, D) : D;
      const int64_t t = it.row0 + tok;
      const int head = it.h * a.p.G + rl - (tok - t0) * a.p.G;
      uint8_t* slot = a.ws + kOffPartials + ((size_t)blockIdx.x * 2 + (it.kt0 == 0 ? 1 : 0)) * partial_bytes(D);
      float4* po = reinterpret_cast<float4*>(slot + sizeof(Partial));
      const unsigned long long dst = reinterpret_cast<unsigned long long>(a.out + t * a.p.o_t + (int64_t)head * a.p.o_h);
      const float2 lp = f2_split(u.l2);
      float M = u.m, lt = lp.x + lp.y, fa = 1.f, fb = 0.f;
      if (!(ok = g.wait_warp(&m.pv_done[grp], ~ph & NV, 11))) break;
      tc_fence_after();
      if (!pair) {
        // what the rows' other parts have to know: of the other stream, and of a few rows' warps
        m.stat[grp][0][r] = M;
        m.stat[grp][1][r] = lt;
        tc_fence_before();
        // Both groups meet at each item that both have visits of, so neither is ever a phase of
        // `sums` ahead; an item of one stream meets within its group.
        warp_arrive(halves ? &m.sums[grp] : &m.group[grp], lane);
        if (halves) {
          if (!(ok = g.wait_warp(&m.sums[grp], ph / EX & 1, 12) && g.wait_warp(&m.sums[grp ^ 1], ph / EX & 1, 13))) break;
          ph ^= EX;
        } else {
          if (!(ok = g.wait_warp(&m.group[grp], ph / GP & 1, 12))) break;
          ph ^= GP;
        }
        tc_fence_after();
        const float *sa = m.stat[halves ? 0 : grp][0], *sb = m.stat[halves ? 1 : grp][0];  // a stream alone counts once
        const float ma = sa[r], mb = sb[r];
        const float nb = halves ? 1.f : 0.f;
        if (few) {
          float x[8], y[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            x[q] = sa[q * 32 + lane], x[q + 4] = sb[q * 32 + lane];
            y[q] = sa[128 + q * 32 + lane], y[q + 4] = sb[128 + q * 32 + lane] * nb;
          }
          M = fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
          lt = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) lt = fmaf(y[k], weight(x[k], M), lt);
        } else {
          M = fmaxf(ma, mb);
          lt = fmaf(sa[128 + r], weight(ma, M), sb[128 + r] * nb * weight(mb, M));
        }
        fa = weight(ma, M);
        fb = weight(mb, M);
      }
      if (whole) {
        const float inv = lt > 0.f ? 1.f / lt : 0.f;
        fa *= inv;
        fb *= inv;
      }
      const uint32_t tA = tO + (halves ? 0 : grp * L::LD_O), tB = tO + L::LD_O;
      if (mine_row && c_lo == 0 && (!few || quarter == 0)) {
        if (whole) {
          a.lse[t * a.p.Hq + head] = M * 0.6931471805599453f + logf(lt);
        } else {
          Partial& pt = *reinterpret_cast<Partial*>(slot);
          pt.m[row] = M;
          pt.l[row] = lt;
        }
      }
      if (few) {
        // the four parts of a row meet in shared memory, as many columns at a time as there is room for
        const int cs = rows > 4 ? 64 : 128, ld = cs + 4, f4 = cs == 64 ? 4 : 5;
        constexpr int part_ld = kStage / 4;
        float* st = reinterpret_cast<float*>(base + L::OFF_STAGE + grp * 4 * kStage);
        const int e = threadIdx.x & 127, rr = e >> f4, c4 = (e & ((1 << f4) - 1)) * 4, tk = by_group(a, rr);
        __nv_bfloat16* o = a.out + (it.row0 + tk) * a.p.o_t + (int64_t)(it.h * a.p.G + rr - tk * a.p.G) * a.p.o_h;
#pragma unroll 1
        for (int c0 = c_lo; ok && c0 < c_hi; c0 += cs) {
#pragma unroll 1
          for (int c = 0; c < cs && c0 + c < c_hi; c += 32) {
            uint32_t v[32];
            tmem_ld32(tA + c0 + c, v);
            if (halves) {
              uint32_t v2[32];
              tmem_ld32(tB + c0 + c, v2);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(fmaf(__uint_as_float(v2[k]), fb, __uint_as_float(v[k]) * fa));
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * fa);
            }
            if (lane < rows) {
              float* to = st + quarter * part_ld + lane * ld + c;
#pragma unroll
              for (int k = 0; k < 32; k += 4) st_shared_v4(smem_u32(to + k), v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
            __syncwarp();
          }
          warp_arrive(&m.group[grp], lane);
          if (!(ok = g.wait_warp(&m.group[grp], ph / GP & 1, 14))) break;
          ph ^= GP;
          if (rr < rows && c0 + c4 < c_hi) {
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 z = *reinterpret_cast<const float4*>(st + q * part_ld + rr * ld + c4);
              y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
            }
            if (whole)
              *reinterpret_cast<uint2*>(o + c0 + c4) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
            else
              po[(size_t)((c0 + c4) / 4) * 256 + rr] = y;
          }
          if (c0 + cs < c_hi) {  // (the last step's sync is the next item's way here)
            warp_arrive(&m.group[grp], lane);
            if (!(ok = g.wait_warp(&m.group[grp], ph / GP & 1, 15))) break;
            ph ^= GP;
          }
        }
        if (!ok) break;
      } else if (active) {
        uint8_t* stage = base + L::OFF_STAGE + (warp - 4) * kStage;
#pragma unroll 1
        for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(tA + c0, v);
          if (halves) {
            uint32_t v2[32];
            tmem_ld32(tB + c0, v2);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(fmaf(__uint_as_float(v2[e]), fb, __uint_as_float(v[e]) * fa));
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * fa);
          }
          if (whole) {
            // through shared memory, so that four lanes write 64 neighbouring bytes of a row
#pragma unroll
            for (int q = 0; q < 4; ++q)
              st_shared_v4(smem_u32(stage + lane * 80 + q * 16),
                           pack_bf16x2(__uint_as_float(v[q * 8 + 0]), __uint_as_float(v[q * 8 + 1])),
                           pack_bf16x2(__uint_as_float(v[q * 8 + 2]), __uint_as_float(v[q * 8 + 3])),
                           pack_bf16x2(__uint_as_float(v[q * 8 + 4]), __uint_as_float(v[q * 8 + 5])),
                           pack_bf16x2(__uint_as_float(v[q * 8 + 6]), __uint_as_float(v[q * 8 + 7])));
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int from = q * 8 + (lane >> 2);
              const uint4 y = *reinterpret_cast<const uint4*>(stage + from * 80 + (lane & 3) * 16);
              const unsigned long long to = __shfl_sync(~0u, dst, from);
              if (__shfl_sync(~0u, (int)mine_row, from))
                *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(to) + c0 + (lane & 3) * 8) = y;
            }
          } else if (mine_row) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              po[(size_t)(c0 / 4 + q) * 256 + row] =
                  make_float4(__uint_as_float(v[q * 4]), __uint_as_float(v[q * 4 + 1]), __uint_as_float(v[q * 4 + 2]),
                              __uint_as_float(v[q * 4 + 3]));
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      if (halves) {
        warp_arrive(&m.o_free[0], lane);
        warp_arrive(&m.o_free[1], lane);
      } else {
        warp_arrive2(&m.o_free[grp], lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// Joins the parts of the item that CTA blockIdx.x began and did not end, 16 of its rows at a
// time. What it reads hangs on the records alone, so that all of it is under way after one
// round trip: a thread takes four columns of a row (or of two), of every n-th part where rows are
// few, and has eight loads in flight.
constexpr int kJoinThreads = 256, kJoinRows = 16, kJoinAhead = 8;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ FwdArgs a) {
  __shared__ int slots[kCtas + 1];
  __shared__ float2 ml[kCtas][kJoinRows];  // the parts' maxima and sums, then their weights
  __shared__ float2 sum[kJoinRows];        // the rows' maxima and sums
  __shared__ float4 share[kJoinThreads];
  __shared__ int count;
  constexpr int C4 = D / 4;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4* recs = reinterpret_cast<const int4*>(a.ws + kOffRecords);
  const int P = gridDim.x, tid = threadIdx.x, lane = tid & 31, b = blockIdx.x;
  const int4 rec = recs[b];
  int head = b + 1 + lane < P ? recs[b + 1 + lane].w : kWhole;
  if ((int)blockIdx.y * kJoinRows >= rec.y) return;
  if (tid < 32) {  // the parts: this CTA's, then the following ones' up to the one that ends the item
    int n = 1;
#pragma unroll 1
    for (int c0 = b + 1;; c0 += 32) {
      const uint32_t stop = __ballot_sync(~0u, head != kGoesOn && head != kEmpty);
      const uint32_t upto = stop ? (2u << (__ffs(stop) - 1)) - 1u : ~0u;  // lanes up to the first that ends it
      const uint32_t part = __ballot_sync(~0u, head == kGoesOn || head == kEnds) & upto;
      if ((part >> lane) & 1) slots[n + __popc(part & ((1u << lane) - 1u))] = (c0 + lane) * 2;
      n += __popc(part);
      if (stop) break;
      head = c0 + 32 + lane < P ? recs[c0 + 32 + lane].w : kWhole;
    }
    if (lane == 0) {
      slots[0] = b * 2 + 1;
      count = n;
    }
  }
  __syncthreads();
  const int n = count;
  const uint8_t* parts = a.ws + kOffPartials;
#pragma unroll 1
  for (int first = blockIdx.y * kJoinRows; first < rec.y; first += gridDim.y * kJoinRows) {
    // rows and columns of this round: 4, 8 or 16 rows, an element a thread, two or a share of one
    const int rows = min(kJoinRows, rec.y - first), shift = rows <= 4 ? 2 : rows <= 8 ? 3 : 4;
    const int E = C4 << shift, per = E > kJoinThreads ? 2 : 1, groups = per == 2 ? 1 : kJoinThreads / E;
    const int grp = per == 2 ? 0 : tid / E, e0 = tid - grp * E, row = e0 & ((1 << shift) - 1);  // E is a multiple of 1 << shift
    const bool on = row < rows && grp < groups;
    const auto o_of = [&](int k, int e) {
      return *(reinterpret_cast<const float4*>(parts + slots[k] * partial_bytes(D) + sizeof(Partial)) + (e >> shift) * 256 + first + row);
    };
    float4 ahead[kJoinAhead];
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i) {
      const int e = e0 + (per == 2 && i >= kJoinAhead / 2 ? kJoinThreads : 0), k = per == 2 ? i % (kJoinAhead / 2) : grp + i * groups;
      if (on && e < E && k < n) ahead[i] = o_of(k, e);
    }
#pragma unroll 1
    for (int e = tid; e < n * kJoinRows; e += kJoinThreads) {
      const int k = e / kJoinRows, r = e % kJoinRows;
      const Partial& pt = *reinterpret_cast<const Partial*>(parts + slots[k] * partial_bytes(D));
      ml[k][r] = make_float2(pt.m[first + r], pt.l[first + r]);
    }
    __syncthreads();
#pragma unroll 1
    for (int r = tid >> 5; r < rows; r += kJoinThreads / 32) {  // a warp a row
      float M = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int k = lane; k < n; k += 32) M = fmaxf(M, ml[k][r].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
#pragma unroll 1
      for (int k = lane; k < n; k += 32) {
        const float2 v = ml[k][r];
        const float x = weight(v.x, M);
        ml[k][r].x = x;
        l = fmaf(v.y, x, l);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
      if (lane == 0) sum[r] = make_float2(M, l);
    }
    __syncthreads();
    float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    const auto add = [](float4& to, const float4& v, float x) {
      to.x = fmaf(v.x, x, to.x);
      to.y = fmaf(v.y, x, to.y);
      to.z = fmaf(v.z, x, to.z);
      to.w = fmaf(v.w, x, to.w);
    };
    if (on) {
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) {
        const int second = per == 2 && i >= kJoinAhead / 2, k = per == 2 ? i % (kJoinAhead / 2) : grp + i * groups;
        if (e0 + second * kJoinThreads < E && k < n) {
          if (second)
            add(o[1], ahead[i], ml[k][row].x);
          else
            add(o[0], ahead[i], ml[k][row].x);
        }
      }
#pragma unroll 4
      for (int k = per == 2 ? kJoinAhead / 2 : grp + kJoinAhead * groups; k < n; k += groups) {
        add(o[0], o_of(k, e0), ml[k][row].x);
        if (e0 + kJoinThreads < E) add(o[1], o_of(k, e0 + kJoinThreads), ml[k][row].x);
      }
    }
    if (groups > 1) {
      share[tid] = o[0];
      __syncthreads();
      if (on && grp == 0)
#pragma unroll 1
        for (int i = 1; i < groups; ++i) add(o[0], share[i * E + e0], 1.f);
    }
    if (on && grp == 0) {
      const float2 t = sum[row];
      const float inv = t.y > 0.f ? 1.f / t.y : 0.f;
      const int tok = by_group(a, first + row), h = rec.z * a.p.G + (first + row - tok * a.p.G);
      const int64_t at = rec.x + tok;
      __nv_bfloat16* out = a.out + at * a.p.o_t + (int64_t)h * a.p.o_h;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (e0 + i * kJoinThreads < E)
          *reinterpret_cast<uint2*>(out + ((e0 + i * kJoinThreads) >> shift) * 4) =
              make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv), pack_bf16x2(o[i].z * inv, o[i].w * inv));
      if (e0 >> shift == 0) a.lse[at * a.p.Hq + h] = t.x * 0.6931471805599453f + logf(t.y);
    }
    __syncthreads();  // the next rows' statistics take the place of these
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
  CUtensorMap tq, tf, tk, tv;
  const uint64_t qd[4] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)p.T, (uint64_t)p.Hkv};
  const int64_t qs[3] = {p.q_h, p.q_t, p.Hkv > 1 ? p.G * p.q_h : D};
  const uint32_t qbox[2] = {(uint32_t)p.G, (uint32_t)a.TQ}, fbox[2] = {(uint32_t)p.G, (uint32_t)a.TQf};
  const uint64_t kd[4] = {(uint64_t)D, (uint64_t)p.page, (uint64_t)p.Hkv, (uint64_t)p.pages};
  const int64_t ks[3] = {p.p_n, p.p_h, p.p_p};
  const uint32_t kbox[2] = {(uint32_t)std::min(p.page, kTile), 1};
  if (!tmap_bf16_4d_sw128(&tq, q, qd, qs, qbox) || !tmap_bf16_4d_sw128(&tf, q, qd, qs, fbox) ||
      !tmap_bf16_4d_sw128(&tk, k_pages, kd, ks, kbox) || !tmap_bf16_4d_sw128(&tv, v_pages, kd, ks, kbox))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(paged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
  if (e != cudaSuccess) return e;
  const int ctas = a.ctas;
  // Both programmatic: each waits for the kernel ahead before it reads or writes memory
  // that others write, and lets the next one start its prologue early.
  cudaLaunchAttribute attr = programmatic_launch();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::SMEM;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, paged_kernel<D>, tq, tf, tk, tv, a)) != cudaSuccess) return e;
  // Nothing is cut, and nothing to be joined, where no context holds two parts' visits.
  if ((p.width * p.page + kTile - 1) / kTile < 2 * kLeastVisits) return cudaSuccess;
  cfg.gridDim = dim3(ctas, std::min(8, (std::min(2 * a.TQ, p.T) * p.G + kJoinRows - 1) / kJoinRows));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, a);
}

}  // namespace

size_t paged_ws_bytes(int D) { return kOffPartials + 2 * kCtas * partial_bytes(D); }

// The step's sizes as the kernel takes them. `most` is the most, in keys, that a step with rising q_start
// and any kv_len can cost; a unit is so many keys that it stays below half of what 32 bits hold.
static FwdArgs sized(const PagedArgs& p, double& most) {
  FwdArgs a{};
  a.p = p;
  a.TQ = kTile / p.G;
  a.TQf = std::max(1, kFew / p.G);
  a.g_inv = (65536 + p.G - 1) / p.G;
  while ((1 << a.page_shift) < p.page) ++a.page_shift;
  // an item's keys: at most the table's ahead of the new tokens, and its sequence's new tokens up to its end,
  // which Costs counts whether the table lists them or not
  most = ((double)p.T / (2 * a.TQ) + p.S) * p.Hkv * (kPairCost * ((double)p.width * p.page + p.T + 2.0 * a.TQ) + kPairItemCost);
  double unit = 1;
  while (most > 2e9 * unit) unit *= 2;
  a.cost_scale = (float)(1 / unit);
  a.least_cost = std::max(1, (int)(kLeastCost / unit));
  return a;
}

uint64_t paged_units(const PagedArgs& p) {
  double most;
  const FwdArgs a = sized(p, most);
  uint64_t sum = 0;
  for (int s = 0; s < p.S; ++s) {
    const Costs c(a, seq_rows(p, s));
    if (c.n) sum += std::max<uint64_t>(1, (uint64_t)c.units(a));
  }
  return sum;
}

cudaError_t launch_paged_fwd(const PagedArgs& p, const void* q, const void* k_pages, const void* v_pages, void* out, float* lse,
                             void* ws, cudaStream_t st) {
  double most;
  FwdArgs a = sized(p, most);
  a.ctas = (int)std::min<double>(std::min(sm_count(), kCtas), std::max(1.0, most / kLeastCost));
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.ws = static_cast<uint8_t*>(ws);
  if (p.D == 64) return launch_d<64>(a, q, k_pages, v_pages, st);
  if (p.D == 96) return launch_d<96>(a, q, k_pages, v_pages, st);
  return launch_d<128>(a, q, k_pages, v_pages, st);
}

}  // namespace pa
