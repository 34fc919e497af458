// tree_attn.cuh -- the attention kernel that tree_attn.cu and prefix_attn.cu launch; its
// mathematics, roles and bounds stand at the head of tree_attn.cu.
#pragma once

#include "attn_common.cuh"
#include "launch.h"

namespace dflash2 {
namespace {   // (the kernel is a template: each file that includes this has its own instances)

constexpr int kThreads = 416;
constexpr int kChunk = 64;              // keys of an S product
constexpr int kMaxSlots = 10;
constexpr int kBufs = 2;                // S buffers per pipeline (a third one, at D = 64, gained nothing)
constexpr uint32_t kTmemO = 2 * kBufs * kChunk;   // first TMEM column of O: pipeline i's at kTmemO + i D
constexpr int kMaxRuns = 512;           // most CTAs
constexpr int kMaxTeam = 8;              // most CTAs of a team (a power of 2)
constexpr int kWholeUnits = 2;           // items of up to so many units are never cut
constexpr float kRescale = 8.0f;        // log2 of how far P may exceed 1

// How a launch deals out its items: equal runs of units over all sequences; a cluster (team)
// for each item; or runs of equal cost over sequences and shared prefixes (prefix_attn.cu).
enum Mode { kRuns, kTeam, kShared };

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                 // 128-byte column blocks of a row
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 10;       // ring of K and V tiles: 160 KB
  static constexpr size_t kRing = static_cast<size_t>(2 + kSlots) * kTileBytes;
};

struct AttnSmem {
  uint64_t kv_full[2 * kMaxSlots], kv_empty[kMaxSlots];
  uint64_t q_full, q_empty;
  uint64_t s_full[2][kBufs], p_ready[2][kBufs], pv_done[2][kBufs], drain;   // [pipeline][S buffer]
  float2 ml[2][kTile];
  uint32_t bad[4];          // drafted nodes that hold a non-finite value
  uint32_t tmem;
  int abort_flag;
  int odd;                  // whether some row's sums have to be taken again
};

// How CTAs are dealt to the pairs of row tiles of a kv head.  With lanes.n = 0 a run
// holds all pairs' units, pair after pair.  Otherwise each pair's units are cut into
// runs of their own: n pairs into `runs` each, run after run, pair beside pair, so
// that the CTAs that read the same keys do so at the same time; and, where a single
// row tile is left over, that one into the CTAs that remain.
struct Lanes {
  int32_t n, runs;
  __device__ __forceinline__ int32_t pair(int32_t cta) const { return cta < n * runs ? cta % n : n; }
  // CTAs from one run to the next (with n = 0 too)
  __device__ __forceinline__ int32_t step(int32_t pair) const { return pair < n ? n : 1; }
};

// What stands in a row of items in a kShared launch: a group's shared prefix, seen by all
// nodes of its sequences, or what one sequence has of its own.
struct Stretch {
  uint32_t cost;            // of all stretches before this one
  int32_t n;                // units of an item (0: no items)
  int32_t node0, nodes;     // its nodes, numbered through all sequences
  int32_t b;                // the sequence whose keys these are
  int32_t tile0, len;       // first key tile, and the end of the cached keys
  int32_t own;              // 0: a prefix
};

struct AttnPlan {
  AttnArgs a;
  int32_t tpt;              // nodes per row tile
  int32_t row_tiles, pairs; // row tiles, and pairs of them
  Lanes lanes;
  int32_t team;             // CTAs of a cluster that takes one item between them, or 0: runs
  int32_t areas;            // partial areas per slot (row tiles of a pair)
  float c;                  // scale * log2(e)
  float* part;              // [2 * runs][areas][D / 4][128] float4
  float2* part_ml;          // [2 * runs][areas][128] (m, l)
  int4* cuts;               // per run, of the item that it begins and does not end: sequence, head * pairs + pair,
                            // the last run with a part of it, the slot of its own part; or x = -1
  bool whole;               // runs take whole items (those that start in them)
  // kShared: the stretches and how many there are; sums of every row's first part, own keys and prefix, by row of the
  // output: O, and (m, l, its other parts).  `part` and `part_ml` then hold the other parts, one place a run:
  // [runs][2][128][D] and [runs][2][128].
  const Stretch* stretches;
  int32_t num_stretches;
  float* first_o[2];
  float4* first_ml[2];
  int32_t box_rows;         // rows of a K or V box
  uint32_t q_box_bytes;
};

// A chunk's S buffer, and how often that has been used before.
struct BufPos {
  int buf = 0;
  uint32_t use = 0;
  __device__ __forceinline__ void advance() {
    if (++buf == kBufs) {
      buf = 0;
      ++use;
    }
  }
  __device__ __forceinline__ BufPos before() const { return {buf == 0 ? kBufs - 1 : buf - 1, buf == 0 ? use - 1 : use}; }
};

// Key tiles of sequence b, the drafted one included (at least one, so that every row is written).
__device__ __forceinline__ int32_t units_of(const AttnArgs& a, int32_t b) {
  const int32_t n = kv_clamp(a.cache_len[b], a.cache.capacity, a.err);
  return max(1, (n + kTile - 1) / kTile + (a.k_new != nullptr ? 1 : 0));
}

// One item's stretch of a run.
template <Mode kMode>
struct Segment {
  int32_t b, h, pair;
  int32_t s, e, n;          // units [s, e) of n
  int32_t tiles;            // row tiles (2: one per pipeline; 1: shared by both)
  int32_t len;              // cached positions
  bool first;               // the run's first segment
  // kShared
  int32_t tile0, node0, nodes;
  uint32_t others;          // the item's runs, the first one and the last one (10 bits each)
  bool own;
  __device__ __forceinline__ int count() const { return e - s; }
  // first position of unit u, the item's nodes, and the first of them among all sequences'
  __device__ __forceinline__ int position(int u) const { return (kMode == kShared ? tile0 + u : u) * kTile; }
  __device__ __forceinline__ int num_nodes(const AttnArgs& a) const { return kMode == kShared ? nodes : a.T; }
  __device__ __forceinline__ int64_t node(const AttnArgs& a, int t) const {
    return kMode == kShared ? static_cast<int64_t>(node0) + t : static_cast<int64_t>(b) * a.T + t;
  }
  // keys of unit u: cached ones, or (the last unit, with drafted nodes) the nodes
  __device__ __forceinline__ bool drafted(const AttnArgs& a, int u) const {
    return a.k_new != nullptr && u == n - 1 && (kMode != kShared || own);
  }
  __device__ __forceinline__ int keys(const AttnArgs& a, int u) const {
    return drafted(a, u) ? a.T : max(0, min(kTile, len - position(u)));
  }
  // units that pipeline i takes
  __device__ __forceinline__ int count(int i) const { return tiles == 2 ? e - s : (e - s + 1 - i) >> 1; }
};

struct RunsWalk : RunWalk {
  bool begun = false;
  // The units of a team's item that are one CTA's.
  __device__ __forceinline__ void start_team(const AttnPlan& p, int32_t at, int32_t rank) {
    const int32_t per_seq = p.a.cache.heads * p.pairs;
    b = at / per_seq;
    item = at - b * per_seq;
    n = uniform(units_of(p.a, b));
    const int32_t share = team_share(p);
    s = min(n, rank * share);
    left = min(n - s, share);
  }
  __device__ __forceinline__ int32_t team_share(const AttnPlan& p) const { return (n + p.team - 1) / p.team; }
  template <Mode kMode>
  __device__ __forceinline__ bool next(const AttnPlan& p, Segment<kMode>* g) {
    const auto units = [&](int32_t i) { return units_of(p.a, i); };
    const int32_t per_seq = p.a.cache.heads * (p.lanes.n == 0 ? p.pairs : 1);
    if (left <= 0) return false;
    if (s == n) {
      next_item(units, per_seq);
    } else if (p.whole && s > 0) {   // the item is the run's that it starts in
      left -= n - s;
      if (left <= 0) return false;
      next_item(units, per_seq);
    }
    g->s = s;
    g->e = p.whole ? n : min(n, s + left);
    g->n = n;
    g->b = b;
    g->h = p.lanes.n == 0 ? item / p.pairs : item;
    g->pair = p.lanes.n == 0 ? item - g->h * p.pairs : p.lanes.pair(blockIdx.x);
    g->tiles = min(2, p.row_tiles - 2 * g->pair);
    g->len = uniform(kv_clamp(p.a.cache_len[b], p.a.cache.capacity, nullptr));
    g->first = !begun;
    begun = true;
    left -= g->e - s;
    s = g->e;
    return true;
  }
};

// A unit with one row tile takes about kSingle / kPair of the time of one with two (48 nodes, 3 row tiles, over
// 16384 and over 700 positions: 233 and 135 us; with 9 / 16 228 and 144, with 11 / 16 238 and 138).
constexpr int kSingle = 10, kPair = 16;

// Walks the units whose cost begins in [run * len, (run + 1) * len), of all stretches' items in order: kv head
// by kv head, pair of row tiles by pair.
struct CostWalk {
  uint32_t at, end, len;    // cost at which the item begins; the run's end; a run's length
  int32_t v, item, s, w;    // stretch, item of it, next unit, cost of a unit
  int32_t tiles, pairs;     // row tiles of the stretch's items
  Stretch st;
  int32_t left;             // whether units are left (0: no)
  bool begun = false;
  __device__ __forceinline__ void take(const AttnPlan& p) {
    st = p.stretches[v];
    tiles = (st.nodes + p.tpt - 1) / p.tpt;
    pairs = (tiles + 1) >> 1;
  }
  __device__ __forceinline__ void weigh() { w = 2 * (item % pairs) + 1 == tiles ? kSingle : kPair; }
  // Whole warp.
  __device__ __forceinline__ void start(const AttnPlan& p, uint32_t run, uint32_t runs) {
    const int lane = threadIdx.x & 31;
    const uint32_t total = p.stretches[p.num_stretches].cost;
    // at least a unit's cost: then a unit of the item begins in every run from an item's first one to its last
    len = max((total + runs - 1) / runs, static_cast<uint32_t>(kPair));
    const uint32_t from = min(total, run * len);
    end = min(total, from + len);
    left = from < total;
    if (left == 0) return;
    // the last stretch that begins at or before `from`: 32 places of the range at a time (costs rise strictly but
    // over stretches without items, of which the last one is then the one with items)
    int32_t lo = 0, hi = p.num_stretches;
    while (hi - lo > 1) {
      const int32_t step = (hi - lo + 31) >> 5, x = lo + lane * step;
      const uint32_t before = __ballot_sync(0xFFFFFFFFu, x < hi && p.stretches[x].cost <= from);
      const int last = 31 - __clz(before);            // lane 0's place is always before
      lo += last * step;
      hi = min(hi, lo + step);
    }
    v = lo;
    take(p);
    const uint32_t per_head = static_cast<uint32_t>(st.n) * (kPair * (tiles >> 1) + kSingle * (tiles & 1));
    uint32_t rel = from - st.cost;
    const uint32_t h = rel / per_head;
    rel -= h * per_head;
    const uint32_t pair = min(rel / (kPair * static_cast<uint32_t>(st.n)), static_cast<uint32_t>(pairs - 1));
    rel -= pair * kPair * st.n;
    item = static_cast<int32_t>(h) * pairs + static_cast<int32_t>(pair);
    weigh();
    s = static_cast<int32_t>((rel + w - 1) / w);      // (st.n where the item's last unit began before)
    at = from - rel;
  }
  __device__ __forceinline__ bool next(const AttnPlan& p, Segment<kShared>* g) {
    if (left == 0) return false;
    if (s == st.n) {
      at += static_cast<uint32_t>(st.n) * w;
      s = 0;
      if (++item == p.a.cache.heads * pairs) {
        if (at >= end) {
          left = 0;
          return false;
        }
        item = 0;
        do {
          ++v;
          take(p);
        } while (st.n == 0);
      }
      weigh();
    }
    if (at + static_cast<uint32_t>(s) * w >= end) {
      left = 0;
      return false;
    }
    g->s = s;
    g->n = st.n;
    g->e = static_cast<int32_t>(min(static_cast<uint32_t>(st.n), (end - at + w - 1) / w));
    g->b = st.b;
    g->h = item / pairs;
    g->pair = item - g->h * pairs;
    g->tiles = min(2, tiles - 2 * g->pair);
    g->len = st.len;
    g->first = !begun;
    g->tile0 = st.tile0;
    g->node0 = st.node0;
    g->nodes = st.nodes;
    g->own = st.own != 0;
    g->others = at / len | (at + static_cast<uint32_t>(st.n - 1) * w) / len << 10;
    begun = true;
    s = g->e;
    if (at + static_cast<uint32_t>(s) * w >= end) left = 0;
    return true;
  }
};

template <Mode kMode>
struct WalkOf {
  using type = RunsWalk;
};
template <>
struct WalkOf<kShared> {
  using type = CostWalk;
};

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ bool finite_bf16(uint32_t bits) { return (bits & 0x7F80u) != 0x7F80u; }

// Zeroes the rows [from, to) of a V tile (this thread's share of `threads`).
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int to, int tid, int threads) {
  const int n = (to - from) * 8;   // 16-byte pieces per column block
#pragma unroll
  for (int half = 0; half < Cfg<D>::kHalves; ++half)
    for (int x = tid; x < n; x += threads)
      *reinterpret_cast<uint4*>(tile + half * kTile * 128 + from * 128 + x * 16) = make_uint4(0, 0, 0, 0);
}

// The warp's rows of O (`cols` columns at tm) times f.  Out of line: it is rarely called.
__device__ __noinline__ void rescale_rows(uint32_t tm, int cols, float f) {
#pragma unroll 1
  for (int x = 0; x < cols; x += 32) {
    float o[32];
    tmem_ld_x32(tm + x, o);
    tmem_ld_wait();
    pin(o);
#pragma unroll
    for (int w = 0; w < 32; w += 16) {
      uint32_t ob[16];
#pragma unroll
      for (int y = 0; y < 16; ++y) ob[y] = __float_as_uint(o[w + y] * f);
      tmem_st_x16(tm + x + w, ob);
    }
  }
}

// A sum's part v, to be weighted by f >= 0.  An infinity stays one where f underflows
// (the weights of the definition do not).
__device__ __forceinline__ float weighted(float v, float f) { return fabsf(v) < INFINITY ? v * f : v; }

// Where a segment's sums go: to the output, or to its parts, a run's in the workspace
// (the first segment's in slot 2 c, another's in 2 c + 1), a team's CTA's in its ring.  With kShared
// always to parts: an item's first one by row of the output, another in the run's place.
template <int D, Mode kMode>
struct PartPlace {
  bool whole;
  int slot;
  float4* parts;
  float2* mls;
  __device__ __forceinline__ PartPlace(const AttnPlan& p, const Segment<kMode>& g, uint8_t* ring)
      : whole(kMode == kRuns && g.s == 0 && g.e == g.n),
        slot(kMode == kTeam     ? 0
             : kMode == kShared ? static_cast<int>(blockIdx.x)
                                : 2 * static_cast<int>(blockIdx.x) + (g.first ? 0 : 1)),
        parts(reinterpret_cast<float4*>(kMode == kTeam ? ring : reinterpret_cast<uint8_t*>(p.part))),
        mls(kMode == kTeam ? reinterpret_cast<float2*>(ring + 2 * kTile * D * 4) : p.part_ml) {}
  // Row r's O in the tile, its first four columns; the next four are kStep float4 on.  orow: its row of the output.
  static constexpr int kStep = kMode == kShared ? 1 : kTile;
  __device__ __forceinline__ float4* part(const AttnPlan& p, const Segment<kMode>& g, int tile, int r, int64_t orow) const {
    if constexpr (kMode == kShared) {
      if (g.s == 0) return reinterpret_cast<float4*>(p.first_o[g.own ? 0 : 1]) + orow * (D / 4);
      return parts + ((static_cast<int64_t>(slot) * 2 + tile) * kTile + r) * (D / 4);
    } else {
      return parts + (static_cast<int64_t>(slot) * p.areas + tile) * (D / 4) * kTile + r;
    }
  }
  // Its m and l.
  __device__ __forceinline__ void put_ml(const AttnPlan& p, const Segment<kMode>& g, int tile, int r, int64_t orow, float m,
                                         float l) const {
    if constexpr (kMode == kShared) {
      if (g.s == 0)
        p.first_ml[g.own ? 0 : 1][orow] = make_float4(m, l, __uint_as_float(g.others | (tile * kTile + r) << 20), 0.0f);
      else
        mls[(static_cast<int64_t>(slot) * 2 + tile) * kTile + r] = make_float2(m, l);
    } else {
      mls[(static_cast<int64_t>(slot) * p.areas + tile) * kTile + r] = make_float2(m, l);
    }
  }
};

// <q, k> over D bf16 each.
template <int D>
__device__ __forceinline__ float dot_bf16(const uint16_t* q, const uint16_t* k) {
  float z = 0.0f;
#pragma unroll 4
  for (int x = 0; x < D; x += 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(q + x), b = *reinterpret_cast<const uint4*>(k + x);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      z = fmaf(bf16_bits_to_float(u[y]), bf16_bits_to_float(w[y]), z);
      z = fmaf(__uint_as_float(u[y] & 0xFFFF0000u), __uint_as_float(w[y] & 0xFFFF0000u), z);
    }
  }
  return z;
}

// Takes the sums of the run's rows that hold a non-finite value again, each by a warp of
// the softmax: 32 keys at a time, a lane each, then all lanes on each key's value.  Out of
// line: it is hardly ever called.
template <int D, Mode kMode>
__device__ __noinline__ void sum_again(const AttnPlan& p, typename WalkOf<kMode>::type walk, uint8_t* ring) {
  constexpr int E = D / 32;              // columns of a lane
  const AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  Segment<kMode> g;
  while (walk.next(p, &g)) {
    const PartPlace<D, kMode> place(p, g, ring);
    for (int tile = 0; tile < g.tiles; ++tile) {
      const int node0 = (2 * g.pair + tile) * p.tpt, rows = min(p.tpt, g.num_nodes(a) - node0) * a.group;
#pragma unroll 1
      for (int r = (threadIdx.x >> 5) - 4; r < rows; r += 2 * kTile / 32) {
        const int t = r / a.group, node = node0 + t, hq = g.h * a.group + r - t * a.group;
        const int64_t orow = g.node(a, node) * a.heads + hq;
        uint16_t* out = a.out + orow * D + lane * E;
        float* part = reinterpret_cast<float*>(place.part(p, g, tile, r, orow) + lane * E / 4 * place.kStep) + lane * E % 4;
        bool finite = true;
#pragma unroll
        for (int e = 0; e < E; ++e) finite &= place.whole ? finite_bf16(out[e]) : fabsf(part[e]) < INFINITY;
        if (__all_sync(0xFFFFFFFFu, finite)) continue;
        const uint16_t* q = a.q + (kMode == kShared ? g.node(a, node) * a.q_t : g.b * a.q_b + node * a.q_t) + hq * a.q_h;
        float m = -INFINITY, l = 0.0f, o[E] = {};   // l: of the lane's keys
#pragma unroll 1
        for (int u = g.s; u < g.e; ++u) {
          const bool drafted = g.drafted(a, u);
          const int keys = g.keys(a, u);
#pragma unroll 1
          for (int x = lane; x - lane < keys; x += 32) {
            bool adds = x < keys;
            if (adds && drafted)
              adds = a.mask == nullptr ? x <= node
                                       : a.mask[(static_cast<int64_t>(g.b) * a.T + node) * ((a.T + 63) >> 6) + (x >> 6)] >>
                                                 (x & 63) & 1;
            const uint16_t* v = nullptr;
            float z = -INFINITY;
            if (adds) {
              bool ok;
              const int64_t at = drafted ? g.b * a.new_b + x * a.new_t + g.h * a.new_h
                                         : kv_offset(a.cache, g.b, g.position(u) + x, g.h, nullptr, &ok);
              v = (drafted ? a.v_new : a.cache.v) + at;
              z = dot_bf16<D>(q, (drafted ? a.k_new : a.cache.k) + at);
              adds = z * a.scale != -INFINITY;
            }
            float top = m;
            if (adds) top = fmaxf(top, z * p.c);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            const float f = m == -INFINITY ? 1.0f : exp2_approx(m - top);
            const float w = adds ? exp2_approx(fmaf(z, p.c, top == -INFINITY ? 0.0f : -top)) : 0.0f;
            m = top;
            l = l * f + w;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = weighted(o[e], f);
            for (uint32_t some = __ballot_sync(0xFFFFFFFFu, adds); some != 0; some &= some - 1) {
              const int y = __ffs(some) - 1;
              const auto* vy =
                  reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(v), y));
              const float wy = __shfl_sync(0xFFFFFFFFu, w, y);
#pragma unroll
              for (int e = 0; e < E; ++e) o[e] += weighted(bf16_bits_to_float(vy[lane * E + e]), wy);
            }
          }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        if (place.whole) {
#pragma unroll
          for (int e = 0; e < E; ++e) out[e] = __bfloat16_as_ushort(__float2bfloat16_rn(l == 0.0f ? 0.0f : o[e] / l));
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) part[e] = o[e];
          if (lane == 0) place.put_ml(p, g, tile, r, orow, m, -l);     // (see PartSum::add)
        }
      }
    }
  }
}

// Partial sums of a row's N columns, added as the softmax adds keys.
template <int N>
struct PartSum {
  float m = -INFINITY, l = 0.0f, o[N] = {};
  bool odd = false;          // whether an infinity may be in o
  // Adds sums (m1, l1, v); with m1 = -inf they saw nothing, and v is not looked at.
  // A negative l1 says that v may hold infinities.
  __device__ __forceinline__ void add(float m1, float l1, const float (&v)[N]) {
    odd |= l1 < 0.0f;
    l1 = fabsf(l1);
    const bool some = m1 != -INFINITY;
    const float top = fmaxf(m, m1);
    // an infinity stays one where its weight underflows: that of the definition does not
    const float least = odd ? 1.4e-45f : 0.0f;
    const float f0 = m == -INFINITY ? 0.0f : fmaxf(exp2_approx(m - top), least);
    const float f1 = some ? fmaxf(exp2_approx(m1 - top), least) : 0.0f;
    m = top;
    l = l * f0 + (some || l1 != l1 ? l1 * (some ? f1 : 1.0f) : 0.0f);   // only NaN scores: l1 is NaN
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = fmaf(some ? v[k] : 0.0f, f1, o[k] * f0);
  }
  // Row r's parts of columns x.. in runs c, c + step, .. c1, kBatch loads at a time.
  template <int D, int kBatch>
  __device__ __forceinline__ void add_parts(const AttnPlan& p, const int4& d, int c0, int c, int step, int tile, int x,
                                            int r) {
    for (; c <= d.z; c += kBatch * step) {
      float2 ml[kBatch];
      float v[kBatch][N];
#pragma unroll
      for (int w = 0; w < kBatch; ++w) {
        const int cw = c + w * step;
        ml[w] = make_float2(-INFINITY, 0.0f);
        if (cw > d.z) continue;
        // a run's first segment leaves its parts in slot 2 c, its last one in 2 c + 1
        const int64_t part = static_cast<int64_t>(cw == c0 ? d.w : 2 * cw) * p.areas + tile;
        ml[w] = p.part_ml[part * kTile + r];
        const float4* src = reinterpret_cast<const float4*>(p.part) + (part * (D / 4) + x / 4) * kTile + r;
#pragma unroll
        for (int k = 0; k < N; k += 4) *reinterpret_cast<float4*>(&v[w][k]) = src[k / 4 * kTile];
      }
#pragma unroll
      for (int w = 0; w < kBatch; ++w)
        if (c + w * step <= d.z) add(ml[w].x, ml[w].y, v[w]);
    }
  }
  __device__ __forceinline__ void write(const AttnArgs& a, int64_t orow, int D, int x) const {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t out[N / 2];
#pragma unroll
    for (int k = 0; k < N; k += 2) out[k / 2] = pack_bf16(o[k] * inv, o[k + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + x);
    if constexpr (N == 8)
      *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    else if constexpr (N == 2)
      *dst = out[0];
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    if (x == 0 && a.lse != nullptr) a.lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
};

// Two or four words at p of the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ float2 ld_cluster(const float2* p, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster(const float4* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr(p, rank))
               : "memory");
  return v;
}

// Adds the parts that a team's CTAs left in their shared memory, in their order: each CTA
// takes every team-th four columns, a thread four columns of a row at a time.
template <int D>
__device__ __forceinline__ void join_team(const AttnPlan& p, const RunsWalk& walk, const uint8_t* ring) {
  const AttnArgs& a = p.a;
  const float4* parts = reinterpret_cast<const float4*>(ring);
  const float2* part_ml = reinterpret_cast<const float2*>(ring + 2 * kTile * D * 4);
  const int share = walk.team_share(p), ranks = (walk.n + share - 1) / share;
  const int h = walk.item / p.pairs, pair = walk.item - h * p.pairs;
  for (int tile = 0; tile < 2; ++tile) {
    const int node0 = (2 * pair + tile) * p.tpt;
    const int rows = min(p.tpt, a.T - node0) * a.group;      // (none: the pair has one tile)
    for (int task = threadIdx.x; task < rows * (D / 4) / p.team; task += kThreads) {
      const int y = task / rows, r = task - y * rows;
      const int x = y * p.team + blockIdx.x % p.team;
      const int t = r / a.group;
      PartSum<4> sum;
      float2 ml[kMaxTeam];
      float v[kMaxTeam][4];
#pragma unroll
      for (int w = 0; w < kMaxTeam; ++w) {
        if (w >= ranks) continue;
        ml[w] = ld_cluster(&part_ml[tile * kTile + r], w);
        *reinterpret_cast<float4*>(v[w]) = ld_cluster(&parts[(tile * (D / 4) + x) * kTile + r], w);
      }
#pragma unroll
      for (int w = 0; w < kMaxTeam; ++w)
        if (w < ranks) sum.add(ml[w].x, ml[w].y, v[w]);
      sum.write(a, (static_cast<int64_t>(walk.b) * a.T + node0 + t) * a.heads + h * a.group + r - t * a.group, D, 4 * x);
    }
  }
}

// 227 KB, the opt-in limit of a block, is just enough at D = 128
static_assert(Cfg<128>::kRing + sizeof(AttnSmem) <= 232448, "shared memory");

template <int D, Mode kMode>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKn,
                     const __grid_constant__ CUtensorMap tmVn, const __grid_constant__ AttnPlan p) {
  using C = Cfg<D>;
  constexpr int S = C::kSlots;
  extern __shared__ __align__(1024) uint8_t q_smem[];   // no static shared memory: the base is 1024-byte aligned
  uint8_t* ring = q_smem + 2 * C::kTileBytes;
  AttnSmem& s = *reinterpret_cast<AttnSmem*>(q_smem + C::kRing);
  const AttnArgs& a = p.a;
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  volatile int* abort_flag = &s.abort_flag;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&s.kv_full[2 * i], 1);
      mbar_init(&s.kv_full[2 * i + 1], 1);
      mbar_init(&s.kv_empty[i], 2);
    }
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      for (int buf = 0; buf < kBufs; ++buf) {
        mbar_init(&s.s_full[i][buf], 1);
        mbar_init(&s.p_ready[i][buf], kTile);
        mbar_init(&s.pv_done[i][buf], 1);
      }
    }
    mbar_init(&s.drain, 4);
    s.abort_flag = 0;
    s.odd = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmKn);
    tma_prefetch_desc(&tmVn);
  }
  if (warp == 0) {
    tmem_alloc(&s.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s.tmem);
  pdl_wait();
  pdl_launch_dependents();
  typename WalkOf<kMode>::type walk;
  RunStart run = {0, 0, 0, 0};
  if constexpr (kMode == kShared) {
    walk.start(p, blockIdx.x, gridDim.x);
  } else if constexpr (kMode == kTeam) {
    walk.start_team(p, blockIdx.x / p.team, blockIdx.x % p.team);
  } else {
    int32_t run_at = blockIdx.x, runs = gridDim.x, per_seq = a.cache.heads * p.pairs;
    if (p.lanes.n > 0) {
      const int32_t dealt = p.lanes.n * p.lanes.runs;
      per_seq = a.cache.heads;
      runs = run_at < dealt ? p.lanes.runs : runs - dealt;
      run_at = run_at < dealt ? run_at / p.lanes.n : run_at - dealt;
    }
    run = find_run([&](int32_t b) { return units_of(a, b); }, static_cast<int32_t>(a.B), per_seq, run_at, runs);
    walk.start(run);
    if (threadIdx.x == 0 && run.units == 0) p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  Segment<kMode> g;
  bool live = true;

  if (warp == 0) {
    // ---- producer ----
    RingPos<S> at;
    uint32_t issued = 0;  // tiles whose copies were started
    int seg = 0, q_issued = 0;
    PageFeed pages;
    for (; walk.next(p, &g); ++seg) {
      if (seg > 0) wait_live(&s.q_empty, (seg - 1) & 1, &live, abort_flag, a.err);
      live = __all_sync(0xFFFFFFFFu, live);
      if (live) q_issued = seg + 1;
      if (lane == 0 && live) {
        mbar_arrive_expect_tx(&s.q_full, g.tiles * p.q_box_bytes);
        for (int i = 0; i < g.tiles; ++i)
          for (int half = 0; half < C::kHalves; ++half)
            tma_load_5d(q_smem + i * C::kTileBytes + half * kTile * 128, &tmQ, half * 64, 0,
                        (kMode == kShared ? g.node0 : 0) + (2 * g.pair + i) * p.tpt, g.h, kMode == kShared ? 0 : g.b,
                        &s.q_full);
      }
      __syncwarp();
      // lane -> (page piece of the tile, column block)
      const int half = lane % C::kHalves, piece = lane / C::kHalves;
      const int row = piece * p.box_rows;       // first row of the lane's box
      pages.start(a.cache, g.b, kMode == kShared ? g.tile0 + g.s : g.s, g.len, lane);
      for (int u = g.s; u < g.e; ++u) {
        const bool drafted = g.drafted(a, u);
        bool has;
        int y = 0, z = g.h, w = g.b;
        uint32_t bytes;
        if (drafted) {
          has = lane < C::kHalves;
          bytes = kTile * 128;
        } else {
          const int j = g.position(u) + row;
          has = row < kTile && j < g.len;
          bytes = p.box_rows * 128;
          y = j;
          if (pages.row != nullptr) {
            w = pages.page(a.cache, g.position(u), j, has, lane, a.err);
            y = j & (a.cache.page_size - 1);
          }
        }
        const uint32_t boxes = __popc(__ballot_sync(0xFFFFFFFFu, has));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, at.advance(1)) {
          const uint32_t slot = at.slot;
          if (at.use > 0) wait_live(&s.kv_empty[slot], (at.use - 1) & 1, &live, abort_flag, a.err);
          live = __all_sync(0xFFFFFFFFu, live);
          if (!live) continue;
          ++issued;
          uint64_t* full = at.full(s.kv_full);
          if (lane == 0) mbar_arrive_expect_tx(full, boxes * bytes);
          __syncwarp();
          if (has)
            tma_load_4d(ring + slot * C::kTileBytes + half * kTile * 128 + (drafted ? 0 : row * 128),
                        drafted ? (kv ? &tmVn : &tmKn) : (kv ? &tmV : &tmK), half * 64, y, z, w, full);
        }
      }
    }
    // after a wait that gave up: this CTA's copies have landed before it exits (else the products have used them)
    if (lane == 0 && !live) {
      if (q_issued > 0) mbar_wait_bounded(&s.q_full, (q_issued - 1) & 1, a.err);
      RingPos<S> last;
      const uint32_t first = issued > S ? issued - S : 0;
      last.advance_far(first);
      for (uint32_t j = first; j < issued; ++j, last.advance(1))
        mbar_wait_bounded(last.full(s.kv_full), last.parity(), a.err);
    }
    __syncwarp();
  } else if (warp <= 2) {
    // ---- S products of pipeline i ----
    const int i = warp - 1;
    const uint32_t elected = elect_lane();
    const uint32_t tm_s = tmem + i * kBufs * kChunk;
    const uint32_t idesc = umma_idesc_bf16(128, kChunk);
    const uint32_t ring_addr = uniform(smem_addr(ring)), q_addr = uniform(smem_addr(q_smem));
    RingPos<S> seg_k;            // the segment's first K tile
    BufPos at_s;       // the pipeline's next chunk
    int seg = 0;
    for (; walk.next(p, &g); ++seg) {
      const int step = g.tiles == 2 ? 1 : 2, off = g.tiles == 2 ? 0 : i;
      const int cnt = g.count(i);
      RingPos<S> at = seg_k;
      at.advance(2 * off);
      wait_live(&s.q_full, seg & 1, &live, abort_flag, a.err);
      __syncwarp();
      if (cnt == 0 && elected) mbar_arrive(&s.q_empty);
      const uint32_t q_lo = desc_lo(q_addr + (g.tiles == 2 ? i : 0) * C::kTileBytes);
      for (int j = 0; j < cnt; ++j) {
        const int chunks = g.keys(a, g.s + j * step + off) <= kChunk ? 1 : 2;
        const uint32_t k_lo = desc_lo(ring_addr + at.slot * C::kTileBytes);
        wait_live(at.full(s.kv_full), at.parity(), &live, abort_flag, a.err);
        for (int c = 0; c < chunks; ++c, at_s.advance()) {
          const int buf = at_s.buf;
          // P of the chunk that had the buffer lies in it until its product is done
          if (at_s.use > 0) wait_live(&s.pv_done[i][buf], (at_s.use - 1) & 1, &live, abort_flag, a.err);
          __syncwarp();
          tc_fence_after();
          const uint32_t lead = live ? elected : 0u;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = ((k >> 2) * kTile * 128 + (k & 3) * 32) >> 4;
            umma_ss(tm_s + buf * kChunk, q_lo + o, k_lo + ((c * kChunk * 128) >> 4) + o, idesc, k > 0 ? 1u : 0u, lead);
          }
          umma_commit_if(&s.s_full[i][buf], lead);
        }
        // a tile goes back after two releases: one per pipeline, or both by the one that has it to itself
        const uint32_t lead = live ? elected : 0u;
        umma_commit_if(&s.kv_empty[at.slot], lead);
        if (g.tiles == 1) umma_commit_if(&s.kv_empty[at.slot], lead);
        if (j == cnt - 1) umma_commit_if(&s.q_empty, lead);
        at.advance(2 * step);
      }
      seg_k.advance_far(2 * g.count());
    }
    umma_commit_if(&s.drain, elected);
    __syncwarp();
  } else if (warp == 3 || warp == 12) {
    // ---- O products of pipeline i ----
    const int i = warp == 3 ? 0 : 1;
    const uint32_t elected = elect_lane();
    const uint32_t tm_s = tmem + i * kBufs * kChunk, tm_o = tmem + kTmemO + i * D;
    const uint32_t idesc = umma_idesc_bf16(128, D) | (1u << 16);   // B is MN-major
    const uint32_t ring_addr = uniform(smem_addr(ring));
    RingPos<S> seg_v;            // the segment's first V tile
    seg_v.advance(1);
    BufPos at_s;
    while (walk.next(p, &g)) {
      const int step = g.tiles == 2 ? 1 : 2, off = g.tiles == 2 ? 0 : i;
      const int cnt = g.count(i);
      RingPos<S> at = seg_v;
      at.advance(2 * off);
      for (int j = 0; j < cnt; ++j) {
        const int chunks = g.keys(a, g.s + j * step + off) <= kChunk ? 1 : 2;
        const uint32_t v_lo = desc_lo(ring_addr + at.slot * C::kTileBytes, kTile * 128);
        for (int c = 0; c < chunks; ++c, at_s.advance()) {
          const int buf = at_s.buf;
          wait_live(&s.p_ready[i][buf], at_s.use & 1, &live, abort_flag, a.err);
          if (c == 0) wait_live(at.full(s.kv_full), at.parity(), &live, abort_flag, a.err);
          __syncwarp();
          tc_fence_after();
          const uint32_t lead = live ? elected : 0u;
          const uint32_t v_c = v_lo + c * ((kChunk * 128) >> 4), tm_p = tm_s + buf * kChunk;
#pragma unroll
          for (int k = 0; k < kChunk / 16; ++k)
            umma_ts(tm_o, tm_p + k * 8, v_c + k * (2048 >> 4), idesc, (j > 0 || c > 0 || k > 0) ? 1u : 0u, lead);
#pragma unroll
          for (int k = 0; k < kChunk / 16; ++k)
            umma_ts(tm_o, tm_p + kChunk / 2 + k * 8, v_c + k * (2048 >> 4), idesc, 1u, lead);
          umma_commit_if(&s.pv_done[i][buf], lead);
        }
        const uint32_t lead = live ? elected : 0u;
        umma_commit_if(&s.kv_empty[at.slot], lead);
        if (g.tiles == 1) umma_commit_if(&s.kv_empty[at.slot], lead);
        at.advance(2 * step);
      }
      seg_v.advance_far(2 * g.count());
    }
    umma_commit_if(&s.drain, elected);
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ---- softmax of pipeline i, one row per thread ----
    const int i = warp >= 8 ? 1 : 0;
    const int r = threadIdx.x & (kTile - 1);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + i * kBufs * kChunk + lanes, tm_o = tmem + kTmemO + lanes;
    RingPos<S> seg_v;            // the segment's first V tile
    seg_v.advance(1);
    BufPos at_s;       // the pipeline's next chunk
    const int t_r = r / a.group;
    for (; walk.next(p, &g);) {
      const int step = g.tiles == 2 ? 1 : 2, off = g.tiles == 2 ? 0 : i;
      const int cnt = g.count(i);
      const int node = (2 * g.pair + (g.tiles == 2 ? i : 0)) * p.tpt + t_r;
      const bool row_ok = r < p.tpt * a.group && node < g.num_nodes(a);
      // a warp none of whose rows is a query's has nothing to do but to keep step
      const bool busy = (warp & 3) * 32 < min(p.tpt, g.num_nodes(a) - (node - t_r)) * a.group;
      float m = -INFINITY, l = 0.0f;
      uint32_t vis[4] = {0, 0, 0, 0}, bad_seen = 0;   // the drafted tile's mask; whether a visible node is non-finite
      for (int j = 0; j < cnt; ++j) {
        const int u = g.s + j * step + off;
        const bool drafted = g.drafted(a, u);
        const int valid = g.keys(a, u);
        const int chunks = valid <= kChunk ? 1 : 2;
        const bool partial_tile = drafted || valid < chunks * kChunk;
        wait_live(&s.s_full[i][at_s.buf], at_s.use & 1, &live, abort_flag, a.err);
        if (partial_tile) {
          // what the row sees of the tile, and a V tile without what nobody may see
          RingPos<S> at_v = seg_v;
          at_v.advance_far(2 * (j * step + off));
          uint8_t* v_tile = ring + at_v.slot * C::kTileBytes;
          wait_live(at_v.full(s.kv_full), at_v.parity(), &live, abort_flag, a.err);
          const int upto = drafted && a.mask == nullptr ? min(valid, node + 1) : valid;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int k = upto - 32 * w;
            vis[w] = k >= 32 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << k) - 1u;
          }
          if (drafted) {
            if (a.mask != nullptr) {
              const int words = (a.T + 63) >> 6;
              const uint64_t* mk = a.mask + (static_cast<int64_t>(g.b) * a.T + node) * words;
              const uint64_t w0 = row_ok ? mk[0] : 0ull, w1 = row_ok && words > 1 ? mk[1] : 0ull;
              vis[0] &= static_cast<uint32_t>(w0);
              vis[1] &= static_cast<uint32_t>(w0 >> 32);
              vis[2] &= static_cast<uint32_t>(w1);
              vis[3] &= static_cast<uint32_t>(w1 >> 32);
            }
            // the pipelines that take the drafted tile look through it together
            const int threads = g.tiles == 2 ? 2 * kTile : kTile;
            const int tid = g.tiles == 2 ? static_cast<int>(threadIdx.x) - kTile : r;
            const int bar = g.tiles == 2 ? 1 : 2 + i;
            if (tid < 4) s.bad[tid] = 0;
            __syncwarp();
            named_bar_sync(bar, threads);
#pragma unroll
            for (int half = 0; half < C::kHalves; ++half)
              for (int x = tid; x < a.T * 8; x += threads) {
                uint4* at = reinterpret_cast<uint4*>(v_tile + half * kTile * 128 + x * 16);
                uint4 q = *at;
                uint32_t* e = &q.x;
                bool hit = false;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  if (!finite_bf16(e[y])) e[y] &= 0xFFFF0000u, hit = true;
                  if (!finite_bf16(e[y] >> 16)) e[y] &= 0x0000FFFFu, hit = true;
                }
                if (hit) {
                  *at = q;
                  atomicOr(&s.bad[x >> 8], 1u << ((x >> 3) & 31));
                }
              }
            __syncwarp();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            named_bar_sync(bar, threads);
#pragma unroll
            for (int w = 0; w < 4; ++w) bad_seen |= vis[w] & s.bad[w];
          } else {
            zero_rows<D>(v_tile, valid, chunks * kChunk, r, kTile);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
#pragma unroll 1
        for (int c = 0; c < chunks; ++c, at_s.advance()) {
          const int buf = at_s.buf;
          const uint32_t tm_sb = tm_s + buf * kChunk;
          if (c > 0) wait_live(&s.s_full[i][buf], at_s.use & 1, &live, abort_flag, a.err);
          __syncwarp();
          tc_fence_after();
          if (busy) {
            float z[2][32];
            tmem_ld_x32(tm_sb, z[0]);
            tmem_ld_x32(tm_sb + 32, z[1]);
            tmem_ld_wait();
            pin(z[0]);
            pin(z[1]);
            if (partial_tile) {
              const uint32_t v0 = c ? vis[2] : vis[0], v1 = c ? vis[3] : vis[1];
#pragma unroll
              for (int y = 0; y < 32; ++y) {
                if (!(v0 >> y & 1u)) z[0][y] = -INFINITY;
                if (!(v1 >> y & 1u)) z[1][y] = -INFINITY;
              }
            }
            float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // four chains of dependent maxima
#pragma unroll
            for (int y = 0; y < 32; ++y) tops[y & 3] = fmaxf(tops[y & 3], fmaxf(z[0][y], z[1][y]));
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * p.c;
            if (j == 0 && c == 0) {
              m = top;
            } else if (__any_sync(0xFFFFFFFFu, row_ok && top > m + kRescale)) {
              // a row's maximum rose far: the warp's O and l move to the new ones (rows of the
              // tile that are no query's hold whatever shared memory held, and have no say)
              const float m1 = fmaxf(m, top);
              const float f = m == -INFINITY ? 1.0f : exp2_approx(m - m1);
              m = m1;
              l *= f;
              const BufPos prev = at_s.before();
              wait_live(&s.pv_done[i][prev.buf], prev.use & 1, &live, abort_flag, a.err);
              __syncwarp();
              tc_fence_after();
              rescale_rows(tm_o + i * D, D, f);
            }
            const float mm = m == -INFINITY ? 0.0f : m;   // a row that has seen nothing: all its P are 2^-inf
            const uint64_t c2 = pack2(p.c, p.c), m2 = pack2(-mm, -mm);
            uint64_t sum0 = pack2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int y = 0; y < 32; y += 2) {
                const float2 e = unpack2(fma2(pack2(z[x][y], z[x][y + 1]), c2, m2));
                const float p0 = exp2_approx(e.x), p1 = exp2_approx(e.y);
                const uint64_t pp = pack2(p0, p1);
                if (y & 2)
                  sum1 = add2(sum1, pp);
                else
                  sum0 = add2(sum0, pp);
                // what P loses when it is rounded to bf16 is the second term
                const uint32_t h = pack_bf16(p0, p1);
                const float2 d = unpack2(add2(pp, pack2(-__uint_as_float(h << 16), -__uint_as_float(h & 0xFFFF0000u))));
                hi[y / 2] = h;
                lo[y / 2] = pack_bf16(d.x, d.y);
              }
              tmem_st_x16(tm_sb + 16 * x, hi);
              tmem_st_x16(tm_sb + kChunk / 2 + 16 * x, lo);
            }
            const float2 sum = unpack2(add2(sum0, sum1));
            l += sum.x + sum.y;
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&s.p_ready[i][buf]);
        }
      }
      seg_v.advance_far(2 * g.count());

      // ---- the item's (or the run's part of the item's) sums ----
      const PartPlace<D, kMode> place(p, g, ring);
      const bool whole = place.whole;
      const bool merge = g.tiles == 1;
      float f0 = 1.0f, f1 = 0.0f;     // weights of O0 and O1 (one tile), or of O_i
      // products complete in the order of their issue: the last one's is enough
      const BufPos prev = at_s.before();
      if (cnt > 0) wait_live(&s.pv_done[i][prev.buf], prev.use & 1, &live, abort_flag, a.err);
      __syncwarp();
      if (merge) {
        // each pipeline has waited for its own products
        s.ml[i][r] = make_float2(m, l);
        tc_fence_before();
        named_bar_sync(1, 2 * kTile);
        const float2 x0 = s.ml[0][r], x1 = s.ml[1][r];
        m = fmaxf(x0.x, x1.x);
        f0 = x0.x == -INFINITY ? 0.0f : exp2_approx(x0.x - m);
        f1 = x1.x == -INFINITY ? 0.0f : exp2_approx(x1.x - m);
        l = x0.y * f0 + x1.y * f1;
        // a row that only saw NaN scores has no maximum and a NaN sum
        if (x0.y != x0.y || x1.y != x1.y) l = f0 = NAN;
        if (g.count(1) == 0) f1 = 0.0f;
      } else if (kMode == kTeam) {
        named_bar_sync(1, 2 * kTile);     // the parts go where the other pipeline's tiles were
      }
      tc_fence_after();
      const bool empty = l == 0.0f;   // the row saw nothing: 0, whatever the values were
      const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
      f0 *= inv;
      f1 *= inv;
      const int c0 = merge ? i * (D / 2) : 0, c1 = merge ? c0 + D / 2 : D;
      const int64_t orow = g.node(a, node) * a.heads + g.h * a.group + r % a.group;
      const int area = merge ? 0 : i;
      if (!merge || i == 0) {
        if (whole) {
          if (row_ok && a.lse != nullptr)
            a.lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        } else if (kMode != kShared || row_ok) {
          place.put_ml(p, g, area, r, orow, m, l);
        }
      }
      if (kMode == kRuns && threadIdx.x == kTile && walk.left <= 0)        // the run's last segment
        p.cuts[blockIdx.x] =
            g.s == 0 && g.e < g.n
                ? make_int4(g.b, g.h * p.pairs + g.pair,
                            static_cast<int>(blockIdx.x) +
                                p.lanes.step(g.pair) * ((g.n - g.e + run.units - 1) / run.units),
                            place.slot)
                : make_int4(-1, 0, 0, 0);
      uint64_t odd[4] = {};           // 0, or NaN once an element of O is not finite (four chains of pairs)
#pragma unroll 1
      for (int x = c0; x < c1; x += 32) {
        float o[32];
        __syncwarp();
        tmem_ld_x32(tm_o + (merge ? 0 : i * D) + x, o);
        tmem_ld_wait();
        pin(o);
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] *= f0;
        if (merge && g.count(1) > 0) {
          float o1[32];
          tmem_ld_x32(tm_o + D + x, o1);
          tmem_ld_wait();
          pin(o1);
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = fmaf(o1[y], f1, o[y]);
        }
        if (empty) {
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = 0.0f;
        }
        if (bad_seen != 0 && !empty) o[0] = NAN;   // the row lacks the values of nodes that were zeroed
#pragma unroll
        for (int y = 0; y < 32; y += 2) odd[y / 2 & 3] = fma2(pack2(o[y], o[y + 1]), 0ull, odd[y / 2 & 3]);
        if (whole) {
          if (row_ok) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + orow * D + x);
#pragma unroll
            for (int y = 0; y < 32; y += 8)
              dst[y / 8] = make_uint4(pack_bf16(o[y], o[y + 1]), pack_bf16(o[y + 2], o[y + 3]),
                                      pack_bf16(o[y + 4], o[y + 5]), pack_bf16(o[y + 6], o[y + 7]));
          }
        } else if (row_ok) {
          float4* dst = place.part(p, g, area, r, orow) + x / 4 * place.kStep;
#pragma unroll
          for (int y = 0; y < 32; y += 4) dst[(y / 4) * place.kStep] = make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
        }
      }
      const float2 odds = unpack2(add2(add2(odd[0], odd[1]), add2(odd[2], odd[3])));
      if (odds.x + odds.y != 0.0f && row_ok && l == l) s.odd = 1;   // (with a NaN score the row is NaN throughout)
      __syncwarp();
      tc_fence_before();
      // O and the shared statistics may be overwritten once both pipelines have read them
      named_bar_sync(1, 2 * kTile);
    }
    if (s.odd != 0) {   // written before the last segment's barrier
      typename WalkOf<kMode>::type anew;
      if constexpr (kMode == kShared)
        anew.start(p, blockIdx.x, gridDim.x);
      else if constexpr (kMode == kTeam)
        anew.start_team(p, blockIdx.x / p.team, blockIdx.x % p.team);
      else
        anew.start(run);
      sum_again<D, kMode>(p, anew, ring);
    }
  }

  if constexpr (kMode == kTeam) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    join_team<D>(p, walk, ring);
    __syncwarp();
    cluster_arrive();                     // nobody leaves while its parts may still be read
    cluster_wait();
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait_bounded(&s.drain, 0, a.err);   // the tensor cores have finished
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct Tiling {
  int32_t tpt, row_tiles, pairs, areas;
};

inline Tiling tile_rows(int64_t T, int64_t group) {
  Tiling t;
  t.tpt = static_cast<int32_t>(kTile / group);
  t.row_tiles = static_cast<int32_t>((T + t.tpt - 1) / t.tpt);
  t.pairs = (t.row_tiles + 1) / 2;
  t.areas = t.row_tiles > 1 ? 2 : 1;
  return t;
}

// Rows of a box of K or V: a box lies in one page.
inline int32_t box_rows(const KvView& c) { return c.table != nullptr && c.page_size < kTile ? c.page_size : kTile; }

struct Maps {
  CUtensorMap q, k, v, kn, vn;
};

// The queries as `batches` times `nodes` nodes (strides q_b and q_t), boxes of tpt of them; pages, and drafted nodes.
template <int D>
bool make_maps(const AttnArgs& a, int32_t tpt, int32_t rows, int64_t nodes, int64_t batches, Maps* m) {
  const KvView& c = a.cache;
  const uint64_t qd[5] = {D, static_cast<uint64_t>(a.group), static_cast<uint64_t>(nodes),
                          static_cast<uint64_t>(c.heads), static_cast<uint64_t>(batches)};
  const uint64_t qs[4] = {static_cast<uint64_t>(a.q_h), static_cast<uint64_t>(a.q_t),
                          static_cast<uint64_t>(a.q_h) * a.group, static_cast<uint64_t>(a.q_b)};
  const uint32_t qb[5] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(tpt), 1, 1};
  if (!make_tmap_bf16_nd(&m->q, a.q, 5, qd, qs, qb)) return false;
  const uint64_t kd[4] = {D, static_cast<uint64_t>(imax64(c.page_size, 1)), static_cast<uint64_t>(c.heads),
                          static_cast<uint64_t>(imax64(c.num_pages, 1))};
  const uint64_t ks[3] = {static_cast<uint64_t>(c.token_stride), static_cast<uint64_t>(c.head_stride),
                          static_cast<uint64_t>(c.page_stride)};
  const uint32_t kb[4] = {64, static_cast<uint32_t>(rows), 1, 1};
  // an empty cache has no memory to describe: any valid address will do, nothing is read
  const void* k = c.capacity > 0 ? c.k : a.q;
  const void* v = c.capacity > 0 ? c.v : a.q;
  if (!make_tmap_bf16_nd(&m->k, k, 4, kd, ks, kb) || !make_tmap_bf16_nd(&m->v, v, 4, kd, ks, kb)) return false;
  m->kn = m->k;
  m->vn = m->v;
  if (a.k_new == nullptr) return true;
  const uint64_t nd[4] = {D, static_cast<uint64_t>(a.T), static_cast<uint64_t>(c.heads), static_cast<uint64_t>(a.B)};
  const uint64_t ns[3] = {static_cast<uint64_t>(a.new_t), static_cast<uint64_t>(a.new_h), static_cast<uint64_t>(a.new_b)};
  const uint32_t nb[4] = {64, kTile, 1, 1};
  return make_tmap_bf16_nd(&m->kn, a.k_new, 4, nd, ns, nb) && make_tmap_bf16_nd(&m->vn, a.v_new, 4, nd, ns, nb);
}

}  // namespace
}  // namespace dflash2
