// tree_attn.cu -- attention from drafted nodes to a paged cache and to one
// another, the target's pass over a draft block.
//
//   z_x = scale <q, k_x>,  lse = log sum exp z_x,  out = sum exp(z_x - lse) v_x
//
// The query rows that share a key/value head, (node t, head g of the group) with
// row t * group + g, are stacked into tiles of up to 128 rows (whole nodes), so
// that a key is read once for all of them and both products fill the tensor
// cores' 128 rows.  Keys come in tiles of 128: the cache's tiles, then one tile
// of the drafted nodes.  An item is (sequence, kv head, pair of row tiles); its
// key tiles are its units.  All units of the call, item after item, are cut into
// equal runs, one per CTA (one CTA per SM): ragged lengths balance whatever they
// are, and an axis is split exactly where runs end.  With more than one pair each
// pair has runs of its own, beside one another (see Lanes).  An item cut by a run's end
// leaves unnormalised partial sums (fp32 O, m, l) in the workspace, and
// tree_attn_join_kernel adds them in run order (same bits on every call).  Where a
// call has few and short items (a sequence or a few), a cluster of CTAs takes each
// item instead: its CTAs leave their sums in their own shared memory and add them
// from there, so that no second kernel has to start (see team_size).
//
// tree_attn_kernel, per CTA:
//   warp 0      TMA producer: the item's query tiles, then each unit's K and V
//               tiles (128 x D bf16, 128-byte swizzle, one box per page piece,
//               the lanes issuing in parallel) into a ring.
//   warps 1, 2  S products of pipelines 0 and 1: S = Q K^T for 64 keys at a time
//               (fp32, two 64-column TMEM buffers per pipeline, so that the next
//               S is computed under a softmax).
//   warps 3, 12 O products: O += P V, with P read from TMEM where it replaced S,
//               as two bf16 terms (P rounded, and what that lost).
//               Each kind of product has its own warp per pipeline: the waits
//               around a batch take about as long to execute as the batch itself.
//   warps 4-7, 8-11  softmax of pipelines 0 and 1, one row per thread: S from
//               TMEM, running maximum m and sum l in base 2, P = 2^(S c - m) back
//               to TMEM.  O is rescaled only when a row's maximum has risen by
//               more than 2^8 since m was set (P then stays below 2^8, exact in
//               scale), so most chunks never touch O outside the tensor cores.
// P needs both terms: rounded to bf16 alone each weight is off by up to 2^-8, as much
// as the output's own rounding, and nothing averages that out where the weights gather on
// a few keys or many keys are alike (a P of 2^5.3 is off the same way each time).  With
// the second term it is 2^-16, and the output is the fp32 sum's rounded once.  It costs the
// tensor cores half as much again: 8 trees of 64 nodes 270 us against 208 with one term.
// The two pipelines alternate on the tensor cores: one's softmax runs under the
// other's products.  With two row tiles in the item each pipeline takes one of
// them over every unit; with one row tile the pipelines take alternate units of
// it and their two (O, m, l) are added at the end.
//
// A value no row sees must not reach the sums even as 0 * NaN: cached V rows past
// the length are zeroed in shared memory, and so are a drafted node's non-finite values,
// which only some rows may see.  A key that a row does see must not reach it as 0 * inf
// (z = -inf, or P's second term) or inf - inf (the two terms), and a finite value times a
// P of 2^8 must not become infinite.  So where a row's O is not finite at the end, or the
// row sees a drafted node that was zeroed, its sums are taken again when the run is done,
// key by key (sum_again): a key with z = -inf is passed over, an infinite or NaN value of
// another one is added as it is, and m is the maximum so far.  The usual call pays one
// operation per two elements of O, which does not show in its time.
//
// What bounds it, and what it measured (GB300, heads in groups of 8 over 8 kv heads,
// D = 128 unless said otherwise; replays of a graph, calls through the binding take up to
// 10% longer where the clocks drop under load):
//   memory   up to about 128 query rows per kv head: 2 sequences of 131072
//            positions, one token each, 167 us = 6.4 TB/s (96% of a copy's rate).
//   tensor cores beyond: 8 trees of 64 nodes over 16384 positions, 270 us = 1.02
//            PFLOP/s of the definition's products, 1.53 with P's second term; the tensor
//            pipe is active 66% of the time, and much of the rest is waiting for S's operands
//            (64-key products read 6 KB of shared memory per 32 cycles of products, at
//            128 B a cycle).  64 keys and not 128 because two S buffers of 128 per
//            pipeline and the O accumulators do not fit 512 columns, and with one buffer the
//            softmax and the products of a pipeline wait for one another (with one term 337 us
//            against 242).
//   latency  in small calls: one token over 500 positions, groups of 4, takes 8.5 us (11.5
//            with runs and a join, of which the join and the writing of parts are 4).
//   64 blocks of 17 over ragged lengths up to 12000, 136 rows per kv head: 420 us
//   against 271 for its bytes; the second row tile holds 8 rows but takes the tensor
//   cores as long as a full one.
// Splitting every item in equal runs, rather than by whole items, is what ragged
// batches and few heads need; the join costs 3 to 15 us.
//
// Every wait is bounded (DFLASH2_DEVERR_TIMEOUT): after one gives up the CTA
// stops issuing copies and products, walks its loops to their end, waits for its
// own copies in flight, frees its TMEM and returns.
#include <mutex>

#include "tree_attn.cuh"

namespace dflash2 {
namespace {

constexpr int kMaxTeam = 8;              // most CTAs of a team (a power of 2)
constexpr int kWholeUnits = 2;           // items of up to so many units are never cut

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
  int32_t box_rows;         // rows of a K or V box
  uint32_t q_box_bytes;
};

// Key tiles of sequence b, the drafted one included (at least one, so that every row is written).
__device__ __forceinline__ int32_t units_of(const AttnArgs& a, int32_t b) {
  const int32_t n = kv_clamp(a.cache_len[b], a.cache.capacity, a.err);
  return max(1, (n + kTile - 1) / kTile + (a.k_new != nullptr ? 1 : 0));
}

// One item's stretch of a run.
struct RunSegment {
  int32_t b, h, pair;
  int32_t s, e, n;          // units [s, e) of n
  int32_t tiles;            // row tiles (2: one per pipeline; 1: shared by both)
  int32_t len;              // cached positions
  bool first;               // the run's first segment
  __device__ __forceinline__ int count() const { return e - s; }
  // first position of unit u, the item's nodes, the row of one of them among all sequences', and of its queries
  __device__ __forceinline__ int position(int u) const { return u * kTile; }
  __device__ __forceinline__ int num_nodes(const AttnArgs& a) const { return a.T; }
  __device__ __forceinline__ int64_t node(const AttnArgs& a, int t) const { return static_cast<int64_t>(b) * a.T + t; }
  __device__ __forceinline__ int64_t q_row(const AttnArgs& a, int t) const { return b * a.q_b + t * a.q_t; }
  // keys of unit u: cached ones, or (the last unit, with drafted nodes) the nodes
  __device__ __forceinline__ bool drafted(const AttnArgs& a, int u) const {
    return a.k_new != nullptr && u == n - 1;
  }
  __device__ __forceinline__ int keys(const AttnArgs& a, int u) const {
    return drafted(a, u) ? a.T : max(0, min(kTile, len - u * kTile));
  }
  // units that pipeline i takes
  __device__ __forceinline__ int count(int i) const { return tiles == 2 ? e - s : (e - s + 1 - i) >> 1; }
};

// Where a segment's sums go: to the output, or to its parts, a run's in the workspace
// (the first segment's in slot 2 c, another's in 2 c + 1), a team's CTA's in its ring.
template <int D, bool kTeam>
struct PartPlace {
  bool whole;
  int slot;
  float4* parts;
  float2* mls;
  __device__ __forceinline__ PartPlace(const AttnPlan& p, const RunSegment& g, uint8_t* ring)
      : whole(!kTeam && g.s == 0 && g.e == g.n),
        slot(kTeam ? 0 : 2 * static_cast<int>(blockIdx.x) + (g.first ? 0 : 1)),
        parts(reinterpret_cast<float4*>(kTeam ? ring : reinterpret_cast<uint8_t*>(p.part))),
        mls(kTeam ? reinterpret_cast<float2*>(ring + 2 * kTile * D * 4) : p.part_ml) {}
  // Row r's O in the tile, four columns every kStep float4, and its m and l.
  static constexpr int kStep = kTile;
  static constexpr int copies() { return 1; }
  __device__ __forceinline__ float4* part(const AttnPlan& p, int tile, int r, int64_t) const {
    return parts + (static_cast<int64_t>(slot) * p.areas + tile) * (D / 4) * kTile + r;
  }
  __device__ __forceinline__ void put_ml(const AttnPlan& p, int tile, int r, int64_t, float m, float l) const {
    mls[(static_cast<int64_t>(slot) * p.areas + tile) * kTile + r] = make_float2(m, l);
  }
};

template <bool kTeam>
struct Walk : RunWalk {
  using Segment = RunSegment;
  template <int D>
  using Place = PartPlace<D, kTeam>;
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
  __device__ __forceinline__ bool next(const AttnPlan& p, Segment* g) {
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

// Adds to `sum` row r's parts of columns x.. in runs c, c + step, .. c1, kBatch loads at a time.
template <int D, int kBatch, int N>
__device__ __forceinline__ void add_parts(PartSum<N>& sum, const AttnPlan& p, const int4& d, int c0, int c, int step,
                                          int tile, int x, int r) {
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
      if (c + w * step <= d.z) sum.add(ml[w].x, ml[w].y, v[w]);
  }
}
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
__device__ __forceinline__ void join_team(const AttnPlan& p, const Walk<true>& walk, const uint8_t* ring) {
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

template <int D, bool kTeam>
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
  Walk<kTeam> walk;
  RunStart run = {0, 0, 0, 0};
  if constexpr (kTeam) {
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
  RunSegment g;
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
                        (2 * g.pair + i) * p.tpt, g.h, g.b, &s.q_full);
      }
      __syncwarp();
      // lane -> (page piece of the tile, column block)
      const int half = lane % C::kHalves, piece = lane / C::kHalves;
      const int row = piece * p.box_rows;       // first row of the lane's box
      pages.start(a.cache, g.b, g.s, g.len, lane);
      for (int u = g.s; u < g.e; ++u) {
        const bool drafted = g.drafted(a, u);
        bool has;
        int y = 0, z = g.h, w = g.b;
        uint32_t bytes;
        if (drafted) {
          has = lane < C::kHalves;
          bytes = kTile * 128;
        } else {
          const int j = u * kTile + row;
          has = row < kTile && j < g.len;
          bytes = p.box_rows * 128;
          y = j;
          if (pages.row != nullptr) {
            w = pages.page(a.cache, u * kTile, j, has, lane, a.err);
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
      const bool row_ok = r < p.tpt * a.group && node < a.T;
      // a warp none of whose rows is a query's has nothing to do but to keep step
      const bool busy = (warp & 3) * 32 < min(p.tpt, a.T - (node - t_r)) * a.group;
      float m = -INFINITY, l = 0.0f;
      uint32_t vis[4] = {0, 0, 0, 0};   // what the row sees of a tile that is not whole
      bool bad_seen = false;            // whether a node that it sees is non-finite
      for (int j = 0; j < cnt; ++j) {
        const int u = g.s + j * step + off;
        const bool drafted = g.drafted(a, u);
        const int valid = g.keys(a, u);
        const int chunks = valid <= kChunk ? 1 : 2;
        const bool partial_tile = drafted || valid < chunks * kChunk;
        wait_live(&s.s_full[i][at_s.buf], at_s.use & 1, &live, abort_flag, a.err);
        if (partial_tile) {
          RingPos<S> at_v = seg_v;
          at_v.advance_far(2 * (j * step + off));
          wait_live(at_v.full(s.kv_full), at_v.parity(), &live, abort_flag, a.err);
          const bool masked = drafted && a.mask != nullptr;
          const int upto = drafted && !masked ? min(valid, node + 1) : valid;
          const uint64_t m0 = masked ? mask_word(a, g.b, node, row_ok, 0) : ~0ull;
          const uint64_t m1 = masked ? mask_word(a, g.b, node, row_ok, 1) : ~0ull;
#pragma unroll
          for (int w = 0; w < 4; ++w) vis[w] = keys_before(upto, w) & static_cast<uint32_t>((w < 2 ? m0 : m1) >> (w & 1) * 32);
          // the pipelines that take the drafted tile look through it together
          const bool both = g.tiles == 2;
          bad_seen |= see_tile<D>(a, ring + at_v.slot * C::kTileBytes, drafted, valid, chunks,
                                  both ? static_cast<int>(threadIdx.x) - kTile : r, both ? 2 * kTile : kTile, r, s.bad,
                                  [&](int w) { return vis[w]; },
                                  [&]() { named_bar_sync(both ? 1 : 2 + i, both ? 2 * kTile : kTile); });
        }
#pragma unroll 1
        for (int c = 0; c < chunks; ++c, at_s.advance()) {
          const int buf = at_s.buf;
          const uint32_t tm_sb = tm_s + buf * kChunk;
          if (c > 0) wait_live(&s.s_full[i][buf], at_s.use & 1, &live, abort_flag, a.err);
          __syncwarp();
          tc_fence_after();
          if (busy) {
            softmax_chunk<D>(tm_sb, tm_o + i * D, p.c, partial_tile,
                             [&](int w) { return w == 0 ? (c ? vis[2] : vis[0]) : c ? vis[3] : vis[1]; },
                             j == 0 && c == 0, row_ok, &m, &l, [&]() {
                               const BufPos prev = at_s.before();
                               wait_live(&s.pv_done[i][prev.buf], prev.use & 1, &live, abort_flag, a.err);
                             });
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&s.p_ready[i][buf]);
        }
      }
      seg_v.advance_far(2 * g.count());

      // ---- the item's (or the run's part of the item's) sums ----
      const PartPlace<D, kTeam> place(p, g, ring);
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
      } else if (kTeam) {
        named_bar_sync(1, 2 * kTile);     // the parts go where the other pipeline's tiles were
      }
      tc_fence_after();
      const bool empty = l == 0.0f;   // the row saw nothing: 0, whatever the values were
      const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
      f0 *= inv;
      f1 *= inv;
      const int c0 = merge ? i * (D / 2) : 0, c1 = merge ? c0 + D / 2 : D;
      const int64_t orow = (static_cast<int64_t>(g.b) * a.T + node) * a.heads + g.h * a.group + r % a.group;
      const int area = merge ? 0 : i;
      if (!merge || i == 0) {
        if (whole) {
          if (row_ok && a.lse != nullptr)
            a.lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        } else {
          place.put_ml(p, area, r, orow, m, l);
        }
      }
      if (!kTeam && threadIdx.x == kTile && walk.left <= 0)        // the run's last segment
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
        if (bad_seen && !empty) o[0] = NAN;   // the row lacks the values of nodes that were zeroed
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
          float4* dst = place.part(p, area, r, orow) + x / 4 * place.kStep;
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
      Walk<kTeam> anew;
      if constexpr (kTeam)
        anew.start_team(p, blockIdx.x / p.team, blockIdx.x % p.team);
      else
        anew.start(run);
      sum_again<D>(p, anew, ring);
    }
  }

  if constexpr (kTeam) {
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

// Adds the parts of the items that runs cut.  Every CTA lists the cut items from
// the runs' records; a task is one of them, one of its row tiles and a group of
// columns; a thread takes a row and a few columns and adds parts as the softmax adds
// keys.  With many cut items (of few parts each) a task is 32 columns, 8 a thread,
// and a thread takes every part.  With few (a few heads, a long cache, many parts
// each) it is 4 columns, thread (r, y) takes every 4th part from the y-th on, and
// the four sums are added in order.
constexpr int kJoinSplit = 4, kJoinThreads = kTile * kJoinSplit, kWideCols = 8, kNarrowCols = 4;

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 2) tree_attn_join_kernel(const __grid_constant__ AttnPlan p, int runs) {
  __shared__ int4 list[kMaxRuns];
  __shared__ int32_t list_run[kMaxRuns];
  __shared__ int32_t warp_n[kJoinThreads / 32];
  __shared__ float s_o[kJoinSplit][kNarrowCols + 2][kTile];
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, r = tid & (kTile - 1), y = tid / kTile;
  pdl_wait();
  pdl_launch_dependents();
  const int4 mine = tid < runs ? p.cuts[tid] : make_int4(-1, 0, 0, 0);
  const bool cut = mine.x >= 0;
  const uint32_t cuts = __ballot_sync(0xFFFFFFFFu, cut);
  if ((tid & 31) == 0) warp_n[tid >> 5] = __popc(cuts);
  __syncthreads();
  int n = 0, at = __popc(cuts & ((1u << (tid & 31)) - 1));
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    if (w < tid >> 5) at += warp_n[w];
    n += warp_n[w];
  }
  if (cut) {
    list[at] = mine;
    list_run[at] = tid;
  }
  __syncthreads();
  const bool wide = 2 * n * p.areas * (D / (kWideCols * kJoinSplit)) >= static_cast<int>(gridDim.x);
  const int groups = wide ? D / (kWideCols * kJoinSplit) : D / kNarrowCols;
  for (int task = blockIdx.x; task < n * p.areas * groups; task += gridDim.x) {
    const int group = task % groups, tile = task / groups % p.areas;
    const int4 d = list[task / groups / p.areas];
    const int c0 = list_run[task / groups / p.areas];
    const int pair = d.y % p.pairs, h = d.y / p.pairs;
    if (2 * pair + tile >= p.row_tiles) continue;
    const int step = p.lanes.step(pair);
    const int node = (2 * pair + tile) * p.tpt + r / a.group;
    const bool row_ok = r < p.tpt * a.group && node < a.T;
    const int64_t orow = (static_cast<int64_t>(d.x) * a.T + node) * a.heads + h * a.group + r % a.group;
    if (wide) {
      const int x = group * kWideCols * kJoinSplit + y * kWideCols;
      PartSum<kWideCols> sum;
      if (row_ok) {
        add_parts<D, 2>(sum, p, d, c0, c0, step, tile, x, r);
        sum.write(a, orow, D, x);
      }
    } else {
      const int x = group * kNarrowCols;
      PartSum<kNarrowCols> sum;
      if (row_ok) add_parts<D, 4>(sum, p, d, c0, c0 + y * step, kJoinSplit * step, tile, x, r);
      s_o[y][kNarrowCols][r] = sum.m;
      s_o[y][kNarrowCols + 1][r] = sum.odd ? -sum.l : sum.l;
#pragma unroll
      for (int k = 0; k < kNarrowCols; ++k) s_o[y][k][r] = sum.o[k];
      __syncthreads();
      if (y == 0 && row_ok) {
#pragma unroll
        for (int w = 1; w < kJoinSplit; ++w) {
          float v[kNarrowCols];
#pragma unroll
          for (int k = 0; k < kNarrowCols; ++k) v[k] = s_o[w][k][r];
          sum.add(s_o[w][kNarrowCols][r], s_o[w][kNarrowCols + 1][r], v);
        }
        sum.write(a, orow, D, x);
      }
      __syncthreads();
    }
  }
}

// A unit with one row tile takes about kSingle / 16 of the time of one with two (48 nodes, 3 row tiles, over
// 16384 and over 700 positions: 233 and 135 us; with 9 228 and 144, with 11 238 and 138).
constexpr int kSingle = 10;

// Measured against runs that hold all pairs' units (8 sequences of 16384, 8 heads of 128 in groups of
// 8): 64 nodes, 4 row tiles, 270 us against 279 (the second pair finds the keys in L2); 48 nodes, 3 row
// tiles, 233 against 269 (the runs of the full pair took the longest); 65 nodes, 5 row tiles, 353
// against 390; 64 short sequences of 48 nodes, whose runs hold many items, 132 to 138 against 136 to 139.
Lanes deal_lanes(int32_t row_tiles, int32_t runs) {
  if (row_tiles <= 2) return {1, runs};
  Lanes l = {row_tiles / 2, 0};
  const int32_t weight = 16 * l.n + (row_tiles % 2) * kSingle;   // of all pairs
  l.runs = 16 * runs / weight;
  // where the CTAs do not divide well (more than 3% lost), all pairs share all runs
  return l.runs * weight * 33 >= 16 * 32 * runs ? l : Lanes{0, 0};
}

// Clusters of k = 2, 4 or 8 CTAs that the GPU holds at once (cluster sizes must fit its parts).
template <int D>
int clusters_at_once(int k, size_t smem) {
  static std::mutex mu;
  static int known[kMaxDevices][kMaxTeam + 1] = {};      // the number + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(mu);
  int& n = known[dev][k];
  if (n == 0) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = k;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(k, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int at_once = 0;
    if (cudaOccupancyMaxActiveClusters(&at_once, tree_attn_kernel<D, true>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      at_once = 0;
    }
    n = at_once + 1;
  }
  return n - 1;
}

// Size of the clusters that take an item each, or 0: equal runs and a join.  A team needs no
// second kernel, which saves 3 to 8 us, but its CTAs may have more units each than a run would; a
// unit takes 1.1 us with one row tile, and more with two.  Measured, runs against teams (8 heads of
// 128 in groups of 4): 1 x 1 over 500 positions 11.5 and 8.5 us, 1 x 17 over 2000 14.0 and 11.5,
// over 8191 18.7 and 18.6, over 16384 22.1 and 29.4, 4 x 17 over 2000 23.6 and 15.5.
template <int D>
int team_size(int64_t items, int64_t units, bool two_tiles, int num_sms, size_t smem) {
  const int64_t run = (items * units + num_sms - 1) / num_sms;
  for (int k = kMaxTeam; k >= 2; k /= 2)
    if (items * k <= num_sms && items <= clusters_at_once<D>(k, smem))
      return (units + k - 1) / k - run <= (two_tiles ? 3 : 5) ? k : 0;
  return 0;
}

template <int D>
cudaError_t launch(const AttnArgs& a, void* workspace, int num_sms, cudaStream_t stream) {
  using C = Cfg<D>;
  const Tiling t = tile_rows(a.T, a.group);
  AttnPlan p;
  p.a = a;
  p.tpt = t.tpt;
  p.row_tiles = t.row_tiles;
  p.pairs = t.pairs;
  p.areas = t.areas;
  p.c = a.scale * 1.4426950408889634f;
  const KvView& c = a.cache;
  p.box_rows = box_rows(c);
  p.q_box_bytes = static_cast<uint32_t>(t.tpt * a.group) * D * 2;
  const int64_t most = tree_attn_units(a.B, a.T, a.group, c.heads, c.capacity);
  if (most >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;   // the entry point has refused it
  // Items of at most one unit per pipeline are left whole: nothing is gained by cutting them, and nothing has to
  // be joined.  (1 x 1 over 500 positions, 5 units, before there were teams: 14.9 us whole, 12.3 in runs.)
  p.whole = (static_cast<int64_t>(c.capacity) + kTile - 1) / kTile + (a.k_new != nullptr) <= kWholeUnits;
  int runs = static_cast<int>(imin64(imin64(num_sms, kMaxRuns), imax64(most, 1)));
  p.lanes = deal_lanes(t.row_tiles, runs);
  if (p.lanes.n == t.pairs) runs = p.lanes.n * p.lanes.runs;
  const size_t smem = C::kRing + sizeof(AttnSmem);
  cudaError_t e = set_smem_limit<tree_attn_kernel<D, true>>(smem);
  if (e != cudaSuccess) return e;
  const int64_t items = a.B * c.heads * t.pairs;
  p.team = p.whole ? 0 : team_size<D>(items, most / items, t.row_tiles > 1, num_sms, smem);
  if (p.team > 0) p.lanes = {0, 0};
  p.part = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part + static_cast<size_t>(2) * num_sms * t.areas * kTile * D);
  p.cuts = reinterpret_cast<int4*>(p.part_ml + static_cast<size_t>(2) * num_sms * t.areas * kTile);

  Maps m;
  if (!make_maps<D>(a, t.tpt, p.box_rows, a.T, a.B, &m)) return cudaErrorInvalidValue;

  cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
  cudaLaunchConfig_t cfg = {};
  if (p.team > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.team;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(items * p.team), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, true>, m.q, m.k, m.v, m.kn, m.vn, p);
  }
  e = set_smem_limit<tree_attn_kernel<D, false>>(smem);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(runs, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, false>, m.q, m.k, m.v, m.kn, m.vn, p);
  if (e != cudaSuccess || runs == 1 || p.whole) return e;
  // one CTA per task up to two per SM; at most runs - 1 items are cut
  cfg.gridDim = dim3(static_cast<unsigned>(imin64(2 * num_sms, static_cast<int64_t>(runs - 1) * t.areas * (D / kNarrowCols))),
                     1, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_attn_join_kernel<D>, p, runs);
}

}  // namespace

int64_t tree_attn_units(int64_t B, int64_t T, int64_t group, int64_t kv_heads, int64_t capacity) {
  return B * kv_heads * tile_rows(T, group).pairs * ((capacity + kTile - 1) / kTile + 1);
}

size_t tree_attn_workspace_bytes(int64_t, int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim, int num_sms) {
  const int64_t group = heads / kv_heads;
  if (group > kTile) return 0;
  return static_cast<size_t>(2) * num_sms * tile_rows(T, group).areas * kTile * (head_dim * 4 + 8) +
         static_cast<size_t>(num_sms) * sizeof(int4);
}

cudaError_t launch_tree_attn(const AttnArgs& a, int64_t head_dim, void* workspace, int num_sms, cudaStream_t stream) {
  return head_dim == 64 ? launch<64>(a, workspace, num_sms, stream) : launch<128>(a, workspace, num_sms, stream);
}

}  // namespace dflash2
