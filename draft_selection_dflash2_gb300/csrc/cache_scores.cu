// cache_scores.cu -- the attention weight that each cached position received
// from a verified block, added to its running total:
//
//   scores[b,h,j] += sum_r exp(scale <q_r, k_j> - lse_r)
//
// over the rows r = (accepted node i, head g of the group) of key/value head h.
// The sum runs over rows, so the product is taken keys by rows, S^T = K Q^T: a
// key is a TMEM lane and one thread adds up its key's columns with no exchange
// between threads.  A unit is 128 keys of one (sequence, head); its rows are taken
// in equal chunks of up to 128 columns.  All units are cut into equal runs, one per
// CTA: equal in weight where sequences may differ in rows and the call is large (a unit
// of 136 rows takes a fifth longer than one of 8), else in units.
//   warp 0      TMA producer of K tiles (128 x D, one box per page piece).
//   warps 1, 2  MMA issuers of the even and the odd units (one warp for both was
//               the slowest part at 136 rows: 2560 cycles a unit).
//   warps 4-7, 8-11  epilogues of the even and the odd units: exp2(S c - lse c')
//               per column, summed in fp32 in column order.  Each has two TMEM buffers
//               of 128 columns, so that a chunk's product runs under the last one's
//               exponentials (with one buffer of 256: 1724 cycles a unit at 136 rows).
// Bound by memory while a unit's products and exponentials hide under its keys (up
// to about 128 rows): 16 blocks of 17 nodes, 1 to 17 of them accepted, in groups of 8
// over 8 kv heads and ragged lengths up to 32768: 109 us for 625 MB, 5.7 TB/s (86% of
// a copy's rate; 118 us with runs equal in units, and 124 when a thread also waited for
// each piece of the query rows before it asked for the next).  With one node accepted
// everywhere a batch that takes 83 us takes 97 with all 17 accepted: the change from one
// head's rows to the next's drains the products, once or twice a run.  One block over
// 4000 positions: 4.6 us in a replayed graph, 5.2 to 5.7 a call, the latency of the first
// tiles.
// When a run enters another (sequence, head) the epilogue warps lay that head's
// query rows out in shared memory (up to 512 rows; more rows take one launch per
// 512) and their lse beside them.  Rows that add nothing (their lse is -inf, and those
// that fill the last 16 up) are zero there; as 0 times an infinite key is NaN, not 0,
// their products are set to 0 before they are used.
#include <cstddef>

#include "attn_common.cuh"
#include "launch.h"

namespace dflash2 {
namespace {

constexpr int kThreads = 384;
constexpr int kMaxQTiles = 4;           // 128-row tiles of queries per launch
constexpr int kMaxSlots = 12;
constexpr int kQBatch = 4;              // 16-byte pieces of query rows that a thread loads at once
constexpr int kSmemLimit = 232448;      // 227 KB

struct ScoresSmem {
  uint64_t k_full[2 * kMaxSlots], k_empty[kMaxSlots];
  uint64_t q_full[2], s_full[2][2], s_free[2][2], drain;   // q: segments by turns; s: [epilogue][TMEM buffer]
  alignas(16) float lse[kMaxQTiles * kTile];   // negated, in base 2: -inf for rows that add nothing (read by fours)
  uint32_t tmem;
  int abort_flag;
};

static_assert(offsetof(ScoresSmem, lse) % 16 == 0, "read as float4");

struct ScoresPlan {
  ScoresArgs a;
  float c;                  // scale * log2(e)
  int32_t limit;            // positions a length may reach
  float inv_group;          // 1 / group
  int32_t row0;             // first row of this launch
  int32_t q_tiles;          // 128-row tiles of queries that shared memory holds
  int32_t slots;            // ring of K tiles
  int32_t box_rows;
};

// Rows of sequence b that this launch takes.
__device__ __forceinline__ int32_t rows_of(const ScoresPlan& p, int64_t b) {
  const int32_t count = p.a.count == nullptr ? p.a.T : kv_clamp(p.a.count[b], p.a.T, p.a.err);
  return max(0, min(count * p.a.group - p.row0, p.q_tiles * kTile));
}

// Units of each of sequence b's heads, and what one takes in runs of equal weight: 32 for
// its keys, 1 for 10 rows (1 for 20 or 5 balanced less well: 112 us each in the case above).
constexpr int kMostWeight = 84;
template <bool kWeighted>
__device__ __forceinline__ int32_t units_of(const ScoresPlan& p, int32_t b, int32_t* weight) {
  const int32_t n = kv_clamp(p.a.cache_len[b], p.limit, p.a.err);
  const int32_t rows = rows_of(p, b);
  *weight = kWeighted ? 32 + rows / 10 : 1;
  return rows > 0 ? (n + kTile - 1) / kTile : 0;
}

struct Segment {
  int32_t b, h, s, e;       // units [s, e) of (b, h)
  int32_t len, rows;
};

// A run is a stretch of weight; the units that begin in it are its own.
template <bool kWeighted>
struct Walk : RunWalk {
  int32_t w;                // a unit's weight; `left` is one too
  __device__ __forceinline__ void start(const ScoresPlan& p, const RunStart& r) {
    RunWalk::start(r);
    w = 1;
    if (!kWeighted || left <= 0) return;
    n = uniform(units_of<kWeighted>(p, b, &w));
    const int32_t at = s;   // in weight
    s = (at + w - 1) / w;
    left -= s * w - at;
  }
  __device__ __forceinline__ bool next(const ScoresPlan& p, Segment* g) {
    if (left <= 0) return false;
    if (s == n) next_item([&](int32_t i) { return units_of<kWeighted>(p, i, &w); }, p.a.cache.heads);
    g->h = uniform(item);
    g->s = uniform(s);
    g->e = uniform(min(n, s + (left + w - 1) / w));
    g->b = uniform(b);
    g->len = uniform(kv_clamp(p.a.cache_len[b], p.limit, nullptr));
    g->rows = uniform(rows_of(p, b));
    left -= (g->e - s) * w;
    s = g->e;
    return true;
  }
};

// 32 lanes x 16 consecutive fp32 columns.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void pin16(float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                 "+f"(v[i + 6]), "+f"(v[i + 7]));
}

// How a segment's rows are cut into chunks of columns.
struct Chunks {
  int width, count, rows;
  __device__ __forceinline__ void set(int rows_) {
    rows = rows_;
    count = (rows + kTile - 1) / kTile;
    width = ((rows + count - 1) / count + 15) & ~15;
    count = (rows + width - 1) / width;
  }
  __device__ __forceinline__ int cols(int c) const { return min(width, (rows - c * width + 15) & ~15); }
};

// A place in the sequence of K tiles through a ring of S slots.  As each issuer
// looks at every other tile only, a slot's uses alternate between two landing
// barriers (see RingPos).
struct KPos {
  uint32_t slot = 0, use = 0;
  __device__ __forceinline__ void advance(uint32_t n, uint32_t S) {   // n <= S
    slot += n;
    if (slot >= S) {
      slot -= S;
      ++use;
    }
  }
  __device__ __forceinline__ uint64_t* full(uint64_t* bars) const { return &bars[2 * slot + (use & 1)]; }
  __device__ __forceinline__ uint32_t parity() const { return use >> 1 & 1; }
};

template <int D, bool kWeighted>
__global__ void __launch_bounds__(kThreads, 1)
    cache_scores_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ ScoresPlan p) {
  constexpr int kHalves = D / 64;
  constexpr int kTileBytes = kTile * D * 2;
  extern __shared__ __align__(1024) uint8_t q_smem[];   // no static shared memory: the base is 1024-byte aligned
  const ScoresArgs& a = p.a;
  const uint32_t S = p.slots;
  const uint32_t q_half = p.q_tiles * kTile * 128;      // bytes of a 64-column block of the query rows
  uint8_t* ring = q_smem + p.q_tiles * kTileBytes;
  ScoresSmem& s = *reinterpret_cast<ScoresSmem*>(ring + S * kTileBytes);
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  volatile int* abort_flag = &s.abort_flag;

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < S; ++i) {
      mbar_init(&s.k_full[2 * i], 1);
      mbar_init(&s.k_full[2 * i + 1], 1);
      mbar_init(&s.k_empty[i], 1);
    }
    mbar_init(&s.q_full[0], 2 * kTile);
    mbar_init(&s.q_full[1], 2 * kTile);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s.s_full[i >> 1][i & 1], 1);
      mbar_init(&s.s_free[i >> 1][i & 1], kTile);
    }
    mbar_init(&s.drain, 2);
    s.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
  }
  if (warp == 3) {
    tmem_alloc(&s.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s.tmem);
  pdl_wait();
  pdl_launch_dependents();
  const auto weight = [&](int32_t b) {
    int32_t w;
    const int32_t n = units_of<kWeighted>(p, b, &w);
    return n * w;
  };
  Walk<kWeighted> walk;
  walk.start(p, find_run(weight, static_cast<int32_t>(a.B), a.cache.heads, blockIdx.x, gridDim.x));
  Segment g;
  bool live = true;

  if (warp == 0) {
    // ---- producer ----
    KPos at;
    uint32_t issued = 0;
    const int half = lane % kHalves, row = lane / kHalves * p.box_rows;
    PageFeed pages;
    while (walk.next(p, &g)) {
      pages.start(a.cache, g.b, g.s, g.len, lane);
      for (int u = g.s; u < g.e; ++u, at.advance(1, S)) {
        const int j = u * kTile + row;
        const bool has = row < kTile && j < g.len;
        int y = j, w = g.b;
        if (pages.row != nullptr) {
          w = pages.page(a.cache, u * kTile, j, has, lane, a.err);
          y = j & (a.cache.page_size - 1);
        }
        const uint32_t boxes = __popc(__ballot_sync(0xFFFFFFFFu, has));
        if (at.use > 0) wait_live(&s.k_empty[at.slot], (at.use - 1) & 1, &live, abort_flag, a.err);
        live = __all_sync(0xFFFFFFFFu, live);
        if (!live) continue;
        ++issued;
        uint64_t* full = at.full(s.k_full);
        if (lane == 0) mbar_arrive_expect_tx(full, boxes * p.box_rows * 128);
        __syncwarp();
        if (has) tma_load_4d(ring + at.slot * kTileBytes + half * kTile * 128 + row * 128, &tmK, half * 64, y, g.h, w, full);
      }
    }
    // after a wait that gave up: this CTA's copies have landed before it exits (else the products have used them)
    if (lane == 0 && !live) {
      KPos last;
      const uint32_t first = issued > S ? issued - S : 0;
      last.slot = first % S;
      last.use = first / S;
      for (uint32_t j = first; j < issued; ++j, last.advance(1, S))
        mbar_wait_bounded(last.full(s.k_full), last.parity(), a.err);
    }
    __syncwarp();
  } else if (warp <= 2) {
    // ---- MMA issuer of the units whose number in the run has parity e ----
    const int e = warp - 1;
    const uint32_t elected = elect_lane();
    const uint32_t ring_addr = uniform(smem_addr(ring)), q_addr = uniform(smem_addr(q_smem));
    KPos at;
    at.advance(e, S);
    uint32_t n = 0;               // chunks so far
    Chunks ch;
    uint32_t it0 = 0;             // the run's units before this segment
    int seg = 0;
    for (; walk.next(p, &g); ++seg) {
      // Nothing holds the epilogues back for an issuer without a unit in the segment: they may have laid out
      // the next one's rows before it looks.  They cannot be two ahead, as of two units in turn one is the
      // issuer's; so segments alternate between two barriers, and a phase cannot be mistaken for the next.
      wait_live(&s.q_full[seg & 1], seg >> 1 & 1, &live, abort_flag, a.err);
      ch.set(g.rows);
      for (int u = g.s + ((it0 ^ e) & 1); u < g.e; u += 2, at.advance(2, S)) {
        wait_live(at.full(s.k_full), at.parity(), &live, abort_flag, a.err);
        const uint32_t k_lo = desc_lo(ring_addr + at.slot * kTileBytes);
        for (int c = 0; c < ch.count; ++c, ++n) {
          const int buf = n & 1;
          if (n >= 2) wait_live(&s.s_free[e][buf], ((n >> 1) - 1) & 1, &live, abort_flag, a.err);
          __syncwarp();
          tc_fence_after();
          const uint32_t lead = live ? elected : 0u;
          const uint32_t q_lo = desc_lo(q_addr + c * ch.width * 128);
          const uint32_t idesc = umma_idesc_bf16(128, ch.cols(c));
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_ss(tmem + e * 2 * kTile + buf * kTile, k_lo + (((k >> 2) * kTile * 128 + (k & 3) * 32) >> 4),
                    q_lo + (((k >> 2) * q_half + (k & 3) * 32) >> 4), idesc, k > 0 ? 1u : 0u, lead);
          umma_commit_if(&s.s_full[e][buf], lead);
        }
        umma_commit_if(&s.k_empty[at.slot], live ? elected : 0u);
      }
      it0 += g.e - g.s;
    }
    umma_commit_if(&s.drain, elected);
    __syncwarp();
  } else if (warp >= 4) {
    // ---- epilogue half e: one key per thread ----
    const int e = warp >= 8 ? 1 : 0;
    const int r = threadIdx.x & (kTile - 1);
    const int tid = static_cast<int>(threadIdx.x) - kTile;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t it0 = 0;             // the run's units before this segment
    uint32_t n = 0;               // chunks so far
    Chunks ch;
    for (int seg = 0; walk.next(p, &g); ++seg) {
      // both halves have read every product of the last segment: its query rows may go
      __syncwarp();
      named_bar_sync(1, 2 * kTile);
      const int padded = (g.rows + 15) & ~15;
      constexpr int kPieces = D / 8, kRowStep = 2 * kTile / kPieces;
      const int piece = tid % kPieces;
      bool empty = false;                // whether one of the thread's rows adds nothing
      // kQBatch pieces a thread, so that their chains path -> lse and query run together
      for (int row0 = tid / kPieces; row0 < padded; row0 += kQBatch * kRowStep) {
        int t[kQBatch], hq[kQBatch];
        float lse[kQBatch];
        uint4 v[kQBatch];
#pragma unroll
        for (int y = 0; y < kQBatch; ++y) {
          const int row = row0 + y * kRowStep;
          t[y] = hq[y] = 0;
          if (row >= g.rows) continue;
          const int i = static_cast<int>((p.row0 + row + 0.5f) * p.inv_group);   // (exact: rows < 2^14)
          hq[y] = g.h * a.group + (p.row0 + row) - i * a.group;
          t[y] = a.path == nullptr ? i : a.path[static_cast<int64_t>(g.b) * a.T + i];
        }
#pragma unroll
        for (int y = 0; y < kQBatch; ++y) {
          lse[y] = -INFINITY;
          if (row0 + y * kRowStep >= g.rows) continue;
          const int node = clamp_node(t[y], a.T, a.err);
          lse[y] = a.lse[(static_cast<int64_t>(g.b) * a.T + node) * a.heads + hq[y]];
          v[y] = *reinterpret_cast<const uint4*>(a.q + g.b * a.q_b + node * a.q_t + hq[y] * a.q_h + piece * 8);
        }
#pragma unroll
        for (int y = 0; y < kQBatch; ++y) {
          const int row = row0 + y * kRowStep;
          if (row >= padded) break;
          // a query that saw nothing adds nothing, nor do the rows past the last
          if (lse[y] == -INFINITY) v[y] = make_uint4(0, 0, 0, 0);
          empty |= row < g.rows && lse[y] == -INFINITY;
          *reinterpret_cast<uint4*>(q_smem + (piece >> 3) * q_half + row * 128 + (((piece & 7) ^ (row & 7)) << 4)) = v[y];
          if (piece == 0) s.lse[row] = lse[y] == -INFINITY ? -INFINITY : lse[y] * -1.4426950408889634f;
        }
      }
      __syncwarp();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&s.q_full[seg & 1]);
      empty = named_bar_or(1, 2 * kTile, empty);      // the rows' lse is there
      ch.set(g.rows);
      for (int u = g.s + ((it0 ^ e) & 1); u < g.e; u += 2) {
        // the key's total so far, on its way while the products are waited for
        const int j = u * kTile + r;
        float* total = a.scores + (static_cast<int64_t>(g.b) * a.cache.heads + g.h) * a.scores_ld + j;
        const float before = j < g.len ? *total : 0.0f;
        uint64_t sum0 = pack2(0.0f, 0.0f), sum1 = sum0;
        const uint64_t c2 = pack2(p.c, p.c);
        for (int c = 0; c < ch.count; ++c, ++n) {
          const int buf = n & 1;
          wait_live(&s.s_full[e][buf], (n >> 1) & 1, &live, abort_flag, a.err);
          __syncwarp();
          tc_fence_after();
          const int cols = ch.cols(c);
          const int sure = empty ? 0 : g.rows - c * ch.width;   // columns below this one add something
          const float* l2 = s.lse + c * ch.width;
          const uint32_t tm = tmem + e * 2 * kTile + buf * kTile + lanes;
          const auto add16 = [&](const float* z, const float* l2x) {
#pragma unroll
            for (int y = 0; y < 16; y += 4) {
              const float4 l = *reinterpret_cast<const float4*>(l2x + y);
              const float2 e0 = unpack2(fma2(pack2(z[y], z[y + 1]), c2, pack2(l.x, l.y)));
              const float2 e1 = unpack2(fma2(pack2(z[y + 2], z[y + 3]), c2, pack2(l.z, l.w)));
              sum0 = add2(sum0, pack2(exp2_approx(e0.x), exp2_approx(e0.y)));
              sum1 = add2(sum1, pack2(exp2_approx(e1.x), exp2_approx(e1.y)));
            }
          };
          const auto clear_empty = [&](auto& z, const float* l2x) {
#pragma unroll
            for (int y = 0; y < static_cast<int>(sizeof(z) / sizeof(z[0])); ++y)
              if (l2x[y] == -INFINITY) z[y] = 0.0f;
          };
          int x = 0;
#pragma unroll 1
          for (; x + 32 <= cols; x += 32) {
            float z[32];
            tmem_ld_x32(tm + x, z);
            tmem_ld_wait();
            pin(z);
            if (x + 32 > sure) clear_empty(z, l2 + x);
            add16(z, l2 + x);
            add16(z + 16, l2 + x + 16);
          }
          if (x < cols) {
            float z[16];
            tmem_ld_x16(tm + x, z);
            tmem_ld_wait();
            pin16(z);
            if (x + 16 > sure) clear_empty(z, l2 + x);
            add16(z, l2 + x);
          }
          tc_fence_before();
          mbar_arrive(&s.s_free[e][buf]);
        }
        const float2 sum = unpack2(add2(sum0, sum1));
        if (j < g.len) *total = before + (sum.x + sum.y);
      }
      it0 += g.e - g.s;
    }
  }

  __syncthreads();
  if (threadIdx.x == 0) mbar_wait_bounded(&s.drain, 0, a.err);   // the tensor cores have finished
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Positions that a length may reach.
int32_t length_limit(const ScoresArgs& a) {
  return static_cast<int32_t>(imin64(a.cache.capacity, a.scores_ld));
}

int64_t most_units(const ScoresArgs& a) {
  return a.B * a.cache.heads * ((static_cast<int64_t>(length_limit(a)) + kTile - 1) / kTile);
}

template <int D, bool kWeighted>
cudaError_t launch(const ScoresArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kTileBytes = kTile * D * 2;
  const KvView& c = a.cache;
  ScoresPlan p;
  p.a = a;
  p.c = a.scale * 1.4426950408889634f;
  p.inv_group = 1.0f / static_cast<float>(a.group);
  p.limit = length_limit(a);
  if (p.limit == 0) return cudaSuccess;
  const int32_t rows = a.T * a.group;
  p.q_tiles = min((rows + kTile - 1) / kTile, kMaxQTiles);
  p.slots = min(kMaxSlots, static_cast<int>((kSmemLimit - sizeof(ScoresSmem)) / kTileBytes) - p.q_tiles);
  p.box_rows = c.table != nullptr && c.page_size < kTile ? c.page_size : kTile;
  CUtensorMap tmK;
  const uint64_t kd[4] = {D, static_cast<uint64_t>(c.page_size), static_cast<uint64_t>(c.heads),
                          static_cast<uint64_t>(c.num_pages)};
  const uint64_t ks[3] = {static_cast<uint64_t>(c.token_stride), static_cast<uint64_t>(c.head_stride),
                          static_cast<uint64_t>(c.page_stride)};
  const uint32_t kb[4] = {64, static_cast<uint32_t>(p.box_rows), 1, 1};
  if (!make_tmap_bf16_nd(&tmK, c.k, 4, kd, ks, kb)) return cudaErrorInvalidValue;
  const size_t smem = static_cast<size_t>(p.q_tiles + p.slots) * kTileBytes + sizeof(ScoresSmem);
  const cudaError_t e = set_smem_limit<cache_scores_kernel<D, kWeighted>>(kSmemLimit);
  if (e != cudaSuccess) return e;
  const int64_t most = most_units(a);
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(imin64(num_sms, most)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  for (p.row0 = 0; p.row0 < rows; p.row0 += kMaxQTiles * kTile) {
    const cudaError_t st = cudaLaunchKernelEx(&cfg, cache_scores_kernel<D, kWeighted>, tmK, p);
    if (st != cudaSuccess) return st;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_cache_scores(const ScoresArgs& a, int64_t head_dim, int num_sms, cudaStream_t stream) {
  const int64_t most = most_units(a);
  // In short runs a weight only breaks the runs' ends away from the heads' (one block over 4000 positions: 6.4 us
  // against 4.6), and the weights' sum has to fit.
  const bool weighted = a.B > 1 && most >= 8 * num_sms && most * kMostWeight < (int64_t(1) << 31);
  if (head_dim == 64) return weighted ? launch<64, true>(a, num_sms, stream) : launch<64, false>(a, num_sms, stream);
  return weighted ? launch<128, true>(a, num_sms, stream) : launch<128, false>(a, num_sms, stream);
}

}  // namespace dflash2
