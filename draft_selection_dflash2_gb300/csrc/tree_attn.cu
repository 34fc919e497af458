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
        sum.template add_parts<D, 2>(p, d, c0, c0, step, tile, x, r);
        sum.write(a, orow, D, x);
      }
    } else {
      const int x = group * kNarrowCols;
      PartSum<kNarrowCols> sum;
      if (row_ok) sum.template add_parts<D, 4>(p, d, c0, c0 + y * step, kJoinSplit * step, tile, x, r);
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

// Measured against runs that hold all pairs' units (8 sequences of 16384, 8 heads of 128 in groups of
// 8): 64 nodes, 4 row tiles, 270 us against 279 (the second pair finds the keys in L2); 48 nodes, 3 row
// tiles, 233 against 269 (the runs of the full pair took the longest); 65 nodes, 5 row tiles, 353
// against 390; 64 short sequences of 48 nodes, whose runs hold many items, 132 to 138 against 136 to 139.
Lanes deal_lanes(int32_t row_tiles, int32_t runs) {
  if (row_tiles <= 2) return {1, runs};
  Lanes l = {row_tiles / 2, 0};
  const int32_t weight = kPair * l.n + (row_tiles % 2) * kSingle;   // of all pairs
  l.runs = kPair * runs / weight;
  // where the CTAs do not divide well (more than 3% lost), all pairs share all runs
  return l.runs * weight * 33 >= kPair * 32 * runs ? l : Lanes{0, 0};
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
    if (cudaOccupancyMaxActiveClusters(&at_once, tree_attn_kernel<D, kTeam>, &cfg) != cudaSuccess) {
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
  cudaError_t e = set_smem_limit<tree_attn_kernel<D, kTeam>>(smem);
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
    return cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, kTeam>, m.q, m.k, m.v, m.kn, m.vn, p);
  }
  e = set_smem_limit<tree_attn_kernel<D, kRuns>>(smem);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(runs, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, kRuns>, m.q, m.k, m.v, m.kn, m.vn, p);
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
