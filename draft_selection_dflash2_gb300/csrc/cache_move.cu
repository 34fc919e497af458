// cache_move.cu -- rows that move between the drafted block, the cache and a
// smaller cache: the commit of an accepted path, and eviction.  Times are of replays of a
// graph; a call through the binding takes up to 1 us more where it is short, and the large
// eviction 195 to 198 us.
#include "attn.h"
#include "launch.h"
#include "tcgen05.cuh"

namespace dflash2 {
namespace {

// ---------------------------------------------------------------------------
// commit: node path[b, i] becomes position cache_len[b] + i, for i < count[b].
// A CTA takes (sequence, a few accepted nodes); a thread takes 16 bytes of K and of
// V of kCommitPieces rows at once, so that the chain path -> page -> row is walked
// once for all of them.  256 trees of 64 nodes over 8 heads of 128: 8.3 us for 33.7 MB
// (4.1 TB/s; one 16-byte piece a thread and no overlap of the chains took 16 us); one
// block of 17: 2.2 us.
// ---------------------------------------------------------------------------
constexpr int kCommitThreads = 256, kCommitPieces = 4;

template <int D>
__global__ void __launch_bounds__(kCommitThreads) cache_commit_kernel(const CommitArgs a, int blocks_per_seq) {
  constexpr int kVecs = D / 8;
  const int64_t b = blockIdx.x / blocks_per_seq;
  const int block = blockIdx.x % blocks_per_seq;
  pdl_wait();
  pdl_launch_dependents();
  const int32_t count = a.count == nullptr ? a.T : kv_clamp(a.count[b], a.T, a.err);
  int32_t limit = a.cache.capacity;
  if (a.scores != nullptr && a.scores_ld < limit) limit = static_cast<int32_t>(a.scores_ld);
  const int32_t len = kv_clamp(a.cache_len[b], limit, a.err);
  const int32_t end = kv_clamp(len + count, limit, a.err);
  if (block == 0 && threadIdx.x == 0) a.new_len[b] = end;
  const int row = a.cache.heads * kVecs;            // 16-byte pieces of one node's K (or V) rows
  const int x0 = block * kCommitThreads * kCommitPieces + threadIdx.x;
  if (x0 >= (end - len) * row) return;
  int64_t dst[kCommitPieces];
  uint4 k[kCommitPieces], v[kCommitPieces];
  bool ok[kCommitPieces];
#pragma unroll
  for (int y = 0; y < kCommitPieces; ++y) {
    const int x = x0 + y * kCommitThreads;
    ok[y] = false;
    if (x >= (end - len) * row) continue;
    const int piece = x % kVecs, h = x / kVecs % a.cache.heads, i = x / row;
    const int t = a.path == nullptr ? i : clamp_node(a.path[b * a.T + i], a.T, a.err);
    const int64_t src = b * a.new_b + t * a.new_t + h * a.new_h + piece * 8;
    k[y] = *reinterpret_cast<const uint4*>(a.k_new + src);
    v[y] = *reinterpret_cast<const uint4*>(a.v_new + src);
    dst[y] = kv_offset(a.cache, b, len + i, h, a.err, &ok[y]) + piece * 8;
    if (a.scores != nullptr && piece == 0) a.scores[(b * a.cache.heads + h) * a.scores_ld + len + i] = 0.0f;
  }
#pragma unroll
  for (int y = 0; y < kCommitPieces; ++y)
    if (ok[y]) {
      *reinterpret_cast<uint4*>(a.cache.k + dst[y]) = k[y];
      *reinterpret_cast<uint4*>(a.cache.v + dst[y]) = v[y];
    }
}

// ---------------------------------------------------------------------------
// eviction, step 1: which positions stay.  A cluster of CTAs per (b, h), each
// with a contiguous slice of its positions.  Wanted is the r-th largest key (the
// order-preserving image of the score) among the positions before the recent
// ones.  Its leading digit (11 bits) comes from counting all keys by theirs: each
// CTA its slice's, the cluster's counts added through distributed shared memory,
// and every CTA finds the digit that the r-th key has.  The keys that share it are
// usually few: they are collected, and each of up to kSelCands is ranked against
// all the others (by key, then position), which ends the search; where there are
// more, another digit is taken first.  Then the kept positions are listed in order:
// those above that key, the first ones equal to it, and the recent ones; a warp
// takes consecutive positions, and its place in the list is the number kept before
// them.  The scores are read once: a slice's keys stay in shared memory (slices of
// more than kSelKeys positions are read again by each step).  128 rows of 32768
// scores: 28 us, its own instructions and shared-memory atomics; the whole eviction of
// 16 x 8 rows to 8001 positions takes 192 us, 160 of them its bytes at a copy's rate.
// One row set of 4096 to 1024: 9.6 us, latency.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelCands = 128;          // (at 1024, ranking took longer than another digit: 40 us over 32768 positions)
constexpr int kSelKeys = 36864;          // 144 KB of keys
constexpr int kSelMaxCluster = 8;

struct SelSmem {
  uint32_t hist[2][kSelBins];            // by turns: a CTA may still read the last one when the next is filled
  uint64_t cand[kSelCands];              // this CTA's candidates: key, then the complement of the position
  uint64_t all[kSelCands];               // the cluster's
  uint32_t warp_sum[kSelWarps];
  uint32_t gt[kSelWarps], eq[kSelWarps]; // per warp: positions above the threshold (or recent), and equal to it
  uint32_t all_gt, all_eq;               // this CTA's
  uint32_t cands, digit, in_digit, need, key;
};

static_assert(kSelBins == 2 * kSelThreads, "two bins a thread");
static_assert(sizeof(SelSmem) + kSelKeys * 4 <= 232448, "shared memory");

__device__ __forceinline__ uint32_t cluster_word(const void* p, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  return at;
}
// The word at `p` of cluster CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t ld_cluster(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_word(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster(const uint64_t* p, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_word(p, rank)) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictArgs a, int cluster, int key_slots) {
  extern __shared__ __align__(16) uint8_t sel_smem[];
  SelSmem& s = *reinterpret_cast<SelSmem*>(sel_smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(sel_smem + sizeof(SelSmem));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = blockIdx.x % cluster;
  const int64_t row = blockIdx.x / cluster;
  const int64_t b = row / a.cache.heads;
  s.hist[0][tid] = s.hist[0][tid + kSelThreads] = 0;
  if (tid == 0) s.cands = 0;
  pdl_wait();
  pdl_launch_dependents();
  const int32_t limit = static_cast<int32_t>(imin64(a.cache.capacity, a.scores_ld));
  const int32_t n = kv_clamp(a.cache_len[b], limit, a.err);
  const int32_t kept_n = n < a.keep ? n : a.keep;
  int32_t* kept = a.kept + row * a.keep;
  const float* sc = a.scores + row * a.scores_ld;
  if (row % a.cache.heads == 0 && rank == 0 && tid == 0) a.new_len[b] = kept_n;
  const int first = static_cast<int>(rank) * kSelThreads + tid, step = cluster * kSelThreads;
  for (int64_t i = kept_n + static_cast<int64_t>(first); i < a.keep; i += step) kept[i] = -1;
  if (n <= a.keep) {                     // the whole cluster leaves together
    for (int64_t i = first; i < n; i += step) kept[i] = static_cast<int32_t>(i);
    return;
  }
  const int32_t m = n - a.recent;        // candidates: positions [0, m)
  // warps take consecutive groups of 32 positions
  const int32_t groups = (n + 31) >> 5;
  const int32_t per_warp = (groups + cluster * kSelWarps - 1) / (cluster * kSelWarps);
  const int32_t g0 = static_cast<int32_t>(rank) * kSelWarps * per_warp;       // the CTA's first group
  const int32_t w0 = min(groups, g0 + warp * per_warp), w1 = min(groups, w0 + per_warp);
  const bool held = per_warp * kSelThreads <= key_slots;
  const auto key_at = [&](int32_t group) -> uint32_t {
    const int32_t j = group * 32 + lane;
    if (held) return keys[(group - g0) * 32 + lane];
    return j < m ? score_order(sc[j]) : 0u;
  };
  const auto sync_cluster = [&]() {
    if (cluster > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };

  // keys above `prefix` stay, and `need` of those equal to it, once `shift` is 0 or
  // the candidates have been ranked; until then those that share the bits from
  // `shift` on are candidates
  uint32_t prefix = 0, need = static_cast<uint32_t>(a.keep - a.recent);
  int shift = 32;
  if (need == 0) {                       // only the recent ones stay: no key is above this one
    prefix = 0xFFFFFFFFu;
    shift = 0;
  }
  __syncthreads();
#pragma unroll 1
  for (int round = 0; shift > 0; ++round) {
    const int bits = shift == 10 ? 10 : 11;
    uint32_t* hist = s.hist[round & 1];
    if (round > 0) {
      hist[tid] = hist[tid + kSelThreads] = 0;
      __syncthreads();
    }
    if (round == 0) {
#pragma unroll 4
      for (int32_t g = w0; g < w1; ++g) {
        const int32_t j = g * 32 + lane;
        const uint32_t key = j < m ? score_order(__ldg(sc + j)) : 0u;
        if (held) keys[(g - g0) * 32 + lane] = key;
        if (j < m) atomicAdd(&hist[key >> 21], 1u);
      }
    } else {
#pragma unroll 4
      for (int32_t g = w0; g < w1; ++g) {
        const uint32_t key = key_at(g);
        if (g * 32 + lane < m && key >> shift == prefix >> shift)
          atomicAdd(&hist[key >> (shift - bits) & ((1u << bits) - 1)], 1u);
      }
    }
    shift -= bits;
    __syncthreads();
    // thread t has bins 2 t and 2 t + 1, added up over the cluster; a scan from the top
    // finds the bin that holds the need-th key
    uint32_t c0 = hist[2 * tid], c1 = hist[2 * tid + 1];
    if (cluster > 1) {
      sync_cluster();
      for (int r = 1; r < cluster; ++r) {
        const uint32_t other = (rank + r) % cluster;
        c0 += ld_cluster(&hist[2 * tid], other);
        c1 += ld_cluster(&hist[2 * tid + 1], other);
      }
    }
    const uint32_t own = c0 + c1;
    uint32_t incl = own;                 // over lanes, from the top lane down
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_down_sync(0xFFFFFFFFu, incl, d);
      if (lane + d < 32) incl += o;
    }
    if (lane == 0) s.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t above = warp + 1 + lane < kSelWarps ? s.warp_sum[warp + 1 + lane] : 0u;   // keys in higher bins
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, d);
    above += incl - own;
    if (above < need && above + own >= need) {
      const bool high = above + c1 >= need;
      s.digit = 2 * tid + (high ? 1 : 0);
      s.in_digit = high ? c1 : c0;
      s.need = need - above - (high ? 0 : c1);
    }
    __syncthreads();
    prefix |= s.digit << shift;
    need = s.need;                       // how many of the keys that share the prefix stay
    const uint32_t count = s.in_digit;
    if (shift == 0 || count > kSelCands) continue;

    // few candidates: rank them (all CTAs of the cluster do, and find the same)
#pragma unroll 4
    for (int32_t g = w0; g < w1; ++g) {
      const uint32_t key = key_at(g);
      const int32_t j = g * 32 + lane;
      if (j < m && key >> shift == prefix >> shift)
        s.cand[atomicAdd(&s.cands, 1u)] = static_cast<uint64_t>(key) << 32 | ~static_cast<uint32_t>(j);
    }
    sync_cluster();
    uint32_t at = 0;
    for (int r = 0; r < cluster; ++r) {
      const uint32_t c = cluster > 1 ? ld_cluster(&s.cands, r) : s.cands;
      if (static_cast<uint32_t>(tid) < c) s.all[at + tid] = cluster > 1 ? ld_cluster(&s.cand[tid], r) : s.cand[tid];
      at += c;
    }
    __syncthreads();
    uint64_t my = 0;
    uint32_t before = 0;
    if (static_cast<uint32_t>(tid) < count) {
      my = s.all[tid];
#pragma unroll 4
      for (uint32_t x = 0; x < count; ++x) before += s.all[x] > my ? 1u : 0u;
      if (before == need - 1) s.key = static_cast<uint32_t>(my >> 32);
    }
    __syncthreads();
    prefix = s.key;
    // of the keys equal to it, those that rank before it, and it, stay
    need = __syncthreads_count(static_cast<uint32_t>(tid) < count && before < need &&
                               static_cast<uint32_t>(my >> 32) == prefix);
    shift = 0;
  }

  // counts per warp, their sums per CTA, and the CTAs before this one
  uint32_t gt = 0, eq = 0;
#pragma unroll 4
  for (int32_t g = w0; g < w1; ++g) {
    const int32_t j = g * 32 + lane;
    const uint32_t key = key_at(g);
    gt += __popc(__ballot_sync(0xFFFFFFFFu, j < n && (j >= m || key > prefix)));
    eq += __popc(__ballot_sync(0xFFFFFFFFu, j < m && key == prefix));
  }
  if (lane == 0) {
    s.gt[warp] = gt;
    s.eq[warp] = eq;
  }
  __syncthreads();
  uint32_t gt_before = lane < warp ? s.gt[lane] : 0u, eq_before = lane < warp ? s.eq[lane] : 0u;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    gt_before += __shfl_xor_sync(0xFFFFFFFFu, gt_before, d);
    eq_before += __shfl_xor_sync(0xFFFFFFFFu, eq_before, d);
  }
  if (cluster > 1) {
    if (tid == kSelThreads - 32) {
      s.all_gt = gt_before + gt;
      s.all_eq = eq_before + eq;
    }
    sync_cluster();
    for (uint32_t r = 0; r < rank; ++r) {
      gt_before += ld_cluster(&s.all_gt, r);
      eq_before += ld_cluster(&s.all_eq, r);
    }
  }
#pragma unroll 2
  for (int32_t g = w0; g < w1; ++g) {
    const int32_t j = g * 32 + lane;
    const uint32_t key = key_at(g);
    const bool is_gt = j < n && (j >= m || key > prefix), is_eq = j < m && key == prefix;
    const uint32_t gts = __ballot_sync(0xFFFFFFFFu, is_gt), eqs = __ballot_sync(0xFFFFFFFFu, is_eq);
    const uint32_t below = (1u << lane) - 1;
    const uint32_t eq_rank = eq_before + __popc(eqs & below);
    if (is_gt || (is_eq && eq_rank < need))
      kept[gt_before + __popc(gts & below) + min(eq_rank, need)] = j;
    gt_before += __popc(gts);
    eq_before += __popc(eqs);
  }
  if (cluster > 1) sync_cluster();       // nobody leaves while its counts may still be read
}

// eviction, step 2: the kept rows to the destination.  A thread takes 16 bytes of K
// and of V of kGatherPasses kept positions at once, so that the chain position ->
// page -> row is walked once for all of them (2 positions in CTAs of 128 threads:
// 192 us for the whole eviction of 16 x 32768 to 8001; 4 in 256: 198, 1 in 256: 198).
constexpr int kGatherThreads = 128, kGatherPasses = 2;

template <int D>
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a, int32_t blocks_per_row) {
  constexpr int kVecs = D / 8, kRowsPerPass = kGatherThreads / kVecs, kPasses = kGatherPasses;
  constexpr int kRows = kRowsPerPass * kPasses;
  const int64_t row = blockIdx.x / blocks_per_row;
  const int32_t i0 = static_cast<int32_t>(blockIdx.x % blocks_per_row) * kRows;
  const int h = static_cast<int>(row % a.cache.heads);
  const int64_t b = row / a.cache.heads;
  const int piece = threadIdx.x % kVecs;
  pdl_wait();
  pdl_launch_dependents();
  int32_t j[kPasses];
  int64_t src[kPasses], dst[kPasses];
  bool ok[kPasses];
#pragma unroll
  for (int x = 0; x < kPasses; ++x) {
    const int32_t i = i0 + x * kRowsPerPass + threadIdx.x / kVecs;
    j[x] = i < a.keep ? a.kept[row * a.keep + i] : -1;
  }
#pragma unroll
  for (int x = 0; x < kPasses; ++x) {
    const int32_t i = i0 + x * kRowsPerPass + threadIdx.x / kVecs;
    ok[x] = false;
    if (j[x] >= 0) {
      bool any;
      src[x] = kv_offset(a.cache, b, j[x], h, a.err, &any) + piece * 8;
      dst[x] = kv_offset(a.dst, b, i, h, a.err, &ok[x]) + piece * 8;
      if (a.dst_scores != nullptr && piece == 0) a.dst_scores[row * a.dst_ld + i] = a.scores[row * a.scores_ld + j[x]];
    }
  }
  uint4 k[kPasses], v[kPasses];
#pragma unroll
  for (int x = 0; x < kPasses; ++x)
    if (ok[x]) {
      k[x] = __ldcs(reinterpret_cast<const uint4*>(a.cache.k + src[x]));
      v[x] = __ldcs(reinterpret_cast<const uint4*>(a.cache.v + src[x]));
    }
#pragma unroll
  for (int x = 0; x < kPasses; ++x)
    if (ok[x]) {
      __stcs(reinterpret_cast<uint4*>(a.dst.k + dst[x]), k[x]);
      __stcs(reinterpret_cast<uint4*>(a.dst.v + dst[x]), v[x]);
    }
}

}  // namespace

cudaError_t launch_cache_commit(const CommitArgs& a, int64_t head_dim, cudaStream_t stream) {
  const int64_t pieces = static_cast<int64_t>(a.T) * a.cache.heads * (head_dim / 8);
  const int blocks = static_cast<int>(imax64(1, (pieces + kCommitThreads * kCommitPieces - 1) /
                                                    (kCommitThreads * kCommitPieces)));
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B * blocks), 1, 1);
  cfg.blockDim = dim3(kCommitThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return head_dim == 64 ? cudaLaunchKernelEx(&cfg, cache_commit_kernel<64>, a, blocks)
                        : cudaLaunchKernelEx(&cfg, cache_commit_kernel<128>, a, blocks);
}

cudaError_t launch_cache_evict(const EvictArgs& a, int64_t head_dim, int num_sms, cudaStream_t stream) {
  const int64_t rows = a.B * a.cache.heads;
  const int64_t limit = imin64(a.cache.capacity, a.scores_ld);
  // CTAs per row: while they all fit at once and a slice is still some thousand positions
  int cluster = 1;
  while (cluster < kSelMaxCluster && rows * cluster * 2 <= num_sms && limit > 8192 * cluster) cluster *= 2;
  const int64_t slice = ((limit + 31) / 32 + cluster * kSelWarps - 1) / (cluster * kSelWarps) * kSelThreads;
  const int key_slots = static_cast<int>(imin64(slice, kSelKeys));
  const size_t smem = sizeof(SelSmem) + static_cast<size_t>(key_slots) * 4;
  cudaError_t e = set_smem_limit<evict_select_kernel>(sizeof(SelSmem) + kSelKeys * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster), 1, 1);
  cfg.blockDim = dim3(kSelThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cluster, key_slots);
  if (e != cudaSuccess) return e;
  const int vecs = static_cast<int>(head_dim / 8);
  const int per_cta = kGatherThreads / vecs * kGatherPasses;
  const int64_t blocks = (a.keep + per_cta - 1) / per_cta;   // grid.x: rows * blocks < 2^31 (checked by the entry point)
  cfg.gridDim = dim3(static_cast<unsigned>(rows * blocks), 1, 1);
  cfg.blockDim = dim3(kGatherThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return head_dim == 64 ? cudaLaunchKernelEx(&cfg, evict_gather_kernel<64>, a, static_cast<int32_t>(blocks))
                        : cudaLaunchKernelEx(&cfg, evict_gather_kernel<128>, a, static_cast<int32_t>(blocks));
}

}  // namespace dflash2
