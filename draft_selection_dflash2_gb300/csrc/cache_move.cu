// cache_move.cu -- rows that move between the drafted block, the cache and a
// smaller cache: the commit of an accepted path, and eviction.
#include "attn.h"
#include "launch.h"

namespace dflash2 {
namespace {

// ---------------------------------------------------------------------------
// commit: node path[b, i] becomes position cache_len[b] + i, for i < count[b].
// One thread per 16 bytes of a row (of K or of V).  Grid (row blocks, B).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) cache_commit_kernel(const CommitArgs a, int vecs) {
  const int64_t b = blockIdx.y;
  const int32_t count = a.count == nullptr ? a.T : kv_clamp(a.count[b], a.T, a.err);
  int32_t limit = a.cache.capacity;
  if (a.scores != nullptr && a.scores_ld < limit) limit = static_cast<int32_t>(a.scores_ld);
  const int32_t len = kv_clamp(a.cache_len[b], limit, a.err);
  const int32_t end = kv_clamp(len + count, limit, a.err);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.new_len[b] = end;
  const int row = a.cache.heads * vecs;   // 16-byte pieces of one node's K (or V) rows
  for (int x = blockIdx.x * blockDim.x + threadIdx.x; x < (end - len) * 2 * row; x += gridDim.x * blockDim.x) {
    const int piece = x % vecs, h = x / vecs % a.cache.heads, kv = x / row & 1, i = x / (2 * row);
    const int t = a.path == nullptr ? i : clamp_node(a.path[b * a.T + i], a.T, a.err);
    bool ok;
    const int64_t dst = kv_offset(a.cache, b, len + i, h, a.err, &ok) + piece * 8;
    const int64_t src = b * a.new_b + t * a.new_t + h * a.new_h + piece * 8;
    if (ok)
      *reinterpret_cast<uint4*>((kv ? a.cache.v : a.cache.k) + dst) =
          *reinterpret_cast<const uint4*>((kv ? a.v_new : a.k_new) + src);
    if (a.scores != nullptr && kv == 0 && piece == 0) a.scores[(b * a.cache.heads + h) * a.scores_ld + len + i] = 0.0f;
  }
}

// ---------------------------------------------------------------------------
// eviction, step 1: which positions stay.  One CTA per (b, h).  The r-th largest
// key (order-preserving image of the score) among the positions before the
// recent ones is found digit by digit from the top (a histogram of 256 digits
// per pass); then positions are listed in order: those above it, the first ones
// equal to it, and the recent ones.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_need, warp_sel[32], warp_eq[32];
  const int h = blockIdx.x % a.cache.heads;
  const int64_t b = blockIdx.x / a.cache.heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t limit = static_cast<int32_t>(imin64(a.cache.capacity, a.scores_ld));
  const int32_t n = kv_clamp(a.cache_len[b], limit, a.err);
  const int32_t kept_n = n < a.keep ? n : a.keep;
  int32_t* kept = a.kept + (b * a.cache.heads + h) * a.keep;
  const float* sc = a.scores + (b * a.cache.heads + h) * a.scores_ld;
  if (h == 0 && tid == 0) a.new_len[b] = kept_n;
  for (int i = kept_n + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
  if (n <= a.keep) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  const int32_t m = n - a.recent;
  if (tid == 0) {
    s_prefix = 0;
    s_need = a.keep - a.recent;
  }
  __syncthreads();
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int32_t j = tid; j < m; j += kSelThreads) {
      const uint32_t key = score_order(sc[j]);
      if (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&hist[key >> shift & 255], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t need = s_need;
      int d = 255;
      while (d > 0 && hist[d] < need) need -= hist[d--];
      s_need = need;
      s_prefix = prefix | static_cast<uint32_t>(d) << shift;
    }
    __syncthreads();
  }
  const uint32_t T = s_prefix;
  const uint32_t need_eq = s_need;   // how many of the keys equal to T stay
  uint32_t base_sel = 0, base_eq = 0;
  for (int32_t j0 = 0; j0 < n; j0 += kSelThreads) {
    const int32_t j = j0 + tid;
    const uint32_t key = j < m ? score_order(sc[j]) : 0u;
    const bool eq = j < m && key == T;
    const uint32_t eqs = __ballot_sync(0xFFFFFFFFu, eq);
    if (lane == 0) warp_eq[warp] = __popc(eqs);
    __syncthreads();
    uint32_t eq_rank = base_eq + __popc(eqs & ((1u << lane) - 1));
    uint32_t eq_all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) eq_rank += warp_eq[w];
      eq_all += warp_eq[w];
    }
    base_eq += eq_all;
    const bool sel = j < n && (j >= m || key > T || (eq && eq_rank < need_eq));
    const uint32_t sels = __ballot_sync(0xFFFFFFFFu, sel);
    if (lane == 0) warp_sel[warp] = __popc(sels);
    __syncthreads();
    uint32_t rank = base_sel + __popc(sels & ((1u << lane) - 1));
    uint32_t sel_all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) rank += warp_sel[w];
      sel_all += warp_sel[w];
    }
    base_sel += sel_all;
    if (sel) kept[rank] = j;
    __syncthreads();
  }
}

// eviction, step 2: the kept rows to the destination.  One thread per 16 bytes.
__global__ void __launch_bounds__(256) evict_gather_kernel(const EvictArgs a, int vecs) {
  const int h = blockIdx.x % a.cache.heads;
  const int64_t b = blockIdx.x / a.cache.heads;
  const int64_t row = b * a.cache.heads + h;
  const int piece = threadIdx.x % vecs, step = blockDim.x / vecs;
  for (int i = blockIdx.y * step + threadIdx.x / vecs; i < a.keep; i += gridDim.y * step) {
  const int32_t j = a.kept[row * a.keep + i];
  if (j < 0) return;
  bool ok, ok_dst;
  const int64_t src = kv_offset(a.cache, b, j, h, a.err, &ok) + piece * 8;
  const int64_t dst = kv_offset(a.dst, b, i, h, a.err, &ok_dst) + piece * 8;
  if (ok_dst) {
    *reinterpret_cast<uint4*>(a.dst.k + dst) = *reinterpret_cast<const uint4*>(a.cache.k + src);
    *reinterpret_cast<uint4*>(a.dst.v + dst) = *reinterpret_cast<const uint4*>(a.cache.v + src);
  }
  if (a.dst_scores != nullptr && piece == 0) a.dst_scores[row * a.dst_ld + i] = a.scores[row * a.scores_ld + j];
  }
}

}  // namespace

cudaError_t launch_cache_commit(const CommitArgs& a, int64_t head_dim, cudaStream_t stream) {
  const int vecs = static_cast<int>(head_dim / 8);
  const int64_t pieces = static_cast<int64_t>(a.T) * 2 * a.cache.heads * vecs;
  const dim3 grid(static_cast<unsigned>(imax64(1, imin64((pieces + 255) / 256, 1024))), static_cast<unsigned>(a.B));
  cache_commit_kernel<<<grid, 256, 0, stream>>>(a, vecs);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const EvictArgs& a, int64_t head_dim, int, cudaStream_t stream) {
  const int vecs = static_cast<int>(head_dim / 8);
  const int64_t rows = a.B * a.cache.heads;
  evict_select_kernel<<<static_cast<unsigned>(rows), kSelThreads, 0, stream>>>(a);
  const dim3 grid(static_cast<unsigned>(rows),
                  static_cast<unsigned>(imin64((static_cast<int64_t>(a.keep) * vecs + 255) / 256, 65535)));
  evict_gather_kernel<<<grid, 256, 0, stream>>>(a, vecs);
  return cudaGetLastError();
}

}  // namespace dflash2
