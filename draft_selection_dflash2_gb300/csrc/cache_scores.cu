// cache_scores.cu -- the attention weight that each cached position received
// from a verified block, added to its running total:
//
//   scores[b,h,j] += sum_r exp(scale <q_r, k_j> - lse_r)
//
// over the rows r = (accepted node, query head of the group) of h.  One warp per
// position, rows in order.
#include "attn.h"
#include "launch.h"

namespace dflash2 {
namespace {

template <int D>
__global__ void __launch_bounds__(256) cache_scores_kernel(const ScoresArgs a, int64_t limit) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.x % a.cache.heads;
  const int64_t b = blockIdx.x / a.cache.heads;
  const int32_t n = kv_clamp(a.cache_len[b], static_cast<int32_t>(limit), a.err);
  const int32_t count = a.count == nullptr ? a.T : kv_clamp(a.count[b], a.T, a.err);
  for (int32_t j = blockIdx.y * 8 + (threadIdx.x >> 5); j < n; j += gridDim.y * 8) {
  bool ok;
  const uint16_t* kp = a.cache.k + kv_offset(a.cache, b, j, h, a.err, &ok) + lane * E;
  float k[E];
#pragma unroll
  for (int e = 0; e < E; ++e) k[e] = bf16_bits_to_float(kp[e]) * a.scale;
  float w = 0.0f;
  for (int i = 0; i < count; ++i) {
    const int t = a.path == nullptr ? i : clamp_node(a.path[b * a.T + i], a.T, a.err);
    for (int g = 0; g < a.group; ++g) {
      const int hq = h * a.group + g;
      const uint16_t* qp = a.q + b * a.q_b + t * a.q_t + hq * a.q_h + lane * E;
      float z = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) z += k[e] * bf16_bits_to_float(qp[e]);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, s);
      const float lse = a.lse[(b * a.T + t) * a.heads + hq];
      if (lse != -INFINITY) w += expf(z - lse);
    }
  }
  if (lane == 0) a.scores[(b * a.cache.heads + h) * a.scores_ld + j] += w;
  }
}

}  // namespace

cudaError_t launch_cache_scores(const ScoresArgs& a, int64_t head_dim, int, cudaStream_t stream) {
  const int64_t limit = imin64(a.cache.capacity, a.scores_ld);
  if (limit == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(a.B * a.cache.heads), static_cast<unsigned>(imin64((limit + 7) / 8, 65535)));
  if (head_dim == 64)
    cache_scores_kernel<64><<<grid, 256, 0, stream>>>(a, limit);
  else
    cache_scores_kernel<128><<<grid, 256, 0, stream>>>(a, limit);
  return cudaGetLastError();
}

}  // namespace dflash2
