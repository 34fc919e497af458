// tree_attn.cu -- attention from drafted nodes to a paged cache and to one
// another, the target's pass over a draft block.
//
//   z_x = scale <q, k_x>,  lse = log sum exp z_x,  out = sum exp(z_x - lse) v_x
//
// One warp per query row (b, t, hq).  The row's keys are taken one by one with
// the running maximum m and sum l of a softmax: o and l are multiplied by
// exp(m - m') when the maximum rises to m'.
#include "kvcache.cuh"
#include "launch.h"
#include "attn.h"

namespace dflash2 {
namespace {

template <int D>
__global__ void __launch_bounds__(256) tree_attn_kernel(const AttnArgs a) {
  constexpr int E = D / 32;   // elements per lane
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (row >= a.B * a.T * a.heads) return;
  const int hq = static_cast<int>(row % a.heads);
  const int t = static_cast<int>(row / a.heads % a.T);
  const int64_t b = row / a.heads / a.T;
  const int h = hq / a.group;
  float q[E], o[E];
  const uint16_t* qp = a.q + b * a.q_b + t * a.q_t + hq * a.q_h + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_bits_to_float(qp[e]) * a.scale;
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const auto take = [&](const uint16_t* k, const uint16_t* v) {
    float z = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) z += q[e] * bf16_bits_to_float(k[lane * E + e]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, s);
    if (z == -INFINITY) return;
    const float m1 = fmaxf(m, z);   // a NaN z leaves m alone and makes l NaN
    const float f = expf(m - m1), p = expf(z - m1);
    m = m1;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * bf16_bits_to_float(v[lane * E + e]);
  };
  const int32_t n = kv_clamp(a.cache_len[b], a.cache.capacity, a.err);
  for (int32_t j = 0; j < n; ++j) {
    bool ok;
    const int64_t off = kv_offset(a.cache, b, j, h, a.err, &ok);
    take(a.cache.k + off, a.cache.v + off);
  }
  if (a.k_new != nullptr) {
    const int words = (a.T + 63) / 64;
    for (int s = 0; s < a.T; ++s) {
      const bool sees = a.mask == nullptr ? s <= t : (a.mask[(b * a.T + t) * words + s / 64] >> (s % 64)) & 1;
      const int64_t off = b * a.new_b + s * a.new_t + h * a.new_h;
      if (sees) take(a.k_new + off, a.v_new + off);
    }
  }
  const float r = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[row * D + lane * E + e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * r));
  if (a.lse != nullptr && lane == 0) a.lse[row] = m + logf(l);
}

}  // namespace

size_t tree_attn_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int) { return 0; }

cudaError_t launch_tree_attn(const AttnArgs& a, int64_t head_dim, void*, int, cudaStream_t stream) {
  const int64_t blocks = (a.B * a.T * a.heads + 7) / 8;
  if (head_dim == 64)
    tree_attn_kernel<64><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
  else
    tree_attn_kernel<128><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dflash2
