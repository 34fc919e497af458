// prefix_attn.cu -- the attention of tree_attn.cu for batches whose sequences share a
// beginning, whose keys and values are then read and multiplied once for the group.
//
// What is summed is cut in two, and the two sums of a row are joined like the parts of a
// split axis (exp's sums with their maxima): the keys of the group's shared positions, as
// whole tiles of 128, for the query rows of all its sequences' nodes, stacked; and each
// sequence's own keys from there on (the shared positions after the last whole tile among
// them) with the drafted nodes.  Both are stretches of items (kv head, pair of row tiles) in
// one list, the prefixes first.  All their units, weighed by what they cost, are cut into
// equal runs, one per CTA, so that the few long items of a prefix and the many short ones of
// the sequences fill the GPU together: the former is bound by the tensor cores, the latter by memory.
//   prefix_plan_kernel   one CTA: the list, with the cost of everything before each stretch
//   tree_attn_kernel     kShared: every item's sums to the workspace
//   prefix_join_kernel   a warp per row of the output: adds its parts, own keys first, in order
// The same inputs give the same bits on every call.
#include "tree_attn.cuh"

namespace dflash2 {
namespace {

constexpr int kPlanThreads = 1024;

struct PrefixPlan {
  PrefixArgs a;
  int32_t tpt;
  int32_t* shared;          // [groups] shared positions, clamped to the lengths of the group's sequences
  Stretch* stretches;       // [groups + B + 1]
};

__device__ __forceinline__ int32_t group_start(const PrefixArgs& a, int32_t g) {
  return a.start != nullptr ? a.start[g] : g == 0 ? 0 : static_cast<int32_t>(a.attn.B);
}

// The group of sequence b (the starts ascend from 0 to B).
__device__ __forceinline__ int32_t group_of(const PrefixArgs& a, int32_t b) {
  int32_t lo = 0, hi = a.groups;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (group_start(a, mid) <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixPlan p) {
  __shared__ uint32_t warp_sum[kPlanThreads / 32];
  const PrefixArgs& a = p.a;
  const AttnArgs& t = a.attn;
  const int32_t B = static_cast<int32_t>(t.B), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;
  for (int32_t g = tid; g < a.groups; g += kPlanThreads) {
    const int32_t s0 = group_start(a, g), s1 = group_start(a, g + 1);
    bad |= s0 < 0 || s1 < s0 || s1 > B || (g == 0 && s0 != 0) || (g == a.groups - 1 && s1 != B);
    p.shared[g] = kv_clamp(a.len[g], t.cache.capacity, t.err);
  }
  // starts that are none: nothing is shared
  const bool none = __syncthreads_or(bad) != 0 || a.groups == 0;
  if (none && a.groups > 0 && tid == 0) raise_error(t.err, DFLASH2_DEVERR_BAD_LENGTH);
  if (!none)
    for (int32_t b = tid; b < B; b += kPlanThreads) {
      const int32_t g = group_of(a, b), len = kv_clamp(t.cache_len[b], t.cache.capacity, t.err);
      if (len < p.shared[g]) {        // (only ever lowered: whatever is read here, the least one stays)
        raise_error(t.err, DFLASH2_DEVERR_BAD_LENGTH);
        atomicMin(&p.shared[g], len);
      }
    }
  __syncthreads();
  // shared tiles of a group: a sequence by itself shares nothing
  const auto tiles_of = [&](int32_t g) {
    return none || group_start(a, g + 1) - group_start(a, g) < 2 ? 0 : *static_cast<volatile int32_t*>(&p.shared[g]) / kTile;
  };
  uint32_t before = 0;
  for (int32_t v0 = 0; v0 < a.groups + B; v0 += kPlanThreads) {
    const int32_t v = v0 + tid;
    Stretch s = {};
    if (v < a.groups) {
      s.n = tiles_of(v);
      s.b = none ? 0 : group_start(a, v);
      s.node0 = s.b * t.T;
      s.nodes = none ? 0 : (group_start(a, v + 1) - s.b) * t.T;
      s.len = s.n * kTile;
    } else if (v < a.groups + B) {
      s.b = v - a.groups;
      s.node0 = s.b * t.T;
      s.nodes = t.T;
      s.tile0 = none ? 0 : tiles_of(group_of(a, s.b));
      s.len = kv_clamp(t.cache_len[s.b], t.cache.capacity, none ? t.err : nullptr);
      s.n = max(1, (s.len + kTile - 1) / kTile - s.tile0 + (t.k_new != nullptr ? 1 : 0));
      s.own = 1;
    }
    const uint32_t tiles = static_cast<uint32_t>((s.nodes + p.tpt - 1) / p.tpt);
    const uint32_t cost = static_cast<uint32_t>(s.n) * t.cache.heads * (kPair * (tiles >> 1) + kSingle * (tiles & 1));
    uint32_t incl = cost;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t sum = warp_sum[lane];       // 32 warps
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += o;
    }
    const uint32_t warps_before = __shfl_sync(0xFFFFFFFFu, sum, (warp + 31) & 31);
    s.cost = before + (warp > 0 ? warps_before : 0) + incl - cost;
    if (v < a.groups + B) p.stretches[v] = s;
    before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    __syncthreads();
  }
  if (tid == 0) {
    Stretch s = {};
    s.cost = before;
    p.stretches[a.groups + B] = s;
  }
}

constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const __grid_constant__ AttnPlan p, int32_t groups) {
  constexpr int E = D / 32;              // columns of a lane
  const AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  if (row >= a.B * a.T * a.heads) return;
  const bool shared = p.stretches[groups + row / (static_cast<int64_t>(a.T) * a.heads)].tile0 > 0;
  struct alignas(4 * E) Cols {
    float v[E];
  };
  PartSum<E> sum;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which == 1 && !shared) break;
    const float4 first = p.first_ml[which][row];
    const Cols o = *reinterpret_cast<const Cols*>(p.first_o[which] + row * D + lane * E);
    sum.add(first.x, first.y, o.v);
    const uint32_t more = __float_as_uint(first.z);
    const int32_t c1 = more >> 10 & 1023, at = more >> 20;
    for (int32_t c = (more & 1023) + 1; c <= c1; ++c) {
      const int64_t part = static_cast<int64_t>(c) * 2 * kTile + at;
      const float2 ml = p.part_ml[part];
      const Cols x = *reinterpret_cast<const Cols*>(p.part + part * D + lane * E);
      sum.add(ml.x, ml.y, x.v);
    }
  }
  sum.write(a, row, D, lane * E);
}

struct Layout {
  size_t stretches, shared, first_o[2], first_ml[2], part, part_ml, bytes;
};

Layout layout(int64_t B, int64_t T, int64_t heads, int64_t head_dim, int num_sms) {
  Layout l;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t x = at;
    at += (bytes + 255) / 256 * 256;
    return x;
  };
  const size_t rows = static_cast<size_t>(B) * T * heads, runs = static_cast<size_t>(imin64(num_sms, kMaxRuns));
  l.stretches = take((2 * static_cast<size_t>(B) + 1) * sizeof(Stretch));
  l.shared = take(static_cast<size_t>(B) * 4);
  for (int i = 0; i < 2; ++i) {
    l.first_o[i] = take(rows * head_dim * 4);
    l.first_ml[i] = take(rows * sizeof(float4));
  }
  l.part = take(runs * 2 * kTile * head_dim * 4);
  l.part_ml = take(runs * 2 * kTile * sizeof(float2));
  l.bytes = at;
  return l;
}

template <int D>
cudaError_t launch(const PrefixArgs& x, void* workspace, int num_sms, cudaStream_t stream) {
  const AttnArgs& a = x.attn;
  const Layout l = layout(a.B, a.T, a.heads, D, num_sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const Tiling t = tile_rows(a.T, a.group);
  PrefixPlan plan;
  plan.a = x;
  plan.tpt = t.tpt;
  plan.shared = reinterpret_cast<int32_t*>(ws + l.shared);
  plan.stretches = reinterpret_cast<Stretch*>(ws + l.stretches);
  AttnPlan p = {};
  p.a = a;
  p.tpt = t.tpt;
  p.areas = 2;
  p.c = a.scale * 1.4426950408889634f;
  p.box_rows = box_rows(a.cache);
  p.q_box_bytes = static_cast<uint32_t>(t.tpt * a.group) * D * 2;
  p.stretches = plan.stretches;
  p.num_stretches = x.groups + static_cast<int32_t>(a.B);
  for (int i = 0; i < 2; ++i) {
    p.first_o[i] = reinterpret_cast<float*>(ws + l.first_o[i]);
    p.first_ml[i] = reinterpret_cast<float4*>(ws + l.first_ml[i]);
  }
  p.part = reinterpret_cast<float*>(ws + l.part);
  p.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  Maps m;
  if (!make_maps<D>(a, t.tpt, p.box_rows, a.B * a.T, 1, &m)) return cudaErrorInvalidValue;
  const size_t smem = Cfg<D>::kRing + sizeof(AttnSmem);
  cudaError_t e = set_smem_limit<tree_attn_kernel<D, kShared>>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kPlanThreads, 1, 1);
  e = cudaLaunchKernelEx(&cfg, prefix_plan_kernel, plan);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(imin64(num_sms, kMaxRuns)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, kShared>, m.q, m.k, m.v, m.kn, m.vn, p);
  if (e != cudaSuccess) return e;
  const int64_t rows = a.B * a.T * a.heads, per_cta = kJoinThreads / 32;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + per_cta - 1) / per_cta), 1, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prefix_join_kernel<D>, p, x.groups);
}

}  // namespace

int64_t prefix_attn_units(int64_t B, int64_t T, int64_t group, int64_t kv_heads, int64_t capacity) {
  const Tiling t = tile_rows(T, group);
  // the prefixes' row tiles: those of all nodes together, and one more for each group
  return kv_heads * (capacity / kTile + 2) * (B * t.pairs + (B * T + t.tpt - 1) / t.tpt / 2 + B + 1);
}

size_t prefix_attn_workspace_bytes(int64_t B, int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim, int num_sms) {
  return heads / kv_heads > kTile ? 0 : layout(B, T, heads, head_dim, num_sms).bytes;
}

cudaError_t launch_prefix_attn(const PrefixArgs& a, int64_t head_dim, void* workspace, int num_sms, cudaStream_t stream) {
  return head_dim == 64 ? launch<64>(a, workspace, num_sms, stream) : launch<128>(a, workspace, num_sms, stream);
}

}  // namespace dflash2
