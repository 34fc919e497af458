// logits.cu -- what sampling parameters make of the target's logits, and the token
// counts that they read.
//
// logits_adjust: a CTA takes 2048 columns of one sequence and walks over its T nodes; a
// thread takes 8 columns.  What does not depend on the node (counts, bias) is read once for
// all of them.  The drafted tokens that fall among the CTA's columns, usually none, are
// listed in shared memory, and a thread that has one among its own adds to each node's counts
// those that the node sees.  Where out is logits, vectors that stay as
// they are are neither read nor written, and vectors of which nothing is allowed only written.
#include "launch.h"
#include "serve.h"

namespace dflash2 {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 8;                // columns of a thread
constexpr int kBlockCols = kThreads * kCols;
constexpr int kRows = 4;                // rows of a thread under way at once

struct Draft {
  int16_t col;                          // of the CTA's columns
  int16_t node;
};

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(lo))) |
         static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(hi))) << 16;
}

__global__ void __launch_bounds__(kThreads) logits_adjust_kernel(const __grid_constant__ LogitsArgs a, int32_t blocks_per_seq) {
  __shared__ Draft drafts[kMaxNodes];
  __shared__ int32_t num_drafts;
  const int64_t b = blockIdx.x / blocks_per_seq;
  const int32_t block = blockIdx.x % blocks_per_seq, c0 = block * kBlockCols;
  const int32_t col = c0 + threadIdx.x * kCols;
  const bool inplace = a.out == a.logits;
  if (threadIdx.x == 0) num_drafts = 0;
  pdl_wait();
  pdl_launch_dependents();
  if (a.tokens != nullptr) {
    __syncthreads();
    if (threadIdx.x < a.T) {
      const int32_t tok = a.tokens[b * a.T + threadIdx.x];
      if (tok < 0 || tok >= a.V) {
        if (block == 0) raise_error(a.err, DFLASH2_DEVERR_BAD_TOKEN);
      } else if (tok >= c0 && tok < c0 + kBlockCols) {
        drafts[atomicAdd(&num_drafts, 1)] = {static_cast<int16_t>(tok - c0), static_cast<int16_t>(threadIdx.x)};
      }
    }
  }
  __syncthreads();
  if (col >= a.V) return;
  const int32_t cols = min(kCols, a.V - col);

  int32_t count[kCols] = {};
  float bias[kCols] = {};
  bool some = false;                    // whether any of the columns changes at every node
  if (a.counts != nullptr) {            // (16-byte vectors that start inside a row are read whole)
    const int4* src = reinterpret_cast<const int4*>(a.counts + b * a.counts_ld + col);
    const int4 x = src[0], y = cols > 4 ? src[1] : make_int4(0, 0, 0, 0);
    count[0] = x.x, count[1] = x.y, count[2] = x.z, count[3] = x.w;
    count[4] = y.x, count[5] = y.y, count[6] = y.z, count[7] = y.w;
  }
  if (a.bias != nullptr) {
    const float4* src = reinterpret_cast<const float4*>(a.bias + b * a.bias_ld + col);
    const float4 x = src[0], y = cols > 4 ? src[1] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    bias[0] = x.x, bias[1] = x.y, bias[2] = x.z, bias[3] = x.w;
    bias[4] = y.x, bias[5] = y.y, bias[6] = y.z, bias[7] = y.w;
  }
#pragma unroll
  for (int i = 0; i < kCols; ++i) some |= (count[i] != 0 || bias[i] != 0.0f) && i < cols;
  bool drafted = false;                 // whether one of the columns is a node's token
  for (int i = 0; i < num_drafts; ++i) drafted |= drafts[i].col >> 3 == threadIdx.x;
  const float repetition = a.repetition == nullptr ? 1.0f : a.repetition[b];
  const float frequency = a.frequency == nullptr ? 0.0f : a.frequency[b];
  const float presence = a.presence == nullptr ? 0.0f : a.presence[b];
  const uint8_t* allowed = a.allowed == nullptr
                               ? nullptr
                               : reinterpret_cast<const uint8_t*>(a.allowed + b * a.allowed_b) + (col >> 3);
  const uint16_t* src = a.logits + b * a.x_b + col;
  uint16_t* dst = a.out + b * a.out_b + col;
  const uint32_t full = (1u << cols) - 1;

  for (int32_t t0 = 0; t0 < a.T; t0 += kRows) {
    uint32_t may[kRows];
    uint4 w[kRows];
    bool change[kRows];
#pragma unroll
    for (int y = 0; y < kRows; ++y)
      may[y] = t0 + y < a.T && allowed != nullptr ? allowed[(t0 + y) * a.allowed_t * 4] & full : full;
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
      change[y] = some || drafted || may[y] != full;
      w[y] = make_uint4(0, 0, 0, 0);
      if (t0 + y < a.T && may[y] != 0 && (change[y] || !inplace))
        w[y] = *reinterpret_cast<const uint4*>(src + (t0 + y) * a.x_t);
    }
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
      const int32_t t = t0 + y;
      if (t >= a.T || (inplace && !change[y])) continue;
      if (change[y]) {
        int32_t n[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) n[i] = count[i];
        if (drafted) {
          uint64_t sees[2];
          if (a.mask == nullptr) {
            sees[0] = t >= 63 ? ~0ull : (2ull << t) - 1;
            sees[1] = t < 64 ? 0ull : t >= 127 ? ~0ull : (2ull << (t - 64)) - 1;
          } else {
            const int words = (a.T + 63) >> 6;
            const uint64_t* m = a.mask + (b * a.T + t) * words;
            sees[0] = m[0];
            sees[1] = words > 1 ? m[1] : 0ull;
          }
          for (int i = 0; i < num_drafts; ++i)
            if (drafts[i].col >> 3 == threadIdx.x && (sees[drafts[i].node >> 6] >> (drafts[i].node & 63) & 1ull)) {
#pragma unroll
              for (int k = 0; k < kCols; ++k) n[k] += (drafts[i].col & 7) == k ? 1 : 0;
            }
        }
        uint32_t* e = &w[y].x;
#pragma unroll
        for (int i = 0; i < kCols; i += 2) {
          float x[2] = {__uint_as_float(e[i / 2] << 16), __uint_as_float(e[i / 2] & 0xFFFF0000u)};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (n[i + k] != 0) {
              const int32_t emitted = n[i + k] & 0x7FFFFFFF;
              x[k] = x[k] > 0.0f ? x[k] / repetition : x[k] * repetition;
              if (emitted > 0) x[k] = x[k] - frequency * static_cast<float>(emitted) - presence;
            }
            if (bias[i + k] != 0.0f) x[k] += bias[i + k];
            if (!(may[y] >> (i + k) & 1u)) x[k] = -INFINITY;
          }
          e[i / 2] = pack(x[0], x[1]);
        }
      }
      if (cols == kCols) {
        *reinterpret_cast<uint4*>(dst + t * a.out_t) = w[y];
      } else {
        const uint16_t* e = reinterpret_cast<const uint16_t*>(&w[y]);
#pragma unroll
        for (int i = 0; i < kCols; ++i)
          if (i < cols) dst[t * a.out_t + i] = e[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// counts: a thread takes a token.  Additions and ORs of whole numbers give the same result in any order.  A
// prompt's common tokens come thousands of times: once a flag is set, later ones
// only read it.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) token_counts_kernel(const CountArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t x = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (x >= a.B * a.N) return;
  const int64_t b = static_cast<uint32_t>(x) / static_cast<uint32_t>(a.N);
  const int32_t i = static_cast<int32_t>(x - b * a.N);
  const int32_t count = a.count == nullptr ? a.N : kv_clamp(a.count[b], a.N, i == 0 ? a.err : nullptr);
  if (i >= count) return;
  const int32_t tok = a.tokens[b * a.N + (a.path == nullptr ? i : clamp_node(a.path[x], a.N, a.err))];
  if (tok < 0 || tok >= a.V) {
    raise_error(a.err, DFLASH2_DEVERR_BAD_TOKEN);
    return;
  }
  int32_t* at = a.counts + b * a.counts_ld + tok;
  if (!a.prompt)
    atomicAdd(at, 1);
  else if (*static_cast<volatile int32_t*>(at) >= 0)
    atomicOr(at, static_cast<int32_t>(0x80000000u));
}

}  // namespace

cudaError_t launch_logits_adjust(const LogitsArgs& a, int, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(a.V) + kBlockCols - 1) / kBlockCols;
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B * blocks), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logits_adjust_kernel, a, static_cast<int32_t>(blocks));
}

cudaError_t launch_token_counts(const CountArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.B * a.N + kThreads - 1) / kThreads), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, token_counts_kernel, a);
}

}  // namespace dflash2
