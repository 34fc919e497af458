// serve.h -- arguments and launchers of the rotary, append, logit and count
// kernels; not exported.
#pragma once

#include <cuda_runtime.h>

#include "kvcache.cuh"

namespace dflash2 {

struct RopeView {
  const uint64_t* turns;          // nullptr: nothing is rotated
  int32_t rd;                     // rotated elements of a head (0 without a table)
  int32_t interleaved;
  float factor;
};

struct RotateArgs {
  RopeView rope;
  const uint16_t* x;              // rows that are rotated to `out` (heads = 0: none)
  int64_t x_b, x_t, x_h;
  uint16_t* out;
  int64_t out_b, out_t, out_h;
  const int32_t* base;            // position of node t: base[b] + depth[b, t] (nullptr: 0, and t)
  const int32_t* depth;
  int64_t B;
  int32_t T, heads, dim;
  bool inverse;
  // the append: keys that are rotated into the cache, values that are copied there
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t new_b, new_t, new_h;
  KvView cache;
  const int32_t* cache_len;
  const int32_t* count;
  float* scores;
  int64_t scores_ld;
  int32_t* new_len;
  uint32_t* err;
};

struct LogitsArgs {
  const uint16_t* logits;
  int64_t x_b, x_t;
  uint16_t* out;
  int64_t out_b, out_t;
  int64_t B;
  int32_t T, V;
  const int32_t* counts;
  int64_t counts_ld;
  const int32_t* tokens;
  const uint64_t* mask;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const float* bias;
  int64_t bias_ld;
  const uint32_t* allowed;
  int64_t allowed_b, allowed_t;
  uint32_t* err;
};

struct CountArgs {
  const int32_t* tokens;
  const int32_t* count;
  const int32_t* path;
  int64_t B;
  int32_t N, V;
  bool prompt;
  int32_t* counts;
  int64_t counts_ld;
  uint32_t* err;
};

cudaError_t launch_rope(const RotateArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_append(const RotateArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_logits_adjust(const LogitsArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_token_counts(const CountArgs& a, cudaStream_t stream);

}  // namespace dflash2
