// attn.h -- arguments and launchers of the cache operators (tree attention,
// commit, scores, eviction); not exported.
#pragma once

#include <cuda_runtime.h>

#include "kvcache.cuh"

namespace dflash2 {

struct AttnArgs {
  const uint16_t* q;
  int64_t q_b, q_t, q_h;          // strides, elements
  KvView cache;
  const int32_t* cache_len;
  const uint16_t* k_new;          // nullptr: the cache alone
  const uint16_t* v_new;
  int64_t new_b, new_t, new_h;
  const uint64_t* mask;           // nullptr: a chain
  int64_t B;
  int32_t T, heads, group;
  float scale;
  uint16_t* out;
  float* lse;
  uint32_t* err;
};

struct ScoresArgs {
  const uint16_t* q;
  int64_t q_b, q_t, q_h;
  const float* lse;
  KvView cache;
  const int32_t* cache_len;
  const int32_t* count;           // nullptr: T
  const int32_t* path;            // nullptr: the identity
  int64_t B;
  int32_t T, heads, group;
  float scale;
  float* scores;
  int64_t scores_ld;
  uint32_t* err;
};

struct CommitArgs {
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t new_b, new_t, new_h;
  KvView cache;
  const int32_t* cache_len;
  const int32_t* count;
  const int32_t* path;
  int64_t B;
  int32_t T;
  float* scores;
  int64_t scores_ld;
  int32_t* new_len;
  uint32_t* err;
};

struct EvictArgs {
  const float* scores;
  int64_t scores_ld;
  KvView cache, dst;
  const int32_t* cache_len;
  int64_t B;
  int32_t keep, recent;
  int32_t* kept;
  int32_t* new_len;
  float* dst_scores;
  int64_t dst_ld;
  uint32_t* err;
};

struct PrefixArgs {
  AttnArgs attn;
  const int32_t* start;           // [groups + 1] first sequence of each group; nullptr: one group
  const int32_t* len;             // [groups] shared positions
  int32_t groups;
};

// Most key tiles that a call's items can have: fewer than 2^31.
int64_t tree_attn_units(int64_t B, int64_t T, int64_t group, int64_t kv_heads, int64_t capacity);
size_t tree_attn_workspace_bytes(int64_t B, int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim, int num_sms);
cudaError_t launch_tree_attn(const AttnArgs& a, int64_t head_dim, void* workspace, int num_sms, cudaStream_t stream);
size_t prefix_attn_workspace_bytes(int64_t B, int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim, int num_sms);
cudaError_t launch_prefix_attn(const PrefixArgs& a, int64_t head_dim, void* workspace, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_scores(const ScoresArgs& a, int64_t head_dim, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_commit(const CommitArgs& a, int64_t head_dim, cudaStream_t stream);
cudaError_t launch_cache_evict(const EvictArgs& a, int64_t head_dim, int num_sms, cudaStream_t stream);

}  // namespace dflash2
