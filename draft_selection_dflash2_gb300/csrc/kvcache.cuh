// kvcache.cuh -- the device view of a paged key/value cache, shared by the
// attention, commit, score and eviction kernels.
#pragma once

#include "common.cuh"

namespace dflash2 {

constexpr int kMaxNodes = 128;   // drafted nodes per sequence (T)

struct KvView {
  uint16_t* k;
  uint16_t* v;
  int64_t page_stride, token_stride, head_stride;   // elements
  const int32_t* table;                             // nullptr: sequence b is page b
  int64_t table_ld;
  int32_t num_pages;
  int32_t page_size;
  int32_t page_shift;                               // log2(page_size) when there is a table
  int32_t capacity;                                 // positions of a sequence
  int32_t heads;
};

// The page of position j of sequence b; an id outside the cache is flagged and
// clamped (*ok = false).
__device__ __forceinline__ int32_t kv_page(const KvView& c, int64_t b, int32_t j, uint32_t* err, bool* ok) {
  *ok = true;
  if (c.table == nullptr) return static_cast<int32_t>(b);
  const int32_t p = c.table[b * c.table_ld + (j >> c.page_shift)];
  if (static_cast<uint32_t>(p) >= static_cast<uint32_t>(c.num_pages)) {
    raise_error(err, DFLASH2_DEVERR_BAD_PAGE);
    *ok = false;
    return p < 0 ? 0 : c.num_pages - 1;
  }
  return p;
}

// Element offset of position j, head h of sequence b (64 bits: caches pass 2^32 elements).
__device__ __forceinline__ int64_t kv_offset(const KvView& c, int64_t b, int32_t j, int32_t h, uint32_t* err, bool* ok) {
  const int64_t page = kv_page(c, b, j, err, ok);
  const int32_t off = c.table == nullptr ? j : j & (c.page_size - 1);
  return page * c.page_stride + off * c.token_stride + h * c.head_stride;
}

// A length or count clamped to [0, limit]; a clamped one is flagged.
__device__ __forceinline__ int32_t kv_clamp(int32_t n, int32_t limit, uint32_t* err) {
  if (n < 0 || n > limit) {
    raise_error(err, DFLASH2_DEVERR_BAD_LENGTH);
    return n < 0 ? 0 : limit;
  }
  return n;
}

__device__ __forceinline__ int32_t clamp_node(int32_t n, int32_t T, uint32_t* err) {
  if (n < 0 || n >= T) {
    raise_error(err, DFLASH2_DEVERR_BAD_NODE);
    return n < 0 ? 0 : T - 1;
  }
  return n;
}

}  // namespace dflash2
