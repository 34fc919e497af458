// host_checks.h -- the handle, and the host-side checks of arguments that the entry
// points share (api.cu, api_serve.cu); not exported.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "dflash2.h"
#include "attn.h"
#include "common.cuh"
#include "launch.h"

struct dflash2_handle {
  int device = 0;
  int num_sms = 0;
  uint32_t* err = nullptr;      // device error word
};

namespace {   // (each file that includes this has its own)

constexpr int64_t kMaxKvHeads = 4096;
constexpr int64_t kMaxElements = int64_t(1) << 36;   // of 4 bytes: no memory holds more
constexpr int64_t kMaxCapacity = (int64_t(1) << 31) - 256;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? DFLASH2_OK : DFLASH2_ERR_CUDA; }

// Launch errors are sticky per thread in the runtime; surface them as a status.
inline int launched(cudaError_t e) {
  if (e != cudaSuccess) return DFLASH2_ERR_CUDA;
  return from_cuda(cudaGetLastError());
}

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

inline bool bad_handle(const dflash2_handle* h) { return h == nullptr || h->err == nullptr; }

// Kernels launch on the calling thread's current device and write the handle's
// error word, which lives on the handle's device: a call made while another
// device is current is refused before anything launches.
inline int wrong_device(const dflash2_handle* h) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return DFLASH2_ERR_CUDA;
  return dev == h->device ? DFLASH2_OK : DFLASH2_ERR_INVALID_ARG;
}

// One NVTX range per compute call, named after the entry point, so a timeline
// (Nsight Systems, or any NVTX tool) shows the library's calls; without a tool
// attached a push/pop costs a few nanoseconds.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// A stride in elements between `extent` pieces of `least` elements each: of no
// effect when there is one piece, else a multiple of 8 that keeps them apart.
inline bool bad_stride(int64_t stride, int64_t extent, int64_t least) {
  return extent > 1 && (stride < least || stride >= (int64_t(1) << 38));
}
inline bool odd_stride(int64_t stride, int64_t extent) { return extent > 1 && stride % 8 != 0; }

// Checks a cache descriptor for B sequences and turns it into the device view.
inline int view_cache(const dflash2_kv_cache* c, int64_t B, dflash2::KvView* out) {
  if (c == nullptr || c->num_pages < 0 || c->page_size < 0 || c->heads <= 0 || c->max_pages < 0)
    return DFLASH2_ERR_INVALID_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || c->heads > kMaxKvHeads || c->num_pages >= (int64_t(1) << 31))
    return DFLASH2_ERR_UNSUPPORTED;
  const bool paged = c->block_table != nullptr;
  if (paged && (c->page_size < 16 || (c->page_size & (c->page_size - 1)) != 0)) return DFLASH2_ERR_UNSUPPORTED;
  if (c->page_size > kMaxCapacity || (paged && c->max_pages > kMaxCapacity / c->page_size))
    return DFLASH2_ERR_UNSUPPORTED;
  if (paged ? (c->table_ld < c->max_pages && B > 1) : c->num_pages < B) return DFLASH2_ERR_INVALID_ARG;
  const int64_t capacity = paged ? c->max_pages * c->page_size : c->page_size;
  if (capacity > 0 && c->num_pages > 0 && (!c->k || !c->v)) return DFLASH2_ERR_INVALID_ARG;
  if (capacity > 0 && c->num_pages == 0 && B > 0) return DFLASH2_ERR_INVALID_ARG;
  if (bad_stride(c->page_stride, c->num_pages, c->head_dim) || bad_stride(c->token_stride, c->page_size, c->head_dim) ||
      bad_stride(c->head_stride, c->heads, c->head_dim))
    return DFLASH2_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->block_table, 4) ||
      odd_stride(c->page_stride, c->num_pages) || odd_stride(c->token_stride, c->page_size) ||
      odd_stride(c->head_stride, c->heads))
    return DFLASH2_ERR_MISALIGNED;
  out->k = c->k;
  out->v = c->v;
  // strides of single pieces are never multiplied by more than 0: any valid one will do
  out->page_stride = c->num_pages > 1 ? c->page_stride : c->head_dim;
  out->token_stride = c->page_size > 1 ? c->token_stride : c->head_dim;
  out->head_stride = c->heads > 1 ? c->head_stride : c->head_dim;
  out->table = c->block_table;
  out->table_ld = c->table_ld;
  out->num_pages = static_cast<int32_t>(c->num_pages);
  out->page_size = static_cast<int32_t>(c->page_size);
  out->page_shift = 0;
  while (paged && (int64_t(1) << out->page_shift) < c->page_size) ++out->page_shift;
  out->capacity = static_cast<int32_t>(capacity);
  out->heads = static_cast<int32_t>(c->heads);
  return DFLASH2_OK;
}

// Whether n 4-byte elements at p and m at q share memory (null shares none).
inline bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
  const auto a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p != nullptr && q != nullptr && a < b + 4 * static_cast<uintptr_t>(m) && b < a + 4 * static_cast<uintptr_t>(n);
}

// Strides of a [B, T, n, d] bf16 operand.
struct RowStrides {
  int64_t b, t, h;
};

inline int check_rows(RowStrides* s, int64_t B, int64_t T, int64_t n, int64_t d) {
  if (bad_stride(s->b, B, d) || bad_stride(s->t, T, d) || bad_stride(s->h, n, d)) return DFLASH2_ERR_INVALID_ARG;
  if (odd_stride(s->b, B) || odd_stride(s->t, T) || odd_stride(s->h, n)) return DFLASH2_ERR_MISALIGNED;
  if (B <= 1) s->b = d;
  if (T <= 1) s->t = d;
  if (n <= 1) s->h = d;
  return DFLASH2_OK;
}

// What the query side of attention and scores shares.
inline int check_queries(int64_t B, int64_t T, int64_t heads, const dflash2_kv_cache* cache, float scale) {
  if (B < 0 || T < 0 || heads <= 0 || cache == nullptr || cache->heads <= 0 || heads % cache->heads != 0 ||
      !(scale > 0.0f) || scale > 1.0e38f)
    return DFLASH2_ERR_INVALID_ARG;
  if (T > dflash2::kMaxNodes || B > 65535 || heads / cache->heads > 128) return DFLASH2_ERR_UNSUPPORTED;
  return DFLASH2_OK;
}

}  // namespace
