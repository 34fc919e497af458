// rope.cu -- rotary positions, and the append of rotated keys and plain values to
// the cache.
//
//   y_1 = f (x_1 cos a - x_2 sin a),  y_2 = f (x_2 cos a + x_1 sin a),  a = 2 pi position rate
//
// The angle: rates are turns per position times 2^64, so position * rate in 64-bit
// arithmetic drops whole turns and nothing else; its upper 32 bits as a signed
// fraction of half a turn go to sincospif.  In fp32 radians the product would be off
// by 2^-24 of the angle, 0.008 at position 131072, as much as bf16's own rounding.
//
// A CTA takes `tokens` consecutive tokens and a stretch of their pieces.  A piece is two
// vectors of kE elements that hold kE whole pairs in either layout: vectors v and v +
// rd / 2 / kE of a head (half), or 2 v and 2 v + 1 (interleaved); after the rotated pieces a head's
// remaining elements are copied two vectors a piece.  The CTA first computes its tokens'
// cos and sin into shared memory, once for all heads, with its first pieces' loads in
// flight.  The append's pieces are those of the queries, the keys and the values, in this order.
#include "launch.h"
#include "serve.h"

namespace dflash2 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;           // tokens of a CTA
constexpr int kMaxRotary = 512;

// kE bf16 elements.
template <int kE>
struct Vec;
template <>
struct Vec<8> {
  uint4 w;
};
template <>
struct Vec<4> {
  uint2 w;
};
template <>
struct Vec<2> {
  uint32_t w;
};
template <>
struct Vec<1> {
  uint16_t w;
};

template <int kE>
__device__ __forceinline__ Vec<kE> load_vec(const uint16_t* p) {
  return *reinterpret_cast<const Vec<kE>*>(p);
}
template <int kE>
__device__ __forceinline__ void store_vec(uint16_t* p, const Vec<kE>& v) {
  *reinterpret_cast<Vec<kE>*>(p) = v;
}
template <int kE>
__device__ __forceinline__ void widen(const Vec<kE>& v, float* x) {
  const uint16_t* e = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
  for (int i = 0; i < kE; ++i) x[i] = bf16_bits_to_float(e[i]);
}
template <int kE>
__device__ __forceinline__ Vec<kE> narrow(const float* x) {
  Vec<kE> v;
  uint16_t* e = reinterpret_cast<uint16_t*>(&v);
#pragma unroll
  for (int i = 0; i < kE; ++i) e[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x[i]));
  return v;
}

// What a CTA does: tokens [first, first + n) of the B T, and of each the pieces [p0, p1).
struct Split {
  int32_t tokens;            // per CTA
  int32_t chunks;            // CTAs that share the same tokens
  int32_t pieces;            // of a token
  int32_t per_chunk;
};

// Positions that a sequence can hold.
__device__ __forceinline__ int32_t append_limit(const RotateArgs& a) {
  return a.scores != nullptr && a.scores_ld < a.cache.capacity ? static_cast<int32_t>(a.scores_ld) : a.cache.capacity;
}

// One piece under way: where it goes, and its two vectors.
template <int kE>
struct Piece {
  uint16_t* dst;             // nullptr: none
  Vec<kE> a, b;
  int32_t apart;             // elements from the first vector to the second
  int32_t angle;             // index of its first pair's cos and sin, or -1: a copy
};

template <int kE, bool kAppend>
__device__ __forceinline__ void load_piece(const RotateArgs& a, const Split& sp, uint32_t first, int32_t n, int32_t at,
                                           int32_t width, Piece<kE>* pc) {
  pc->dst = nullptr;
  if (at >= n * width) return;
  const int32_t tok = at / width;
  const int32_t x = blockIdx.x % sp.chunks * sp.per_chunk + at - tok * width;
  const uint32_t token = first + tok, b = token / static_cast<uint32_t>(a.T);
  const int32_t t = static_cast<int32_t>(token - b * a.T);
  const int32_t per_head = a.dim / (2 * kE);
  const int32_t head = x / per_head, v = x - head * per_head;
  const bool rotated = v < a.rope.rd / (2 * kE);
  int32_t e0 = 2 * kE * v;
  pc->apart = kE;
  pc->angle = -1;
  if (rotated) {
    if (!a.rope.interleaved) {
      e0 = kE * v;
      pc->apart = a.rope.rd >> 1;
    }
    pc->angle = tok * (a.rope.rd >> 1) + kE * v;
  }
  const uint16_t* src;
  if (!kAppend || head < a.heads) {
    if (kAppend && a.count != nullptr && t >= a.count[b]) return;
    src = a.x + b * a.x_b + t * a.x_t + head * a.x_h;
    pc->dst = a.out + b * a.out_b + t * a.out_t + head * a.out_h + e0;
  } else {
    const int32_t limit = append_limit(a), len = kv_clamp(a.cache_len[b], limit, nullptr);
    if ((a.count != nullptr && t >= a.count[b]) || t >= limit - len) return;
    const bool value = head >= a.heads + a.cache.heads;
    const int32_t h = head - a.heads - (value ? a.cache.heads : 0);
    bool ok;
    const int64_t to = kv_offset(a.cache, b, len + t, h, a.err, &ok);
    if (!value && v == 0 && a.scores != nullptr) a.scores[(static_cast<int64_t>(b) * a.cache.heads + h) * a.scores_ld + len + t] = 0.0f;
    if (!ok) return;
    if (value) {                       // plain vectors, side by side
      e0 = 2 * kE * v;
      pc->apart = kE;
      pc->angle = -1;
    }
    src = (value ? a.v_new : a.k_new) + b * a.new_b + t * a.new_t + h * a.new_h;
    pc->dst = (value ? a.cache.v : a.cache.k) + to + e0;
  }
  pc->a = load_vec<kE>(src + e0);
  pc->b = load_vec<kE>(src + e0 + pc->apart);
}

template <int kE>
__device__ __forceinline__ void store_piece(const RotateArgs& a, const Piece<kE>& pc, const float2* cs) {
  if (pc.dst == nullptr) return;
  if (pc.angle < 0) {
    store_vec<kE>(pc.dst, pc.a);
    store_vec<kE>(pc.dst + pc.apart, pc.b);
    return;
  }
  float x[2 * kE], y[2 * kE];
  widen<kE>(pc.a, x);
  widen<kE>(pc.b, x + kE);
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    const float2 c = cs[pc.angle + i];
    // half: pair (i, kE + i); interleaved: (2 i, 2 i + 1)
    const float x1 = a.rope.interleaved ? x[2 * i] : x[i], x2 = a.rope.interleaved ? x[2 * i + 1] : x[kE + i];
    const float y1 = x1 * c.x - x2 * c.y, y2 = x2 * c.x + x1 * c.y;
    if (a.rope.interleaved) {
      y[2 * i] = y1;
      y[2 * i + 1] = y2;
    } else {
      y[i] = y1;
      y[kE + i] = y2;
    }
  }
  store_vec<kE>(pc.dst, narrow<kE>(y));
  store_vec<kE>(pc.dst + pc.apart, narrow<kE>(y + kE));
}

template <int kE, bool kAppend>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateArgs a, const Split sp) {
  __shared__ float2 cs[kMaxTokens * (kMaxRotary / 2)];
  constexpr int kBatch = 2;              // pieces of a thread under way at once
  const uint32_t first = blockIdx.x / sp.chunks * sp.tokens;           // B T < 2^31
  const int32_t n = static_cast<int32_t>(imin64(sp.tokens, a.B * a.T - first));
  const int32_t p0 = blockIdx.x % sp.chunks * sp.per_chunk;
  const int32_t width = min(sp.per_chunk, sp.pieces - p0);   // pieces of a token that are this CTA's
  pdl_wait();
  pdl_launch_dependents();
  Piece<kE> pc[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) load_piece<kE, kAppend>(a, sp, first, n, threadIdx.x + i * kThreads, width, &pc[i]);
  const int32_t half = a.rope.rd >> 1;
  for (int32_t x = threadIdx.x; x < n * half; x += kThreads) {
    const int32_t tok = x / half;
    const uint32_t token = first + tok, b = token / static_cast<uint32_t>(a.T);
    const int64_t position = static_cast<int64_t>(a.base == nullptr ? 0 : a.base[b]) +
                             (a.depth == nullptr ? static_cast<int32_t>(token - b * a.T) : a.depth[token]);
    const uint64_t turn = static_cast<uint64_t>(position) * __ldg(a.rope.turns + (x - tok * half));
    const int32_t part = static_cast<int32_t>(static_cast<uint32_t>((turn + (1ull << 31)) >> 32));   // of a turn, times 2^32
    float s, c;
    sincospif(static_cast<float>(part) * 4.656612873077393e-10f, &s, &c);
    cs[x] = make_float2(c * a.rope.factor, (a.inverse ? -s : s) * a.rope.factor);
  }
  if (kAppend)
    for (int64_t b = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; b < a.B; b += static_cast<int64_t>(gridDim.x) * kThreads) {
      const int32_t limit = append_limit(a), len = kv_clamp(a.cache_len[b], limit, a.err);
      const int32_t count = a.count == nullptr ? a.T : kv_clamp(a.count[b], a.T, a.err);
      if (count > limit - len) raise_error(a.err, DFLASH2_DEVERR_BAD_LENGTH);
      a.new_len[b] = len + min(count, limit - len);
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBatch; ++i) store_piece<kE>(a, pc[i], cs);
  for (int32_t at = threadIdx.x + kBatch * kThreads; at < n * width; at += kBatch * kThreads) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) load_piece<kE, kAppend>(a, sp, first, n, at + i * kThreads, width, &pc[i]);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) store_piece<kE>(a, pc[i], cs);
  }
}

template <int kE, bool kAppend>
cudaError_t launch(const RotateArgs& a, int num_sms, cudaStream_t stream) {
  Split sp;
  const int64_t all = a.B * a.T;
  const int64_t heads = a.heads + (kAppend ? 2 * static_cast<int64_t>(a.cache.heads) : 0);
  sp.pieces = static_cast<int32_t>(heads * (a.dim / (2 * kE)));
  // several tokens a CTA where there are CTAs enough; else the pieces of a token are shared out
  sp.tokens = all >= static_cast<int64_t>(kMaxTokens) * 8 * num_sms ? kMaxTokens : 1;
  sp.chunks = 1;
  if (sp.tokens == 1) sp.chunks = static_cast<int32_t>(imin64((sp.pieces + 2 * kThreads - 1) / (2 * kThreads), ((int64_t(1) << 31) - 1) / imax64(all, 1)));
  sp.chunks = sp.chunks < 1 ? 1 : sp.chunks;
  sp.per_chunk = (sp.pieces + sp.chunks - 1) / sp.chunks;
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(imax64(1, (all + sp.tokens - 1) / sp.tokens * sp.chunks)), 1, 1);   // (T = 0: new_len)
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotate_kernel<kE, kAppend>, a, sp);
}

// Elements of a vector: the widest of which whole pieces make up both the rotated part
// and the rest of a head.
template <bool kAppend>
cudaError_t dispatch(const RotateArgs& a, int num_sms, cudaStream_t stream) {
  const auto fits = [&](int e) { return a.rope.rd % (2 * e) == 0 && a.dim % (2 * e) == 0; };
  if (fits(8)) return launch<8, kAppend>(a, num_sms, stream);
  if (fits(4)) return launch<4, kAppend>(a, num_sms, stream);
  if (fits(2)) return launch<2, kAppend>(a, num_sms, stream);
  return launch<1, kAppend>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope(const RotateArgs& a, int num_sms, cudaStream_t stream) { return dispatch<false>(a, num_sms, stream); }
cudaError_t launch_cache_append(const RotateArgs& a, int num_sms, cudaStream_t stream) {
  return dispatch<true>(a, num_sms, stream);
}

}  // namespace dflash2
