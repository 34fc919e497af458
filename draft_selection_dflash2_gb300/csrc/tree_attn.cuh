// tree_attn.cuh -- what the attention kernels of tree_attn.cu and prefix_attn.cu share: the
// softmax of a chunk of keys, tiles that rows see in part, sums that have to be taken again,
// partial sums, and the tensor maps.  The mathematics stands at the head of tree_attn.cu.
#pragma once

#include "attn_common.cuh"
#include "launch.h"

namespace dflash2 {
namespace {   // (each file that includes this has its own instances)

constexpr int kThreads = 416;
constexpr int kChunk = 64;              // keys of an S product
constexpr int kMaxSlots = 10;
constexpr int kBufs = 2;                // S buffers per pipeline (a third one, at D = 64, gained nothing)
constexpr uint32_t kTmemO = 2 * kBufs * kChunk;   // first TMEM column of O: pipeline i's at kTmemO + i D
constexpr int kMaxRuns = 512;           // most CTAs
constexpr float kRescale = 8.0f;        // log2 of how far P may exceed 1

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                 // 128-byte column blocks of a row
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 10;       // ring of K and V tiles: 160 KB
  static constexpr size_t kRing = static_cast<size_t>(2 + kSlots) * kTileBytes;
};

// A chunk's S buffer, and how often that has been used before.
struct BufPos {
  int buf = 0;
  uint32_t use = 0;
  __device__ __forceinline__ void advance() {
    if (++buf == kBufs) {
      buf = 0;
      ++use;
    }
  }
  __device__ __forceinline__ BufPos before() const { return {buf == 0 ? kBufs - 1 : buf - 1, buf == 0 ? use - 1 : use}; }
};

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ bool finite_bf16(uint32_t bits) { return (bits & 0x7F80u) != 0x7F80u; }

// Zeroes the rows [from, to) of a V tile (this thread's share of `threads`).
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int to, int tid, int threads) {
  const int n = (to - from) * 8;   // 16-byte pieces per column block
#pragma unroll
  for (int half = 0; half < Cfg<D>::kHalves; ++half)
    for (int x = tid; x < n; x += threads)
      *reinterpret_cast<uint4*>(tile + half * kTile * 128 + from * 128 + x * 16) = make_uint4(0, 0, 0, 0);
}

// The warp's rows of O (`cols` columns at tm) times f.  Out of line: it is rarely called.
__device__ __noinline__ void rescale_rows(uint32_t tm, int cols, float f) {
#pragma unroll 1
  for (int x = 0; x < cols; x += 32) {
    float o[32];
    tmem_ld_x32(tm + x, o);
    tmem_ld_wait();
    pin(o);
#pragma unroll
    for (int w = 0; w < 32; w += 16) {
      uint32_t ob[16];
#pragma unroll
      for (int y = 0; y < 16; ++y) ob[y] = __float_as_uint(o[w + y] * f);
      tmem_st_x16(tm + x + w, ob);
    }
  }
}

// A sum's part v, to be weighted by f >= 0.  An infinity stays one where f underflows
// (the weights of the definition do not).
__device__ __forceinline__ float weighted(float v, float f) { return fabsf(v) < INFINITY ? v * f : v; }

// The nodes 64 y .. 64 y + 63 that the mask lets the row see.
__device__ __forceinline__ uint64_t mask_word(const AttnArgs& a, int64_t b, int node, bool row_ok, int y) {
  const int words = (a.T + 63) >> 6;
  return row_ok && y < words ? a.mask[(b * a.T + node) * words + y] : 0ull;
}
// Which of the keys 32 w .. 32 w + 31 come before `upto`, a bit each.
__device__ __forceinline__ uint32_t keys_before(int upto, int w) {
  const int k = upto - 32 * w;
  return k >= 32 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << k) - 1u;
}
// The keys 32 w .. 32 w + 31 of a tile that is not whole which the row sees: of `valid` cached keys, or of the drafted nodes.
__device__ __forceinline__ uint32_t seen_keys(const AttnArgs& a, bool drafted, int valid, int64_t b, int node, bool row_ok,
                                              int w) {
  const uint32_t see = keys_before(drafted && a.mask == nullptr ? min(valid, node + 1) : valid, w);
  return drafted && a.mask != nullptr ? see & static_cast<uint32_t>(mask_word(a, b, node, row_ok, w / 2) >> (w & 1) * 32) : see;
}

// Zeroes what is not finite of T drafted nodes' values (this thread's share of `threads`), and notes the nodes in bad.
template <int D>
__device__ __forceinline__ bool clear_nonfinite(uint8_t* v_tile, int T, int tid, int threads, uint32_t* bad) {
  bool any = false;
#pragma unroll
  for (int half = 0; half < Cfg<D>::kHalves; ++half)
    for (int x = tid; x < T * 8; x += threads) {
      uint4* at = reinterpret_cast<uint4*>(v_tile + half * kTile * 128 + x * 16);
      uint4 q = *at;
      uint32_t* e = &q.x;
      bool hit = false;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (!finite_bf16(e[y])) e[y] &= 0xFFFF0000u, hit = true;
        if (!finite_bf16(e[y] >> 16)) e[y] &= 0x0000FFFFu, hit = true;
      }
      if (hit) {
        *at = q;
        atomicOr(&bad[x >> 8], 1u << ((x >> 3) & 31));
        any = true;
      }
    }
  return any;
}

// Whether the row sees one of the bad nodes: seen(w) are the nodes 32 w .. 32 w + 31 that it sees.
template <class Seen>
__device__ __forceinline__ bool sees_bad(const uint32_t* bad, const Seen& seen) {
  uint32_t some = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w)
    if (bad[w] != 0) some |= seen(w) & bad[w];
  return some != 0;
}

// The V tile of a tile that is not whole, without what nobody may see.  A drafted tile is looked through by
// `threads` threads (tid), which meet() waits for; returns whether the row sees a node that was zeroed.
template <int D, class Seen, class Meet>
__device__ __forceinline__ bool see_tile(const AttnArgs& a, uint8_t* v_tile, bool drafted, int valid, int chunks, int tid,
                                         int threads, int r, uint32_t* bad, const Seen& seen, const Meet& meet) {
  if (!drafted) {
    zero_rows<D>(v_tile, valid, chunks * kChunk, r, kTile);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    return false;
  }
  if (tid < 4) bad[tid] = 0;
  __syncwarp();
  meet();
  clear_nonfinite<D>(v_tile, a.T, tid, threads, bad);
  __syncwarp();
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  meet();
  return sees_bad(bad, seen);
}

// The softmax of a chunk, of the thread's row: S (64 columns at tm_s) becomes P in two terms, and the row's maximum m and
// sum l move on.  sees(0), sees(1): which keys of each half the row sees, where not all (partial).  first: O (at tm_o) is not begun yet; else
// wait_products() returns when the products so far have been added to it.
template <int D, class Sees, class Wait>
__device__ __forceinline__ void softmax_chunk(uint32_t tm_sb, uint32_t tm_o, float scale, bool partial, const Sees& sees,
                                              bool first, bool row_ok, float* m, float* l, const Wait& wait_products) {
  float z[2][32];
  tmem_ld_x32(tm_sb, z[0]);
  tmem_ld_x32(tm_sb + 32, z[1]);
  tmem_ld_wait();
  pin(z[0]);
  pin(z[1]);
  if (partial) {
    const uint32_t v0 = sees(0), v1 = sees(1);
#pragma unroll
    for (int y = 0; y < 32; ++y) {
      if (!(v0 >> y & 1u)) z[0][y] = -INFINITY;
      if (!(v1 >> y & 1u)) z[1][y] = -INFINITY;
    }
  }
  float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // four chains of dependent maxima
#pragma unroll
  for (int y = 0; y < 32; ++y) tops[y & 3] = fmaxf(tops[y & 3], fmaxf(z[0][y], z[1][y]));
  const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale;
  if (first) {
    *m = top;
  } else if (__any_sync(0xFFFFFFFFu, row_ok && top > *m + kRescale)) {
    // a row's maximum rose far: the warp's O and l move to the new ones (rows of the
    // tile that are no query's hold whatever shared memory held, and have no say)
    const float m1 = fmaxf(*m, top);
    const float f = *m == -INFINITY ? 1.0f : exp2_approx(*m - m1);
    *m = m1;
    *l *= f;
    wait_products();
    __syncwarp();
    tc_fence_after();
    rescale_rows(tm_o, D, f);
  }
  const float mm = *m == -INFINITY ? 0.0f : *m;   // a row that has seen nothing: all its P are 2^-inf
  const uint64_t c2 = pack2(scale, scale), m2 = pack2(-mm, -mm);
  uint64_t sum0 = pack2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int y = 0; y < 32; y += 2) {
      const float2 e = unpack2(fma2(pack2(z[x][y], z[x][y + 1]), c2, m2));
      const float p0 = exp2_approx(e.x), p1 = exp2_approx(e.y);
      const uint64_t pp = pack2(p0, p1);
      if (y & 2)
        sum1 = add2(sum1, pp);
      else
        sum0 = add2(sum0, pp);
      // what P loses when it is rounded to bf16 is the second term
      const uint32_t h = pack_bf16(p0, p1);
      const float2 d = unpack2(add2(pp, pack2(-__uint_as_float(h << 16), -__uint_as_float(h & 0xFFFF0000u))));
      hi[y / 2] = h;
      lo[y / 2] = pack_bf16(d.x, d.y);
    }
    tmem_st_x16(tm_sb + 16 * x, hi);
    tmem_st_x16(tm_sb + kChunk / 2 + 16 * x, lo);
  }
  const float2 sum = unpack2(add2(sum0, sum1));
  *l += sum.x + sum.y;
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// The softmax of a quarter of a chunk: the 16 keys from 16 w on; P is 0 for the others.  sees(): which of the 16 the row sees.
template <int D, class Sees, class Wait>
__device__ __forceinline__ void softmax_quarter(uint32_t tm_sb, uint32_t tm_o, float scale, int w, bool partial,
                                                const Sees& sees, bool first, bool row_ok, float* m, float* l,
                                                const Wait& wait_products) {
  float z[16];
  tmem_ld_x16(tm_sb + 16 * w, z);
  tmem_ld_wait();
  asm volatile("" : "+f"(z[0]), "+f"(z[1]), "+f"(z[2]), "+f"(z[3]), "+f"(z[4]), "+f"(z[5]), "+f"(z[6]), "+f"(z[7]));
  asm volatile("" : "+f"(z[8]), "+f"(z[9]), "+f"(z[10]), "+f"(z[11]), "+f"(z[12]), "+f"(z[13]), "+f"(z[14]), "+f"(z[15]));
  if (partial) {
    const uint32_t v = sees();
#pragma unroll
    for (int y = 0; y < 16; ++y)
      if (!(v >> y & 1u)) z[y] = -INFINITY;
  }
  float tops[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int y = 0; y < 16; y += 2) tops[y / 2 & 1] = fmaxf(tops[y / 2 & 1], fmaxf(z[y], z[y + 1]));
  const float top = fmaxf(tops[0], tops[1]) * scale;
  if (first) {
    *m = top;
  } else if (__any_sync(0xFFFFFFFFu, row_ok && top > *m + kRescale)) {   // (see softmax_chunk)
    const float m1 = fmaxf(*m, top);
    const float f = *m == -INFINITY ? 1.0f : exp2_approx(*m - m1);
    *m = m1;
    *l *= f;
    wait_products();
    __syncwarp();
    tc_fence_after();
    rescale_rows(tm_o, D, f);
  }
  const float mm = *m == -INFINITY ? 0.0f : *m;
  float sum = 0.0f;
  uint32_t hi[8], lo[8], zero[8] = {};
#pragma unroll
  for (int y = 0; y < 16; y += 2) {
    const float p0 = exp2_approx(fmaf(z[y], scale, -mm)), p1 = exp2_approx(fmaf(z[y + 1], scale, -mm));
    sum += p0 + p1;
    const uint32_t b = pack_bf16(p0, p1);
    hi[y / 2] = b;
    lo[y / 2] = pack_bf16(p0 - __uint_as_float(b << 16), p1 - __uint_as_float(b & 0xFFFF0000u));
  }
  *l += sum;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if (x == w) {
      tmem_st_x8(tm_sb + 8 * x, hi);
      tmem_st_x8(tm_sb + kChunk / 2 + 8 * x, lo);
    } else {
      tmem_st_x8(tm_sb + 8 * x, zero);
      tmem_st_x8(tm_sb + kChunk / 2 + 8 * x, zero);
    }
  }
}

// <q, k> over D bf16 each.
template <int D>
__device__ __forceinline__ float dot_bf16(const uint16_t* q, const uint16_t* k) {
  float z = 0.0f;
#pragma unroll 4
  for (int x = 0; x < D; x += 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(q + x), b = *reinterpret_cast<const uint4*>(k + x);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      z = fmaf(bf16_bits_to_float(u[y]), bf16_bits_to_float(w[y]), z);
      z = fmaf(__uint_as_float(u[y] & 0xFFFF0000u), __uint_as_float(w[y] & 0xFFFF0000u), z);
    }
  }
  return z;
}

// Takes the sums of the run's rows that hold a non-finite value again, each by a warp of
// the softmax: 32 keys at a time, a lane each, then all lanes on each key's value.  Out of
// line: it is hardly ever called.
template <int D, class Plan, class Walk>
__device__ __noinline__ void sum_again(const Plan& p, Walk walk, uint8_t* ring) {
  constexpr int E = D / 32;              // columns of a lane
  const AttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  typename Walk::Segment g;
  while (walk.next(p, &g)) {
    const typename Walk::template Place<D> place(p, g, ring);
    for (int tile = 0; tile < g.tiles; ++tile) {
      const int node0 = (2 * g.pair + tile) * p.tpt, rows = min(p.tpt, g.num_nodes(a) - node0) * a.group;
#pragma unroll 1
      for (int r = (threadIdx.x >> 5) - 4; r < rows; r += 2 * kTile / 32) {
        const int t = r / a.group, node = node0 + t, hq = g.h * a.group + r - t * a.group;
        const int64_t orow = g.node(a, node) * a.heads + hq;
        uint16_t* out = a.out + orow * D + lane * E;
        float* part = reinterpret_cast<float*>(place.part(p, tile, r, orow) + lane * E / 4 * place.kStep) + lane * E % 4;
        bool finite = true;
#pragma unroll
        for (int e = 0; e < E; ++e) finite &= place.whole ? finite_bf16(out[e]) : fabsf(part[e]) < INFINITY;
        for (int k = 1; k < place.copies(); ++k) {
          const float* more = reinterpret_cast<const float*>(place.part(p, tile, r + k * 32, orow)) + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) finite &= fabsf(more[e]) < INFINITY;
        }
        if (__all_sync(0xFFFFFFFFu, finite)) continue;
        const uint16_t* q = a.q + g.q_row(a, node) + hq * a.q_h;
        float m = -INFINITY, l = 0.0f, o[E] = {};   // l: of the lane's keys
#pragma unroll 1
        for (int u = g.s; u < g.e; ++u) {
          const bool drafted = g.drafted(a, u);
          const int keys = g.keys(a, u);
#pragma unroll 1
          for (int x = lane; x - lane < keys; x += 32) {
            bool adds = x < keys;
            if (adds && drafted)
              adds = a.mask == nullptr ? x <= node
                                       : a.mask[(static_cast<int64_t>(g.b) * a.T + node) * ((a.T + 63) >> 6) + (x >> 6)] >>
                                                 (x & 63) & 1;
            const uint16_t* v = nullptr;
            float z = -INFINITY;
            if (adds) {
              bool ok;
              const int64_t at = drafted ? g.b * a.new_b + x * a.new_t + g.h * a.new_h
                                         : kv_offset(a.cache, g.b, g.position(u) + x, g.h, nullptr, &ok);
              v = (drafted ? a.v_new : a.cache.v) + at;
              z = dot_bf16<D>(q, (drafted ? a.k_new : a.cache.k) + at);
              adds = z * a.scale != -INFINITY;
            }
            float top = m;
            if (adds) top = fmaxf(top, z * p.c);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            const float f = m == -INFINITY ? 1.0f : exp2_approx(m - top);
            const float w = adds ? exp2_approx(fmaf(z, p.c, top == -INFINITY ? 0.0f : -top)) : 0.0f;
            m = top;
            l = l * f + w;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = weighted(o[e], f);
            for (uint32_t some = __ballot_sync(0xFFFFFFFFu, adds); some != 0; some &= some - 1) {
              const int y = __ffs(some) - 1;
              const auto* vy =
                  reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(v), y));
              const float wy = __shfl_sync(0xFFFFFFFFu, w, y);
#pragma unroll
              for (int e = 0; e < E; ++e) o[e] += weighted(bf16_bits_to_float(vy[lane * E + e]), wy);
            }
          }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        if (place.whole) {
#pragma unroll
          for (int e = 0; e < E; ++e) out[e] = __bfloat16_as_ushort(__float2bfloat16_rn(l == 0.0f ? 0.0f : o[e] / l));
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) part[e] = o[e];
          if (lane == 0) place.put_ml(p, tile, r, orow, m, -l);        // (see PartSum::add)
          for (int k = 1; k < place.copies(); ++k)
            if (lane == 0) place.put_ml(p, tile, r + k * 32, orow, -INFINITY, 0.0f);
        }
      }
    }
  }
}

// Partial sums of a row's N columns, added as the softmax adds keys.
template <int N>
struct PartSum {
  float m = -INFINITY, l = 0.0f, o[N] = {};
  bool odd = false;          // whether an infinity may be in o
  // Adds sums (m1, l1, v); with m1 = -inf they saw nothing, and v is not looked at.
  // A negative l1 says that v may hold infinities.
  __device__ __forceinline__ void add(float m1, float l1, const float (&v)[N]) {
    odd |= l1 < 0.0f;
    l1 = fabsf(l1);
    const bool some = m1 != -INFINITY;
    const float top = fmaxf(m, m1);
    // an infinity stays one where its weight underflows: that of the definition does not
    const float least = odd ? 1.4e-45f : 0.0f;
    const float f0 = m == -INFINITY ? 0.0f : fmaxf(exp2_approx(m - top), least);
    const float f1 = some ? fmaxf(exp2_approx(m1 - top), least) : 0.0f;
    m = top;
    l = l * f0 + (some || l1 != l1 ? l1 * (some ? f1 : 1.0f) : 0.0f);   // only NaN scores: l1 is NaN
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = fmaf(some ? v[k] : 0.0f, f1, o[k] * f0);
  }
  __device__ __forceinline__ void write(const AttnArgs& a, int64_t orow, int D, int x) const {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t out[N / 2];
#pragma unroll
    for (int k = 0; k < N; k += 2) out[k / 2] = pack_bf16(o[k] * inv, o[k + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + x);
    if constexpr (N == 8)
      *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    else if constexpr (N == 2)
      *dst = out[0];
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    if (x == 0 && a.lse != nullptr) a.lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
};

struct Tiling {
  int32_t tpt, row_tiles, pairs, areas;
};

inline Tiling tile_rows(int64_t T, int64_t group) {
  Tiling t;
  t.tpt = static_cast<int32_t>(kTile / group);
  t.row_tiles = static_cast<int32_t>((T + t.tpt - 1) / t.tpt);
  t.pairs = (t.row_tiles + 1) / 2;
  t.areas = t.row_tiles > 1 ? 2 : 1;
  return t;
}

// Rows of a box of K or V: a box lies in one page.
inline int32_t box_rows(const KvView& c) { return c.table != nullptr && c.page_size < kTile ? c.page_size : kTile; }

struct Maps {
  CUtensorMap q, k, v, kn, vn;
};

// The queries as `batches` times `nodes` nodes (strides q_b and q_t), boxes of tpt of them; pages, and drafted nodes.
template <int D>
bool make_maps(const AttnArgs& a, int32_t tpt, int32_t rows, int64_t nodes, int64_t batches, Maps* m) {
  const KvView& c = a.cache;
  const uint64_t qd[5] = {D, static_cast<uint64_t>(a.group), static_cast<uint64_t>(nodes),
                          static_cast<uint64_t>(c.heads), static_cast<uint64_t>(batches)};
  const uint64_t qs[4] = {static_cast<uint64_t>(a.q_h), static_cast<uint64_t>(a.q_t),
                          static_cast<uint64_t>(a.q_h) * a.group, static_cast<uint64_t>(a.q_b)};
  const uint32_t qb[5] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(tpt), 1, 1};
  if (!make_tmap_bf16_nd(&m->q, a.q, 5, qd, qs, qb)) return false;
  const uint64_t kd[4] = {D, static_cast<uint64_t>(imax64(c.page_size, 1)), static_cast<uint64_t>(c.heads),
                          static_cast<uint64_t>(imax64(c.num_pages, 1))};
  const uint64_t ks[3] = {static_cast<uint64_t>(c.token_stride), static_cast<uint64_t>(c.head_stride),
                          static_cast<uint64_t>(c.page_stride)};
  const uint32_t kb[4] = {64, static_cast<uint32_t>(rows), 1, 1};
  // an empty cache has no memory to describe: any valid address will do, nothing is read
  const void* k = c.capacity > 0 ? c.k : a.q;
  const void* v = c.capacity > 0 ? c.v : a.q;
  if (!make_tmap_bf16_nd(&m->k, k, 4, kd, ks, kb) || !make_tmap_bf16_nd(&m->v, v, 4, kd, ks, kb)) return false;
  m->kn = m->k;
  m->vn = m->v;
  if (a.k_new == nullptr) return true;
  const uint64_t nd[4] = {D, static_cast<uint64_t>(a.T), static_cast<uint64_t>(c.heads), static_cast<uint64_t>(a.B)};
  const uint64_t ns[3] = {static_cast<uint64_t>(a.new_t), static_cast<uint64_t>(a.new_h), static_cast<uint64_t>(a.new_b)};
  const uint32_t nb[4] = {64, kTile, 1, 1};
  return make_tmap_bf16_nd(&m->kn, a.k_new, 4, nd, ns, nb) && make_tmap_bf16_nd(&m->vn, a.v_new, 4, nd, ns, nb);
}

}  // namespace
}  // namespace dflash2
