// attn_common.cuh -- what the attention and score kernels share: equal runs over
// ragged sequences, waits that give up together, the ring's landing barriers,
// TMA loads of pages, and packed fp32 arithmetic.
#pragma once

#include "attn.h"
#include "tcgen05.cuh"

namespace dflash2 {

constexpr int kTile = 128;              // rows of a query tile, keys of a unit

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// two independent fp32 operations per instruction
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Lane 0's value, which the compiler then knows to be the whole warp's.
template <class T>
__device__ __forceinline__ T uniform(T x) {
  return __shfl_sync(0xFFFFFFFFu, x, 0);
}

// Where a run starts: unit `rel` of sequence b, whose items have n units each, and
// how many units the run has.
struct RunStart {
  int32_t rel, units, b, n;
};

// Cuts the units of B sequences, per_seq items of units(b) each (fewer than 2^31 in
// all), into runs of equal length and finds run `run`.  Every warp does this for
// itself, so that no block-wide step stands between the lengths and the first copy;
// it is kept short, since a small call meets it with an empty instruction cache.
template <class Units>
__device__ __forceinline__ RunStart find_run(const Units& units, int32_t B, int32_t per_seq, int32_t run, int32_t runs) {
  const int lane = threadIdx.x & 31;
  // the lane's sequence of the 32 at hand, and the units (of one item) up to and with it
  int32_t n = 0, incl = 0, before = 0, b0 = 0;
  const auto scan = [&]() {
    n = b0 + lane < B ? units(b0 + lane) : 0;
    incl = n;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, s);
      if (lane >= s) incl += o;
    }
    incl += before;
  };
#pragma unroll 1
  for (;; b0 += 32) {
    scan();
    if (b0 + 32 >= B) break;
    before = __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  const uint32_t total = uniform(__shfl_sync(0xFFFFFFFFu, incl, 31)) * static_cast<uint32_t>(per_seq);
  const uint32_t len = (total + runs - 1) / runs;
  const uint32_t u0 = min(run * len, total);
  RunStart r = {0, static_cast<int32_t>(min(len, total - u0)), 0, 0};
  if (r.units == 0) return r;
  if (B > 32) {                  // again from the first 32, up to those that hold u0
    before = 0;
#pragma unroll 1
    for (b0 = 0;; b0 += 32) {
      scan();
      before = __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (u0 < static_cast<uint32_t>(before * per_seq)) break;
    }
  }
  // the first lane whose sequence ends beyond u0
  const int at = __ffs(__ballot_sync(0xFFFFFFFFu, u0 < static_cast<uint32_t>(incl * per_seq))) - 1;
  r.b = b0 + at;
  r.n = __shfl_sync(0xFFFFFFFFu, n, at);
  r.rel = static_cast<int32_t>(u0) - (__shfl_sync(0xFFFFFFFFu, incl, at) - r.n) * per_seq;
  return r;
}

// Walks a run's stretches of items; each warp keeps its own (whole warps call it).
struct RunWalk {
  int32_t left;             // units of the run still to come
  int32_t b, item, s, n;    // the next stretch: from unit s of n of the sequence's item
  __device__ __forceinline__ void start(const RunStart& r) {
    left = r.units;
    if (left <= 0) return;
    b = r.b;
    n = r.n;
    item = static_cast<uint32_t>(r.rel) / static_cast<uint32_t>(n);
    s = r.rel - item * n;
  }
  // The item after this one (sequences without units are passed over).
  template <class Units>
  __device__ __forceinline__ void next_item(const Units& units, int32_t per_seq) {
    s = 0;
    if (++item < per_seq) return;
    item = 0;
    do {
      n = uniform(units(++b));
    } while (n == 0);
  }
};

// A bounded wait that also gives up when another role of the CTA has; once one
// has given up (*live = false) later waits return at once.
__device__ __forceinline__ void wait_live(uint64_t* bar, uint32_t parity, bool* live, volatile int* abort_flag,
                                          uint32_t* err) {
  if (!*live) return;
  uint64_t start = 0;
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 255u) == 0) {   // rarely: reading the timer takes longer than most of these waits
      if (*abort_flag) {
        *live = false;
        return;
      }
      const uint64_t now = global_timer_ns();
      if (start == 0) start = now;
      if (now - start > kWaitLimitNs) {
        raise_error(err, DFLASH2_DEVERR_TIMEOUT);
        *abort_flag = 1;
        *live = false;
        return;
      }
    }
  }
}

// A place in the sequence of tiles that go through a ring of S slots, and the
// barrier on which that tile lands.  A parity wait can only tell a phase from the
// one before it, and the pipelines do not look at every tile when they share a row
// tile.  So a slot's uses alternate between two barriers: when a pipeline asks for a
// slot's use k the producer has issued use k - 1 (it issues in order, and the
// pipeline has seen a later tile or the item's queries), for which use k - 2 had
// landed and been used, and use k cannot be passed by without this pipeline.
template <int S>
struct RingPos {
  uint32_t slot = 0, use = 0;
  __device__ __forceinline__ void advance(uint32_t n) {   // n < S
    slot += n;
    if (slot >= S) {
      slot -= S;
      ++use;
    }
  }
  __device__ __forceinline__ void advance_far(uint32_t n) {
    slot += n;
    use += slot / S;
    slot %= S;
  }
  __device__ __forceinline__ uint64_t* full(uint64_t* bars) const { return &bars[2 * slot + (use & 1)]; }
  __device__ __forceinline__ uint32_t parity() const { return use >> 1 & 1; }
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, int v,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_addr(bar))
      : "memory");
}

// The pages of consecutive tiles of one sequence, for a whole warp: 32 entries of
// its row of the block table a window, a lane each, and the next window's loads in
// flight while this one's are used (one by one they would cost a memory latency
// per tile).
struct PageFeed {
  const int32_t* row;       // the sequence's row; nullptr without a table
  int32_t base, last;       // the window's first entry; the last entry that may be read
  int32_t cur, next;        // entries base + lane and base + 32 + lane
  __device__ __forceinline__ int32_t fetch(int32_t i) const { return i <= last ? row[i] : 0; }
  // Tiles from `tile` on of sequence b, which holds len positions.
  __device__ __forceinline__ void start(const KvView& c, int64_t b, int32_t tile, int32_t len, int lane) {
    row = c.table == nullptr || len <= 0 ? nullptr : c.table + b * c.table_ld;
    if (row == nullptr) return;
    base = (tile * kTile) >> c.page_shift;
    last = (len - 1) >> c.page_shift;
    cur = fetch(base + lane);
    next = fetch(base + 32 + lane);
  }
  // The page of position j of the tile that starts at position `first` (a tile's
  // pages lie in one window: windows start at a tile, and a tile's pages, a power
  // of two of at most 8, or a page's tiles divide it).  Whole warp; ids outside the
  // cache are clamped and, where `used`, flagged.
  __device__ __forceinline__ int32_t page(const KvView& c, int32_t first, int32_t j, bool used, int lane, uint32_t* err) {
    if ((first >> c.page_shift) >= base + 32) {
      base += 32;
      cur = next;
      next = fetch(base + 32 + lane);
    }
    const int32_t p = __shfl_sync(0xFFFFFFFFu, cur, ((j >> c.page_shift) - base) & 31);
    if (static_cast<uint32_t>(p) < static_cast<uint32_t>(c.num_pages)) return p;
    if (used) raise_error(err, DFLASH2_DEVERR_BAD_PAGE);
    return p < 0 ? 0 : c.num_pages - 1;
  }
};

// A named barrier whose threads learn whether any of them brought `x`.
__device__ __forceinline__ bool named_bar_or(int id, int count, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %3, 0;\n\t"
      "bar.red.or.pred p, %1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(x))
      : "memory");
  return any != 0;
}

// Products are issued by whole warps of which one elected lane acts: the code
// around them stays warp-uniform, so operands are computed in uniform registers,
// and a product costs a few instructions instead of the tens that one lane alone
// takes (a batch of 8 + 4 products beside busy softmax warps: 876 against 1160
// cycles).
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p;
}

// The words of a shared-memory matrix descriptor with the 128-byte swizzle: the
// address and leading offset change, the rest (stride offset 1024, version 1,
// swizzle mode 2) does not.  A K-major operand's leading offset is not used (1); an
// MN-major one's is the distance between its 64-element column blocks.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t leading = 16) {
  return ((saddr & 0x3FFFFu) >> 4) | ((leading >> 4) << 16);
}

// D[tmem] (+)= A[smem] * B[smem]^T and D[tmem] (+)= A[tmem] * B[smem], one K = 16
// step, by the lane whose `lead` is set.  A in TMEM is 128 rows of 16 bf16 (8 columns).
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate,
                                        uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 x, {%1, %3};\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate,
                                        uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(lead)
      : "memory");
}

// Keeps uses of loaded values after the wait that precedes this in the program.
__device__ __forceinline__ void pin(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                 "+f"(v[i + 6]), "+f"(v[i + 7]));
}

}  // namespace dflash2
