// Attention of drafted rows over a cache of 8-bit entries: spec_verify_attend.
//
//   out[r, h] = sum_p softmax_p(scale q[r, h] . K[p]) V[p],  p over the committed positions and the row's path
//
// Keys go from memory to the tensor cores as they are, in 8 bits: a query of eight
// significant bits is the exact sum of two e4m3 numbers (times a power of two for its
// row; an entry below 2^-11 of the row's largest is off by 2^-17.8 of it at most), so
// S = K (Qhi + Qlo)^T is two products at twice the rate of bf16's.  O = V^T P is a product
// of fp16 numbers: values become that exactly, and weights are rounded to it.
//
// A key head's query rows (all rows of the step times the query heads of its group) are
// the columns: up to kN of them make a block, and one or two blocks a unit.  Positions are rows, 128 to a tile: thread
// t of a warpgroup has position t of every column, so that a position's scale and
// visibility are the thread's own.
//
// A weight times its value's scale stands against a reference of its column, under which
// the largest such product of some tile was 2^6.  It is taken anew where a tile has one
// that is above 2^15, and at every 16th tile if that tile's are all below 2.  Else a tile
// needs no reduction: sums of weights stay with the threads until a segment ends, and the
// products' sums in tensor memory.
//
// Weights in fp16 have eleven bits down to 2^-14, 2^-20 of that tile's largest, and are off
// by 2^-25 at most below: eight bits down to 2^-23 of the largest, 16 below its logit.  That
// range is needed: a few positions may tower above all others, as a model's first tokens
// do, with values near zero, and then the others are the result.  Two e4m3 numbers, hi + lo / 32,
// have eight bits over 2^15 only: a first position 11 above 4000 others took half of the
// others' weight.  (A reference for each tile, and two rounds for tiles with such
// positions, mended that too; on blocks whose scales differ it cost more: 64 chains 202 us, 167 so, and
// trees 149, 114.)  A group of softmax threads widens its tile's values itself, where two blocks of columns
// share a tile each group half of it.
//
// Work is cut evenly over the SMs, whatever the lengths: all tiles of all units (sequence, key
// head, columns) in a row, a CTA taking the n-th part of them.  A unit that
// is cut leaves its parts in the workspace, and a second kernel joins them.
//
// Measured (with the joining kernel; in brackets what the bytes take at the rate of a copy):
//   64 chains of five drafts after up to 8192 positions, 8 key heads of 128, 4 query heads
//     to each: 167 us (121); widening V takes 20 of them
//   the same with one row and 4096 positions each: 83.6 us (60.2)
//   2 chains of four after 131071, 8 key heads of 64, 5 query heads to each: 95.0 us (40.1)
//   32 trees of up to 21 nodes after up to 4000, 4 key heads of 128, 8 query heads to each:
//     114 us (16.0); 176 columns are three units of 64
//   one row after 1000 positions: 16.6 us, two launches and a chain of waits
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "cache.cuh"
#include "entry.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

constexpr int kTile = 128;  // positions
constexpr int kGroupThreads = 256;  // of a tile's softmax: a thread has one position of half of the columns
constexpr int kAttendThreads = 128 + 2 * kGroupThreads;
constexpr float kMost = 15.f;  // log2 of the largest weight over the reference; fp16 ends at 2^16
constexpr float kNew = 6.f;    // log2 of the largest one under a new reference
constexpr float kLow = 1.f;    // log2 of what a tile's largest may have fallen to where the reference stays
constexpr int kRefresh = 16;   // tiles of a group after which that is looked at
constexpr float kDeep = 60.f;  // log2 of how far a reference may fall below the highest: what is below adds nothing

// where a tile lies among all
struct Start {
  int64_t total;
  int b;
  int64_t off;  // in sequence b's work
};

struct AttendParams {
  CacheView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t q_row, q_head, out_row, out_head;
  int group;
  float scale;  // times log2(e)
  const int32_t *context, *node_start, *parent;
  int B, total, max_nodes;
  int boxes, box_tokens;  // boxes of a tile
  int page_scales;        // scales of a page
  unsigned in_page;       // a mask of positions in a page
  int grid;      // CTAs that share the tiles
  Start* cuts;   // where a CTA's first tile lies: for the second kernel
  float* parts;
};

struct Maps {
  CUtensorMap k, v;
};

// ---- the plan: units and tiles in a row

struct Sequence {
  int64_t context, end;
  int start, nodes, cols, pairs, tiles;
  bool lost;  // positions without a place in the table
  int64_t units, work;
};

template <int kColumns>  // of a unit
__device__ __forceinline__ Sequence sequence_of(const AttendParams& P, int b) {
  Sequence s = {};
  s.context = P.context[b];
  const int start = P.node_start[b], stop = P.node_start[b + 1];
  if (s.context < 0 || start < 0 || stop < start || stop > P.total || stop - start > P.max_nodes) return s;
  s.start = start, s.nodes = stop - start;
  s.end = s.context + 1 + s.nodes;
  s.lost = s.end > static_cast<int64_t>(P.c.table_cols) << P.c.page_log;
  s.tiles = s.lost ? 1 : static_cast<int>((s.end + kTile - 1) / kTile);
  s.cols = (s.nodes + 1) * P.group;
  s.pairs = (s.cols + kColumns - 1) / kColumns;
  s.units = static_cast<int64_t>(P.c.heads) * s.pairs;
  s.work = s.units * s.tiles;
  return s;
}

// the first tile of the i-th of n parts of all tiles
__device__ __forceinline__ int64_t cut(int64_t total, int i, int n) {
  if (total < 1 << 22) return static_cast<unsigned>(total) * static_cast<unsigned>(i) / static_cast<unsigned>(n);  // (n below 2^10)
  const int64_t each = total / n;
  return each * i + static_cast<unsigned>(total - each * n) * static_cast<unsigned>(i) / static_cast<unsigned>(n);
}

// Where tile `at(total)` of all lies; every thread of the CTA calls it.
template <int kColumns, typename F>
__device__ __forceinline__ void find_tile(const AttendParams& P, F&& at, Start* s, int64_t* warp_sums) {
  const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (P.B + threads - 1) / threads;
  const int lo = min(P.B, static_cast<int>(threadIdx.x) * per), hi = min(P.B, lo + per);
  int64_t mine = 0;
  for (int b = lo; b < hi; ++b) mine += sequence_of<kColumns>(P, b).work;
  int64_t sum = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(~0u, sum, o);
    if (lane >= o) sum += u;
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  int64_t base = sum - mine, total = 0;
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) base += warp_sums[w];
    total += warp_sums[w];
  }
  const int64_t tile = at(total);
  if (threadIdx.x == 0) s->total = total, s->b = P.B, s->off = 0;
  __syncthreads();
  if (tile >= base && tile < base + mine) {
    for (int b = lo; b < hi; ++b) {
      const int64_t w = sequence_of<kColumns>(P, b).work;
      if (tile < base + w) {
        s->b = b, s->off = tile - base;
        break;
      }
      base += w;
    }
  }
  __syncthreads();
}

// short where it can be
__device__ __forceinline__ int64_t divide(int64_t a, int b) {
  return a < INT32_MAX ? static_cast<int64_t>(static_cast<unsigned>(a) / static_cast<unsigned>(b)) : a / b;
}

// A run of tiles of one unit.  (Positions are below 2^31 + SV_MAX_NODES.)
struct Segment {
  int b, h, c0, t0, t1;  // c0: the first column; t1 = 0: there are no more
  int start, nodes, cols;
  unsigned root, end;    // the root's position, and behind the last one
  bool two, lost;        // two blocks of columns; positions without a place in the table
  bool front, whole;     // from the unit's first tile on; all of the unit's tiles
};

template <int kN, int kBlocks>
struct Walk {
  const AttendParams& P;
  int64_t pos, hi, off;
  int b;
  Sequence s;
  bool loaded = false;

  __device__ __forceinline__ Walk(const AttendParams& P, const Start& at, int64_t lo, int64_t hi)
      : P(P), pos(lo), hi(hi), off(at.off), b(at.b) {}

  __device__ __forceinline__ Segment next() {
    Segment g = {};
    if (pos >= hi) return g;
    while (!loaded || off >= s.work) {
      if (loaded) ++b, off = 0;
      if (b >= P.B) return g;
      s = sequence_of<kN * kBlocks>(P, b);
      loaded = true;
    }
    const int64_t unit = divide(off, s.tiles);
    g.b = b;
    g.h = static_cast<int>(divide(unit, s.pairs));
    g.c0 = static_cast<int>(unit - static_cast<int64_t>(g.h) * s.pairs) * kN * kBlocks;
    g.t0 = static_cast<int>(off - unit * s.tiles);
    const int64_t left = hi - pos, here = s.tiles - g.t0, n = left < here ? left : here;
    g.t1 = g.t0 + static_cast<int>(n);
    g.start = s.start, g.nodes = s.nodes, g.cols = s.cols;
    g.root = static_cast<unsigned>(s.context), g.end = s.lost ? 0u : static_cast<unsigned>(s.end);
    g.two = kBlocks == 2 && s.cols - g.c0 > kN;
    g.lost = s.lost;
    g.front = g.t0 == 0;
    g.whole = g.t0 == 0 && g.t1 == s.tiles;
    pos += n, off += n;
    return g;
  }
};

// ---- tensor core and tensor memory

__device__ __forceinline__ bool elect_one() {
  unsigned e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ void tma_load(const CUtensorMap* map, uint32_t dst, uint64_t* bar, int token, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(smem_addr(bar)), "r"(0), "r"(token), "r"(head), "r"(page)
      : "memory");
}

__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, unsigned idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned>(add))
      : "memory");
}

__device__ __forceinline__ void tc_mma_half(uint32_t d, uint64_t a, uint64_t b, unsigned idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned>(add))
      : "memory");
}

__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// kCols columns (a multiple of 4) of this warp's 32 lanes
template <int kCols>
__device__ __forceinline__ void tc_load(uint32_t addr, float (&f)[kCols]) {
  constexpr int k16 = kCols / 16 * 16, k8 = k16 + (kCols - k16) / 8 * 8;
#pragma unroll
  for (int c = 0; c < k16; c += 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=f"(f[c]), "=f"(f[c + 1]), "=f"(f[c + 2]), "=f"(f[c + 3]), "=f"(f[c + 4]), "=f"(f[c + 5]), "=f"(f[c + 6]),
          "=f"(f[c + 7]), "=f"(f[c + 8]), "=f"(f[c + 9]), "=f"(f[c + 10]), "=f"(f[c + 11]), "=f"(f[c + 12]),
          "=f"(f[c + 13]), "=f"(f[c + 14]), "=f"(f[c + 15])
        : "r"(addr + c)
        : "memory");
#pragma unroll
  for (int c = k16; c < k8; c += 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(f[c]), "=f"(f[c + 1]), "=f"(f[c + 2]), "=f"(f[c + 3]), "=f"(f[c + 4]), "=f"(f[c + 5]), "=f"(f[c + 6]),
                   "=f"(f[c + 7])
                 : "r"(addr + c)
                 : "memory");
#pragma unroll
  for (int c = k8; c < kCols; c += 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(f[c]), "=f"(f[c + 1]), "=f"(f[c + 2]), "=f"(f[c + 3])
                 : "r"(addr + c)
                 : "memory");
  // the registers pass through the wait, so that nothing reads them in front of it
#pragma unroll
  for (int c = 0; c < kCols; c += 4)
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(f[c]), "+f"(f[c + 1]), "+f"(f[c + 2]), "+f"(f[c + 3]) : : "memory");
}

// four columns back
__device__ __forceinline__ void tc_store(uint32_t addr, const float (&f)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};" ::"f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "r"(addr)
               : "memory");
}

// Two floats in a 64-bit register: one instruction for both, each rounded by itself.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void both(Two t, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(t)); }
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Operands in shared memory (all of their offsets in units of 16 bytes).
// Tiles of K: rows of kD bytes, 128- or 64-byte swizzle, groups of 8 rows behind one another.  Q's rows lie like K's.
template <int kD>
__device__ __forceinline__ uint64_t rows_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (1ull << 16) | (static_cast<uint64_t>(kD * 8 / 16) << 32) | (1ull << 46) |
         (kD == 128 ? 2ull << 61 : 4ull << 61);
}
// V in fp16: runs of 64 entries, 128 bytes for each position, 128-byte swizzle, a run's 128 positions behind one another.  The
// positions are the inner dimension, so that it lies transposed.  Eight positions on: 1024 bytes; a run on: 16384.
__device__ __forceinline__ uint64_t values_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (1024ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Weights: runs of 8 columns, 16 bytes for each position, a run's 128 positions behind one another; no swizzle; transposed like
// V.  Eight positions on: 128 bytes; a run on: 2048.
__device__ __forceinline__ uint64_t weights_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (8ull << 16) | (128ull << 32) | (1ull << 46);
}

// mbar_wait in fewer instructions: the loops of all warps together should stay in the instruction caches.
__device__ __forceinline__ void wait_for(uint64_t* bar, unsigned parity, volatile int* dead) {
  if (mbar_try(bar, parity)) return;
  unsigned since, t;
  asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(since));
#pragma unroll 1
  while (!mbar_try(bar, parity)) {
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
    if (t - since > 2000000000u || *dead) {
      *dead = 1;
      return;
    }
  }
}

__device__ __forceinline__ uint4 shared_load(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void shared_store(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ float power(float x) {  // 2^x; results below 2^-126 become 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// two weights to fp16, to nearest
__device__ __forceinline__ uint32_t half2_of(Two w) {
  float a, b;
  both(w, a, b);
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
  return h;
}

// two e4m3 entries as fp16 (exact)
__device__ __forceinline__ uint32_t half2_of(uint16_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return h;
}

// Each column's largest, or sum, over a warp's lanes: halves of the columns change hands until a lane has its own.  Of kCols
// columns lane i gets column i / (32 / kCols).
template <int kCols, bool kSum>
__device__ __forceinline__ float over_lanes(const float* f) {
  const int lane = threadIdx.x & 31;
  float v[kCols / 2];
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) {
    const float send = lane & 16 ? f[i] : f[i + kCols / 2], keep = lane & 16 ? f[i + kCols / 2] : f[i];
    const float got = __shfl_xor_sync(~0u, send, 16);
    v[i] = kSum ? keep + got : fmaxf(keep, got);
  }
#pragma unroll
  for (int o = 8, n = kCols / 4; o; o >>= 1, n /= 2) {
    if (n > 0) {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = lane & o ? v[i] : v[i + n], keep = lane & o ? v[i + n] : v[i];
        const float got = __shfl_xor_sync(~0u, send, o);
        v[i] = kSum ? keep + got : fmaxf(keep, got);
      }
    } else {
      const float got = __shfl_xor_sync(~0u, v[0], o);
      v[0] = kSum ? v[0] + got : fmaxf(v[0], got);
    }
  }
  return v[0];
}

// Tiles of K and of V have rings of their own: K's is free after the first product, V's where it is widened.
template <int kN, int kBlocks, int kD>
struct AttendShared {
  static constexpr int kK = kD == 64 ? 10 : kBlocks == 2 ? 3 : 4, kV = kD == 64 ? 8 : 4;
  // Waits tell a phase only from the one next to it.  The first warp, kK tiles ahead of a product of which up to four tiles
  // may be in use, looks at V's stages: two rounds of them are more than that.  And a group's next tile in a stage is its own.
  static_assert(2 * kV >= kK + 4 && kV % 2 == 0);
  static constexpr int kWords = (kBlocks * kN + 31) / 32;  // of a unit's columns
  // of a special tile's positions: the columns that see it; whether what they see is no number
  uint32_t seen[kV][kTile][kWords];
  uint32_t none[kV][kTile / 32];
  float most[2][4][kN];  // a warp's largest logits, and at last its sums
  // (read in fours)
  alignas(16) float zero[kN];  // references of a segment's first items
  alignas(16) float ref[2][kN];   // references, negative
  alignas(16) float step[2][kN];  // how far a reference moved
  alignas(16) float keep[2][kN];  // what the sums so far are worth against the new one
  float m[2][kN];
  uint32_t moved[2], unset[2];  // of a group: columns whose sums have to be multiplied, that have no reference yet
  // at a segment's end: factors of the groups' sums (of the blocks' in a segment of two) and of the result
  float worth[2][kN], whole[2][kN], last[2][kN];
  alignas(16) float row[kBlocks][kN];  // of a query row: its power of two, the softmax's scale
  int64_t out[kBlocks][kN];            // where its result goes
  float anchors[2][4], second_anchor;  // of a group's warps; of the second group
  uint32_t path[SV_MAX_NODES][kWords];
  int parent[SV_MAX_NODES];
  Segment segment[4];  // the first warp walks ahead
  uint64_t g_full[4], g_free[4];
  uint64_t k_full[kK], k_empty[kK], v_full[kV], v_empty[kV], ready[kV];
  uint64_t s_full[2], s_free[2], wide_full[2], p_full[2], o_full[2], q_full, o_read;
  int64_t warp_sums[kAttendThreads / 32];
  Start start;
  uint32_t tmem;
  volatile int dead;
};

template <int kN, int kBlocks, int kD>
struct Sizes {
  using Shared = AttendShared<kN, kBlocks, kD>;
  static constexpr int kTileBytes = kTile * kD;
  static constexpr int kQ = kN * kD;  // one of the two numbers of a block's entries
  static constexpr int kWide = kTile * kD * 2, kWeights = kTile * kN * 2;  // fp16
  static constexpr int kColumns = kBlocks * kN;              // of a unit
  static constexpr int kSmem = static_cast<int>(sizeof(Shared)) + 1024 + (Shared::kK + Shared::kV) * kTileBytes +
                               2 * kBlocks * kQ + 2 * kWide + 2 * kWeights;
  static constexpr int kPart = kColumns * (kD + 2);  // floats of a part in the workspace
  static_assert(kSmem <= 227 * 1024);
};

// a stage of a ring, and how often it has been passed modulo 2
template <int kStages>
struct Ring {
  int at = 0;
  unsigned phase = 0;
  __device__ __forceinline__ void step() {
    if (++at == kStages) at = 0, phase ^= 1;
  }
};

// The pages of a segment's tiles, a lane's of its box, looked up a tile ahead.
struct Pages {
  const AttendParams& P;
  const int32_t* table;
  unsigned end, box;  // box: the first position of this lane's box in a tile, or far behind
  int t1, ahead;
  __device__ __forceinline__ Pages(const AttendParams& P, const Segment& g, int lane)
      : P(P), table(P.c.table + g.b * P.c.table_stride), end(g.end), t1(g.t1) {
    box = lane < P.boxes ? lane * P.box_tokens : ~0u;
    ahead = look(g.t0);
  }
  __device__ __forceinline__ int look(int t) const {
    const unsigned pos = static_cast<unsigned>(t) * kTile + box;
    return box != ~0u && t < t1 && pos < end ? table[pos >> P.c.page_log] : -1;
  }
  // of tile t, the one after the last asked for; behind the last page (zeros) where there is none
  __device__ __forceinline__ int next(int t) {
    const int page = ahead;
    ahead = look(t + 1);
    return static_cast<unsigned>(page) < static_cast<unsigned>(P.c.pages) ? page : max(1, P.c.pages);
  }
  __device__ __forceinline__ int token(int t) const {
    return static_cast<int>((static_cast<unsigned>(t) * kTile + box) & P.in_page);
  }
};

__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 256;" ::"r"(1 + group) : "memory"); }
// whether any thread of a group says so
__device__ __forceinline__ bool group_any(int group, bool mine) {
  unsigned any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 256, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"(static_cast<unsigned>(mine)), "r"(1 + group)
      : "memory");
  return any != 0;
}
// the same of both groups
__device__ __forceinline__ bool groups_any(bool mine) {
  unsigned any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 3, 512, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"(static_cast<unsigned>(mine))
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void groups_sync() { asm volatile("bar.sync 3, 512;" ::: "memory"); }

__device__ __forceinline__ bool holds_nan(uint4 e) {
  // 0x7f in the low seven bits of a byte
  const auto hit = [](uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
  return (hit(e.x) | hit(e.y) | hit(e.z) | hit(e.w)) != 0;
}

// kC: columns of a thread, half of those of a block that are used.
template <int kN, int kBlocks, int kC, int kD>
__global__ void __launch_bounds__(kAttendThreads, 1) attend_kernel(const __grid_constant__ AttendParams P,
                                                                   const __grid_constant__ Maps maps) {
  using Z = Sizes<kN, kBlocks, kD>;
  using Shared = AttendShared<kN, kBlocks, kD>;
  constexpr int kWords = Shared::kWords;
  constexpr unsigned kK = Shared::kK, kV = Shared::kV;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  uint8_t* const base = raw + sizeof(Shared) + ((1024 - (smem_addr(raw + sizeof(Shared)) & 1023)) & 1023);
  uint8_t* const tiles_k = base;
  uint8_t* const tiles_v = tiles_k + kK * Z::kTileBytes;
  uint8_t* const queries = tiles_v + kV * Z::kTileBytes;            // [hi, lo][block]
  uint8_t* const wides = queries + 2 * kBlocks * Z::kQ;         // of a group's tile; with two blocks of every other tile
  uint8_t* const weights = wides + 2 * Z::kWide;                // [group]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (unsigned i = 0; i < kK; ++i) mbar_init(&s.k_full[i], 1), mbar_init(&s.k_empty[i], 1);
    for (unsigned i = 0; i < kV; ++i) mbar_init(&s.v_full[i], 1), mbar_init(&s.v_empty[i], 16), mbar_init(&s.ready[i], 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(&s.s_full[i], 1), mbar_init(&s.s_free[i], 8), mbar_init(&s.wide_full[i], 16), mbar_init(&s.p_full[i], 8),
          mbar_init(&s.o_full[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&s.g_full[i], 1), mbar_init(&s.g_free[i], 19);
    mbar_init(&s.q_full, 16), mbar_init(&s.o_read, 16);
    for (int c = 0; c < kN; ++c) s.zero[c] = 0.f;
    s.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // columns that are not used have weights too
  for (int i = threadIdx.x; i < 2 * Z::kWeights / 16; i += kAttendThreads)
    reinterpret_cast<uint4*>(weights)[i] = make_uint4(0, 0, 0, 0);
  async_fence();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s.tmem)), "n"(4 * kN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  wait_for_stream();
  int64_t lo = 0;
  find_tile<Z::kColumns>(P, [&](int64_t total) { return cut(total, blockIdx.x, P.grid); }, &s.start, s.warp_sums);
  tc_before();
  __syncthreads();
  tc_after();
  const Start start = s.start;
  if (threadIdx.x == 0) P.cuts[blockIdx.x] = start;
  lo = cut(start.total, blockIdx.x, P.grid);
  const int64_t hi = cut(start.total, blockIdx.x + 1, P.grid);
  const uint32_t tmem = s.tmem;  // S of the two groups (kN columns each), then O
  // The next segment of a warp that takes them from the first; false behind the last, and where a wait gave up.
  auto next_segment = [&](unsigned n, Segment& g) {
    wait_for(&s.g_full[n & 3], n >> 2 & 1, &s.dead);
    g = s.segment[n & 3];
    return g.t1 > 0 && !s.dead;
  };
  auto free_segment = [&](unsigned n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.g_free[n & 3]);
  };
  // A tile of K or of V by TMA, a lane for each of its boxes.  (One warp for K, one for V: with one for both 1500 cycles a tile,
  // more than anything else of it.)
  auto copy_tile = [&](Pages& pages, int t, const CUtensorMap* map, uint8_t* tiles, uint64_t* full, uint64_t* empty, int st,
                       unsigned phase, int h) {
    const int page = pages.next(t);
    wait_for(&empty[st], phase ^ 1, &s.dead);
    if (lane == 0) mbar_expect(&full[st], Z::kTileBytes);
    if (lane < P.boxes)
      tma_load(map, smem_addr(tiles) + st * Z::kTileBytes + lane * P.box_tokens * kD, &full[st], pages.token(t), h, page);
  };
  if (warp == 0) {
    // ---- segments; their tiles of K; the visibility of the positions of special tiles, those with drafted positions or with
    // the sequence's end
    Walk<kN, kBlocks> walk(P, start, lo, hi);
    Ring<kK> ring;
    Ring<kV> ring_v;
    for (unsigned n = 0;; ++n) {
      const Segment g = walk.next();
      if (n > 3) wait_for(&s.g_free[n & 3], (n >> 2) - 1 & 1, &s.dead);
      if (s.dead) break;
      if (lane == 0) {
        s.segment[n & 3] = g;
        mbar_arrive(&s.g_full[n & 3]);
      }
      __syncwarp();
      if (g.t1 == 0) break;
      Pages pages(P, g, lane);
      bool built = false, bad = false;
#pragma unroll 1
      for (int t = g.t0; t < g.t1; ++t, ring.step(), ring_v.step()) {
        copy_tile(pages, t, &maps.k, tiles_k, s.k_full, s.k_empty, ring.at, ring.phase, g.h);
        const unsigned p0 = static_cast<unsigned>(t) * kTile;
        const int st = ring_v.at;
        if (!(g.lost || p0 + kTile > g.root + 1)) continue;
        if (!built && !g.lost && P.parent) {
          // the columns whose path a node is on
          built = true;
          for (int i = lane; i < g.nodes; i += 32) {
            const int up = P.parent[g.start + i];
            bad |= up < -1 || up >= i;
            s.parent[i] = up;
#pragma unroll
            for (int w = 0; w < kWords; ++w) s.path[i][w] = 0;
          }
          bad = __any_sync(~0u, bad);
          __syncwarp();
          const int last = min(g.nodes, (g.c0 + Z::kColumns - 1) / P.group);
          for (int i = g.c0 / P.group + lane; !bad && i <= last; i += 32) {
            const int from = i * P.group - g.c0, to = from + P.group;
            for (int node = i - 1; node >= 0; node = s.parent[node])
#pragma unroll
              for (int w = 0; w < kWords; ++w) {
                const int a = max(0, from - w * 32), e = min(32, to - w * 32);
                if (e > a) atomicOr(&s.path[node][w], (e - a == 32 ? ~0u : ((1u << (e - a)) - 1u)) << a);
              }
          }
          __syncwarp();
        }
        // (a parity tells a phase only from the one next to it: not before the tile that was there has been used)
        wait_for(&s.v_empty[st], ring_v.phase ^ 1, &s.dead);
        wait_for(&s.v_full[st], ring_v.phase, &s.dead);
        {
          uint8_t* const v = tiles_v + st * Z::kTileBytes;
#pragma unroll 1
          for (int i = 0; i < kTile / 32; ++i) {
            const int at = lane + 32 * i;
            const unsigned pos = p0 + at;
            const int node = static_cast<int>(pos - g.root - 1);
            bool none = g.lost;
            uint32_t seen[kWords];
#pragma unroll
            for (int w = 0; w < kWords; ++w) seen[w] = ~0u;
            if (!g.lost && node >= 0) {
              // What a position holds that not every row sees goes through the product of every row: nothing but numbers
              // may stand there.  (Lanes begin at different places of their rows: at the same one all of them would meet
              // in four banks: 5 % of 256 contexts of 300 positions.)
              uint4* row = reinterpret_cast<uint4*>(v + at * kD);
              const bool behind = pos >= g.end;
              bool nan = false;
              if (!behind)
                for (int c = 0; c < kD / 16; ++c) nan |= holds_nan(row[(c + lane) % (kD / 16)]);
              if (nan || behind)
                for (int c = 0; c < kD / 16; ++c) row[(c + lane) % (kD / 16)] = make_uint4(0, 0, 0, 0);
              none = nan || bad;
              const bool lost = !behind && P.c.page_of(g.b, pos) < 0;  // every row of the sequence is
              if (behind) {
#pragma unroll
                for (int w = 0; w < kWords; ++w) seen[w] = 0;
              } else if (!bad && !lost && P.parent) {
#pragma unroll
                for (int w = 0; w < kWords; ++w) seen[w] = s.path[node][w];
              } else if (!bad && !lost) {
                const int from = (node + 1) * P.group - g.c0;  // the first column that sees it
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                  const int a = from - w * 32;
                  seen[w] = a <= 0 ? ~0u : a >= 32 ? 0u : ~0u << a;
                }
              }
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w) s.seen[st][at][w] = seen[w];
            const uint32_t bits = __ballot_sync(~0u, none);
            if (lane == 0) s.none[st][i] = bits;
          }
          async_fence();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.ready[st]);
      }
    }
  } else if (warp == 1) {
    // ---- products with K; of two blocks at once, whose sums lie side by side
    constexpr unsigned kShape = (1u << 4) | (8u << 24);
    unsigned count = 0, asked = 0, begun = 0;  // asked: a bit for each group, how often modulo 2
    const uint64_t q = rows_desc<kD>(smem_addr(queries));
    Segment g;
    for (unsigned segment = 0; next_segment(segment, g); free_segment(segment++)) {
      wait_for(&s.q_full, segment & 1, &s.dead);
      const unsigned shape = kShape | static_cast<unsigned>((g.two ? 2 * kN : kN) / 8) << 17;
      for (int i = 0; i < g.t1 - g.t0; ++i) {
        const unsigned n = count + i, st = n % kK;
        wait_for(&s.k_full[st], n / kK & 1, &s.dead);
        const unsigned groups = g.two ? 3u : 1u << (i & 1);
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (groups & begun & 1u << w) wait_for(&s.s_free[w], ~asked >> w & 1u, &s.dead);
        asked ^= groups, begun |= groups;
        tc_after();
        const uint64_t k = rows_desc<kD>(smem_addr(tiles_k + st * Z::kTileBytes));
        const uint32_t to = tmem + (groups == 2u ? kN : 0);
        if (elect_one()) {
#pragma unroll
          for (int piece = 0; piece < 2; ++piece)
#pragma unroll
            for (int d = 0; d < kD / 32; ++d)
              tc_mma(to, k + 2 * d, q + piece * (kBlocks * Z::kQ / 16) + 2 * d, shape, piece + d > 0);
          if (groups & 1u) tc_commit(&s.s_full[0]);
          if (groups & 2u) tc_commit(&s.s_full[1]);
          tc_commit(&s.k_empty[st]);
        }
        __syncwarp();
      }
      count += g.t1 - g.t0;
    }
  } else if (warp == 2) {
    // ---- products with V
    constexpr unsigned kShape =
        (1u << 4) | (1u << 15) | (1u << 16) | (static_cast<unsigned>(kN / 8) << 17) | (static_cast<unsigned>(kD / 16) << 24);
    unsigned count = 0, done = 0, used = 0;  // done, used: a bit for each group and each tile of wide values, how often modulo 2
    Segment g;
    for (unsigned segment = 0; next_segment(segment, g); free_segment(segment++)) {
      const int items = (g.t1 - g.t0) << (g.two ? 1 : 0);
      for (int i = 0; i < items; ++i) {
        const int w = i & 1, b = kBlocks == 2 && g.two ? (count + i / 2) & 1 : w;
        if (kBlocks == 2 && g.two && w == 0) wait_for(&s.wide_full[b], used >> b & 1u, &s.dead), used ^= 1u << b;
        wait_for(&s.p_full[w], done >> w & 1u, &s.dead);
        done ^= 1u << w;
        tc_after();
        const uint64_t v = values_desc(smem_addr(wides + b * Z::kWide));
        const uint64_t p = weights_desc(smem_addr(weights + w * Z::kWeights));
        if (elect_one()) {
#pragma unroll
          for (int t = 0; t < kTile / 16; ++t)
            tc_mma_half(tmem + (2 + w) * kN, v + t * (16 * 128 / 16), p + t * 16, kShape,
                        i > 1 || t > 0);  // a group's first item of a segment begins its sums
          tc_commit(&s.o_full[w]);
        }
        __syncwarp();
      }
      count += g.t1 - g.t0;
    }
  } else if (warp == 3) {
    // ---- tiles of V
    Segment g;
    Ring<kV> ring;
    for (unsigned segment = 0; next_segment(segment, g); free_segment(segment++)) {
      Pages pages(P, g, lane);
      for (int t = g.t0; t < g.t1; ++t, ring.step())
        copy_tile(pages, t, &maps.v, tiles_v, s.v_full, s.v_empty, ring.at, ring.phase, g.h);
    }
  } else {
    // ---- softmax
    const int me = (warp - 4) / 8, half = (warp - 4) / 4 & 1, quad = warp & 3;
    const int t = threadIdx.x - 128 - me * kGroupThreads, position = t & (kTile - 1);
    constexpr int kPad = kC == 12 ? 16 : kC, kUsed = 2 * kC;
    const uint32_t lanes = static_cast<uint32_t>(quad) << 21;  // 32 lanes of tensor memory each
    const uint32_t tmem_s = tmem + lanes + me * kN + half * kC, tmem_o = tmem + lanes + (2 + me) * kN + half * kC;
    unsigned count = 0, items = 0, ready = 0;  // ready: a bit for each stage, its barrier's parity
    uint8_t* const mine = weights + me * Z::kWeights;
    // A query row is read by kLanes lanes, eight entries each, kRows rows a warp at once.  The rows of a segment and the page of
    // its first tile are on their way while the segment in front is finished.
    constexpr int kLanes = kD / 8, kRows = 32 / kLanes, kPasses = (Z::kColumns + 16 * kRows - 1) / (16 * kRows);
    uint4 ahead[kPasses] = {};
    int page_ahead = -1;
    auto look_ahead = [&](unsigned n) {
      wait_for(&s.g_full[n & 3], n >> 2 & 1, &s.dead);
      page_ahead = -1;
      if (s.dead) return;
      const Segment& g = s.segment[n & 3];
      const unsigned pos = static_cast<unsigned>(g.t0 + (g.two ? 0 : me)) * kTile + position;
      page_ahead = pos < g.end && g.t0 + (g.two ? 0 : me) < g.t1 ? P.c.table[g.b * P.c.table_stride + (pos >> P.c.page_log)] : -1;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int col = g.c0 + ((warp - 4) + 16 * p) * kRows + lane / kLanes, i = col / P.group;
        ahead[p] = make_uint4(0, 0, 0, 0);
        if (g.t1 > 0 && col < g.cols)
          ahead[p] = *reinterpret_cast<const uint4*>(P.q + (static_cast<int64_t>(g.start) + g.b + i) * P.q_row +
                                                     (static_cast<int64_t>(g.h) * P.group + col - i * P.group) * P.q_head +
                                                     lane % kLanes * 8);
      }
    };
    look_ahead(0);
    for (unsigned segment = 0;; ++segment) {
      const Segment& g = s.segment[segment & 3];
      const int t0 = g.t0, t1 = g.t1;
      const bool two_blocks = kBlocks == 2 && g.two;
      // all of the warps that meet at barriers go on, or none
      if (groups_any(t1 == 0 || s.dead)) break;
      const int step = two_blocks ? 1 : 2, first_tile = t0 + (two_blocks ? 0 : me);
      // pages and scales of this thread's position, an item and two ahead
      const int32_t* const table = P.c.table + g.b * P.c.table_stride;
      const int of_head = g.h << (P.c.page_log - P.c.block_log);
      const unsigned end = g.end;
      const bool lost = g.lost;
      auto page_at = [&](int tile) {
        const unsigned pos = static_cast<unsigned>(tile) * kTile + position;
        return tile < t1 && pos < end ? table[pos >> P.c.page_log] : -1;
      };
      auto scales_at = [&](int tile, int page) {
        const unsigned pos = static_cast<unsigned>(tile) * kTile + position;
        float2 f = make_float2(lost || pos < end ? NAN : 0.f, 0.f);
        if (static_cast<unsigned>(page) < static_cast<unsigned>(P.c.pages)) {
          const int64_t at = static_cast<int64_t>(page) * P.page_scales + of_head + ((pos & P.in_page) >> P.c.block_log);
          f.x = P.c.scales[0][at], f.y = P.c.scales[1][at];
        }
        return f;
      };
      float2 scales_next = scales_at(first_tile, page_ahead);
      int page_next = page_at(first_tile + step);
      // the queries over a power of two for each row, as two e4m3 numbers an entry
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int r = ((warp - 4) + 16 * p) * kRows + lane / kLanes, col = g.c0 + r, block = r / kN, row = r % kN;
        if (r - lane / kLanes >= (two_blocks ? 2 : 1) * kN) break;
        const uint32_t w[4] = {ahead[p].x, ahead[p].y, ahead[p].z, ahead[p].w};
        float most = 0.f, q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          q[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
          most = fabsf(q[e]) < INFINITY ? fmaxf(most, fabsf(q[e])) : INFINITY;
        }
        for (int o = kLanes / 2; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
        const bool fine = most < INFINITY;
        const float unit = fine ? scale_for(most) : 1.f, inverse = 1.f / unit;
        uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float a = q[e] * inverse, b = q[e + 1] * inverse;
          const uint32_t h = e4m3x2(a, b);
          const float2 f = from_e4m3x2(h);
          hi[e / 4] |= h << (e % 4 * 8), lo[e / 4] |= e4m3x2(a - f.x, b - f.y) << (e % 4 * 8);
        }
        if (r < (two_blocks ? 2 : 1) * kN) {
          const int byte = lane % kLanes * 8, chunk = byte / 16;
          const int swizzled = kD == 128 ? chunk ^ (row & 7) : chunk ^ (row >> 1 & 3);
          uint8_t* const to = queries + block * Z::kQ + row * kD + swizzled * 16 + byte % 16;
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to + kBlocks * Z::kQ) = make_uint2(lo[0], lo[1]);
          if (lane % kLanes == 0) {
            const int i = col / P.group;
            s.row[block][row] = fine ? unit * P.scale : NAN;
            s.out[block][row] = (static_cast<int64_t>(g.start) + g.b + i) * P.out_row +
                                (static_cast<int64_t>(g.h) * P.group + col - i * P.group) * P.out_head;
          }
        }
      }
      // the anchor of the group's value scales: a power of two near the first tile's largest, 2^-110 at least
      float anchor = scales_next.y < INFINITY ? scales_next.y : 0.f;
      for (int o = 16; o; o >>= 1) anchor = fmaxf(anchor, __shfl_xor_sync(~0u, anchor, o));
      if (lane == 0) s.anchors[me][quad] = anchor;
      async_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_full);
      // the first tile with drafted positions or the sequence's end
      const int first_special = lost ? 0 : static_cast<int>(min((g.root + 1) / kTile, static_cast<unsigned>(t1)));
      wait_for(&s.q_full, segment & 1, &s.dead);
      anchor = fmaxf(fmaxf(s.anchors[me][0], s.anchors[me][1]), fmaxf(s.anchors[me][2], s.anchors[me][3]));
      anchor = __uint_as_float(__float_as_uint(fminf(fmaxf(anchor, 0x1p-110f), 0x1p100f)) & 0x7f800000u);
      const float per_anchor = 1.f / anchor;
      const float* const factors = s.row[two_blocks ? me : 0] + half * kC;
      Two l[kC / 2];
#pragma unroll
      for (int c = 0; c < kC / 2; ++c) l[c] = 0;
      float m = -INFINITY, top = -INFINITY;  // m: of column t, its reference
      bool unset = true;
      const unsigned begun = items;
      const int own = lane / (32 / kPad);  // the column of its half that reductions leave to this lane
      // each column's largest, or sum, over this warp's positions
      auto post = [&](const float (&v)[kC], auto sum) {
        float r;
        if constexpr (kPad == kC) {
          r = over_lanes<kC, sum.value>(v);
        } else {
          float w[kPad];
#pragma unroll
          for (int c = 0; c < kPad; ++c) w[c] = c < kC ? v[c < kC ? c : 0] : sum.value ? 0.f : -INFINITY;
          r = over_lanes<kPad, sum.value>(w);
        }
        if (own < kC) s.most[me][quad][half * kC + own] = r;
      };
      for (int tile = first_tile; tile < t1; tile += step) {
        const unsigned n = count + (tile - t0), st = n % kV;
        const float2 scales = scales_next;
        scales_next = scales_at(tile + step, page_next);
        page_next = page_at(tile + 2 * step);
        // V's scale over the anchor: rest * 2^e, rest in (1/2, 1], e -12 at least.  One that is no number, or too large for that:
        // the rows that see it become NaN by their logits, and a weight of 0 stays one.  (Looked at here, where it has come: 185 us
        // for 64 chains behind the load, 167 so.)
        float kf = scales.x, ratio = scales.y * per_anchor;
        if (!(fabsf(ratio) <= 0x1p120f)) kf = NAN, ratio = 0.f;
        const uint32_t u = __float_as_uint(ratio);
        const int e = max(-12, min(120, static_cast<int>(u >> 23 & 0xff) - 126 - ((u & 0x7fffffu) == 0)));
        const float inverse = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        uint32_t seen = ~0u;
        if (tile >= first_special) {
          wait_for(&s.ready[st], ready >> st & 1u, &s.dead);
          if (s.none[st][quad] >> lane & 1u) kf = NAN;
          const int col = (two_blocks ? me * kN : 0) + half * kC;
          seen = s.seen[st][position][col / 32] >> col % 32;
        }
        wait_for(&s.s_full[me], items & 1, &s.dead);
        tc_after();
        float x[kC];
        tc_load<kC>(tmem_s, x);
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.s_free[me]);
        {
          // x becomes the logit, log2 of V's scale added, over the reference
          const Two kf2 = two(kf, kf), shift = two(static_cast<float>(e), static_cast<float>(e));
          const float* const refs = (items == begun ? s.zero : s.ref[me]) + half * kC;
#pragma unroll
          for (int c = 0; c < kC; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(factors + c), r = *reinterpret_cast<const float4*>(refs + c);
            both(fma2(two(x[c], x[c + 1]), mul2(two(f.x, f.y), kf2), add2(shift, two(r.x, r.y))), x[c], x[c + 1]);
            both(fma2(two(x[c + 2], x[c + 3]), mul2(two(f.z, f.w), kf2), add2(shift, two(r.z, r.w))), x[c + 2], x[c + 3]);
          }
          if (tile >= first_special) {
#pragma unroll
            for (int c = 0; c < kC; ++c)
              if (!(seen >> c & 1u)) x[c] = -INFINITY;
          }
          float most = x[0];
#pragma unroll
          for (int c = 1; c < kC; ++c) most = fmaxf(most, x[c]);
          // with a weight that is too large in any thread, or for a new reference, the tile's largest are found
          if (group_any(me, most > kMost || unset || (items - begun) % kRefresh == 0)) {
            post(x, std::false_type());
            group_sync(me);
            if (t < kUsed) {
              const float zt = fmaxf(fmaxf(s.most[me][0][t], s.most[me][1][t]), fmaxf(s.most[me][2][t], s.most[me][3][t]));
              const bool first = m == -INFINITY;
              const float from = first ? 0.f : m;
              float to = from, keep = 1.f;
              if (zt != -INFINITY) {
                if (first || !(zt <= kMost && zt >= kLow)) to = from + (zt - kNew);
                if (!first) to = fmaxf(to, top - kDeep), keep = power(from - to);
                m = to, top = fmaxf(top, to);
              }
              s.ref[me][t] = -to, s.step[me][t] = from - to, s.keep[me][t] = keep;
              const unsigned lanes_here = kUsed < 32 ? (1u << (kUsed & 31)) - 1u : ~0u;
              const uint32_t moved = __ballot_sync(lanes_here, keep != 1.f), none = __ballot_sync(lanes_here, m == -INFINITY);
              if (lane == 0) s.moved[me] = moved, s.unset[me] = none;
            }
            group_sync(me);
            unset = s.unset[me] != 0;
            const float *const steps = s.step[me] + half * kC, *const keeps = s.keep[me] + half * kC;
#pragma unroll
            for (int c = 0; c < kC; c += 2) {
              const float2 d = *reinterpret_cast<const float2*>(steps + c), k = *reinterpret_cast<const float2*>(keeps + c);
              x[c] += d.x, x[c + 1] += d.y;
              l[c / 2] = mul2(l[c / 2], two(k.x, k.y));
            }
            if (s.moved[me] != 0 && items != begun) {
              wait_for(&s.o_full[me], (items - 1) & 1, &s.dead);
              tc_after();
#pragma unroll 1
              for (int c = 0; c < kC; c += 4) {
                float o[4];
                tc_load<4>(tmem_o + c, o);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] *= keeps[c + k];
                tc_store(tmem_o + c, o);
              }
              asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
              tc_before();
            }
          }
        }
        const Two inverse2 = two(inverse, inverse), rest = two(ratio * inverse, ratio * inverse);
        // the weights in front and their values have been read; the sums of the segment in front too
        if (items != begun)
          wait_for(&s.o_full[me], (items - 1) & 1, &s.dead);
        else if (segment > 0)
          wait_for(&s.o_read, (segment - 1) & 1, &s.dead);
        // This thread's part of its position's values becomes fp16: half of them, or, where both groups need them, a quarter.
        wait_for(&s.v_full[st], n / kV & 1, &s.dead);
        {
          // 16 entries at once, the i-th of a row; chunks are mixed by exclusive or, in the tile and in the runs
          const uint32_t row =
              smem_addr(tiles_v) + st * Z::kTileBytes + position * kD + (kD == 128 ? position & 7 : position >> 1 & 3) * 16;
          const uint32_t to_row = smem_addr(wides) + (two_blocks ? n & 1 : me) * Z::kWide + position * 128 + (position & 7) * 16;
          auto store = [&](int i, uint4 e) {
            const uint32_t four[4] = {e.x, e.y, e.z, e.w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              h[2 * k] = half2_of(static_cast<uint16_t>(four[k]));
              h[2 * k + 1] = half2_of(static_cast<uint16_t>(four[k] >> 16));
            }
            const uint32_t to = to_row + i / 4 * (kTile * 128);
            shared_store(to ^ (2 * i & 7) * 16, make_uint4(h[0], h[1], h[2], h[3]));
            shared_store(to ^ (2 * i + 1 & 7) * 16, make_uint4(h[4], h[5], h[6], h[7]));
          };
          constexpr int kQuarter = kD / 64;
          if (two_blocks) {
            const int first = (me * 2 + half) * kQuarter;
            uint4 e[kQuarter];
#pragma unroll
            for (int c = 0; c < kQuarter; ++c) e[c] = shared_load(row ^ (first + c) * 16);
#pragma unroll
            for (int c = 0; c < kQuarter; ++c) store(first + c, e[c]);
            async_fence();
          } else {
            const int first = half * 2 * kQuarter;
            uint4 e[2 * kQuarter];
#pragma unroll
            for (int c = 0; c < 2 * kQuarter; ++c) e[c] = shared_load(row ^ (first + c) * 16);
#pragma unroll
            for (int c = 0; c < 2 * kQuarter; ++c) store(first + c, e[c]);
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.v_empty[st], two_blocks ? 1 : 2);
          if (two_blocks) mbar_arrive(&s.wide_full[n & 1]);
        }
        uint32_t w[kC / 2];
#pragma unroll
        for (int c = 0; c < kC; c += 2) {
          const Two p = two(power(x[c]), power(x[c + 1]));
          l[c / 2] = fma2(p, inverse2, l[c / 2]);
          w[c / 2] = half2_of(mul2(p, rest));
        }
        // runs of 8 columns, 16 bytes a position
        uint8_t* const to = mine + position * 16;
        auto run = [&](int col) { return to + col / 8 * (kTile * 16) + col % 8 * 2; };
        if constexpr (kC % 8 == 0) {
#pragma unroll
          for (int c = 0; c < kC; c += 8)
            *reinterpret_cast<uint4*>(run(half * kC + c)) = make_uint4(w[c / 2], w[c / 2 + 1], w[c / 2 + 2], w[c / 2 + 3]);
        } else {
#pragma unroll
          for (int c = 0; c < kC; c += 4) *reinterpret_cast<uint2*>(run(half * kC + c)) = make_uint2(w[c / 2], w[c / 2 + 1]);
        }
        async_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[me]);
        ++items;
      }
      for (int tile = max(t0, first_special); tile < t1; ++tile) ready ^= 1u << (count + (tile - t0)) % kV;
      count += t1 - t0;
      look_ahead(segment + 1);
      // ---- the segment's end.  Lane d of tensor memory is entry d: with 64 of them the first 16 lanes of each warp have one.
      if (items != begun) wait_for(&s.o_full[me], (items - 1) & 1, &s.dead);
      {
        float v[kC];
#pragma unroll
        for (int k = 0; k < kC; k += 2) both(l[k / 2], v[k], v[k + 1]);
        post(v, std::true_type());
      }
      if (t < kUsed) s.m[me][t] = m;
      if (me == 1 && t == 0) s.second_anchor = anchor;
      auto sync = [&]() {
        if (two_blocks)
          group_sync(me);
        else
          groups_sync();
      };
      sync();
      if (t < kUsed && (two_blocks || me == 0)) {
        auto sum = [&](int group) {
          return s.most[group][0][t] + s.most[group][1][t] + s.most[group][2][t] + s.most[group][3][t];
        };
        const float m1 = two_blocks ? -INFINITY : s.m[1][t], to = fmaxf(m, m1);
        const float f0 = m == to ? 1.f : power(m - to), f1 = m1 == -INFINITY ? 0.f : m1 == to ? 1.f : power(m1 - to);
        float all = sum(me) * f0;
        if (!two_blocks && f1 != 0.f) all += sum(1) * f1;
        const float over = s.dead ? NAN : g.whole ? 1.f / all : 1.f;
        s.worth[me][t] = f0 * over * anchor;
        if (!two_blocks) s.worth[1][t] = f1 * over * s.second_anchor;
        s.whole[me][t] = s.dead ? NAN : all;
        s.last[me][t] = to;
      }
      sync();
      tc_after();
      {
        const int d = kD == 128 ? position : quad * 16 + lane;
        const bool has = kD == 128 || lane < 16;
        const int block = two_blocks ? me : 0, cols = min(kN, g.cols - g.c0 - block * kN);
        float* const part = P.parts + (2 * static_cast<int64_t>(blockIdx.x) + g.front) * Z::kPart;
        const bool others = !two_blocks && t1 - t0 > 1;  // the second group has sums too
        // of one block eight columns a warp, which reads both groups' sums; of two each group's own
        const int from = two_blocks ? half * kC : (me * 2 + half) * 8, to = two_blocks ? from + kC : min(kUsed, from + 8);
#pragma unroll 1
        for (int c = from; c < to; c += 8) {
          const uint32_t at = tmem + lanes + (2 + block) * kN + c;
          float o[8], v[8];
          tc_load<8>(at, o);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = o[k] * s.worth[block][c + k];
          if (others) {
            tc_load<8>(at + kN, o);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = fmaf(o[k], s.worth[1][c + k], v[k]);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (has && c + k < cols) {
              if (g.whole)
                P.out[s.out[block][c + k] + d] = __float2bfloat16(v[k]);
              else
                part[(block * kN + c + k) * kD + d] = v[k];
            }
        }
        if (!g.whole && t < cols && (two_blocks || me == 0)) {
          part[Z::kColumns * kD + block * kN + t] = s.last[me][t];
          part[Z::kColumns * (kD + 1) + block * kN + t] = s.whole[me][t];
        }
      }
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_read), mbar_arrive(&s.g_free[segment & 3]);
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (s.dead) stay_behind();
  __syncwarp();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(4 * kN) : "memory");
}

// ---- parts of a unit together

constexpr int kJoinThreads = 128;

template <int kColumns, int kD>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttendParams P) {
  constexpr int kPart = kColumns * (kD + 2);
  wait_for_stream();
  // CTA i looks at the cut in front of the i + 1-st of the CTAs that shared the tiles
  const int at = blockIdx.x + 1;
  const Start start = P.cuts[at];
  const int64_t tile = cut(start.total, at, P.grid);
  if (start.b >= P.B) return;
  const Sequence s = sequence_of<kColumns>(P, start.b);
  const int64_t unit = divide(start.off, s.tiles), first = tile - (start.off - unit * s.tiles), last = first + s.tiles;
  // nothing is cut here, or an earlier cut is in this unit too
  if (tile == first || cut(start.total, at - 1, P.grid) > first) return;
  int parts = 1;
  while (at + parts - 1 < P.grid && cut(start.total, at + parts - 1, P.grid) < last) ++parts;
  const int h = static_cast<int>(unit / s.pairs), c0 = static_cast<int>(unit % s.pairs) * kColumns,
            cols = min(kColumns, s.cols - c0);
  const int lane = threadIdx.x & 31;
  const int64_t before = static_cast<int64_t>(at) - 1;  // the CTA with the first part
  // a CTA without tiles has no part: its place is skipped
  auto part = [&](int k) { return P.parts + (2 * (before + k) + (k == 0)) * kPart; };
  auto empty = [&](int k) {
    return cut(start.total, static_cast<int>(before) + k, P.grid) == cut(start.total, static_cast<int>(before) + k + 1, P.grid);
  };
  for (int c = blockIdx.y * (kJoinThreads / 32) + threadIdx.x / 32; c < cols; c += gridDim.y * (kJoinThreads / 32)) {
    // a lane has the factors of every 32nd part
    float m = -INFINITY;
    for (int k = lane; k < parts; k += 32)
      if (!empty(k)) m = fmaxf(m, part(k)[kColumns * kD + c]);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    float l = 0.f, v[kD / 32] = {};
    for (int k0 = 0; k0 < parts; k0 += 32) {
      float f = -1.f;  // there is none.  (A factor of 0 counts: what a part far below the others holds may be NaN.)
      if (k0 + lane < parts && !empty(k0 + lane)) {
        const float mk = part(k0 + lane)[kColumns * kD + c];
        f = mk == m ? 1.f : power(mk - m);
        l += part(k0 + lane)[kColumns * (kD + 1) + c] * f;
      }
#pragma unroll 4
      for (int k = 0; k < min(32, parts - k0); ++k) {
        const float fk = __shfl_sync(~0u, f, k);
        const float* p = part(k0 + k) + c * kD + lane;
        if (!(fk < 0.f))
#pragma unroll
          for (int e = 0; e < kD / 32; ++e) v[e] += p[32 * e] * fk;
      }
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    const int i = (c0 + c) / P.group;
    __nv_bfloat16* const to = P.out + (static_cast<int64_t>(s.start) + start.b + i) * P.out_row +
                              (static_cast<int64_t>(h) * P.group + c0 + c - i * P.group) * P.out_head;
#pragma unroll
    for (int e = 0; e < kD / 32; ++e) to[lane + 32 * e] = __float2bfloat16(v[e] / l);
  }
}

// ------------------------------------------------------------ host

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::atomic<EncodeTiled> found{nullptr};
  EncodeTiled f = found.load();
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult r;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
      r != cudaDriverEntryPointSuccess) {
    (void)cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<EncodeTiled>(p);
  found.store(f);
  return f;
}

// a map of [pages, heads, tokens, dim] entries in boxes of box x dim
bool map_entries(CUtensorMap* map, const sv_cache& c, void* base, void* none, int box) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const int64_t any = c.dim;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_tokens),
                              static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(std::max(1, c.pages))};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride), static_cast<cuuint64_t>(c.heads > 1 ? c.head_stride : any),
                                 static_cast<cuuint64_t>(c.pages > 1 ? c.page_stride : any)};
  const cuuint32_t boxes[4] = {static_cast<cuuint32_t>(c.dim), static_cast<cuuint32_t>(box), 1, 1}, step[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.pages > 0 ? base : none, dims, strides, boxes, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, c.dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Columns of a unit: as few as hold a sequence's rows, 64 at most (two blocks of 32).
int unit_columns(int group, int max_nodes) {
  const int64_t cols = static_cast<int64_t>(max_nodes + 1) * group;
  return cols <= 16 ? 16 : cols <= 32 ? 32 : 64;
}

template <int kN, int kBlocks, int kC, int kD>
sv_status launch_attend(const AttendParams& P, const Maps& maps, int device, cudaStream_t st) {
  constexpr int smem = Sizes<kN, kBlocks, kD>::kSmem;
  const auto kernel = attend_kernel<kN, kBlocks, kC, kD>;
  static std::atomic<bool> opted_in[64];
  if (device >= 64 || !opted_in[device].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return SV_ECUDA;
    if (device < 64) opted_in[device].store(true);
  }
  if (launch_waiting(kernel, P.grid, kAttendThreads, smem, 1, st, P, maps) != cudaSuccess) return SV_ECUDA;
  if (P.grid > 1 && launch_waiting(join_kernel<kN * kBlocks, kD>, dim3(P.grid - 1, kN * kBlocks / 8), kJoinThreads, 0, 1, st, P) !=
                        cudaSuccess)
    return SV_ECUDA;
  return SV_OK;
}

template <int kD>
sv_status launch_attend(const AttendParams& P, const Maps& maps, int columns, int64_t used, int device, cudaStream_t st) {
  // a thread takes half of the columns that there are, in fours
  if (columns == 16) return used <= 8 ? launch_attend<16, 1, 4, kD>(P, maps, device, st) : launch_attend<16, 1, 8, kD>(P, maps, device, st);
  if (columns == 32)
    return used <= 24 ? launch_attend<32, 1, 12, kD>(P, maps, device, st) : launch_attend<32, 1, 16, kD>(P, maps, device, st);
  return launch_attend<32, 2, 16, kD>(P, maps, device, st);
}

int sms_of(int device) {
  int sms = 0;
  return cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess ? sms : 0;
}

}  // namespace
}  // namespace sv

extern "C" size_t spec_verify_attend_workspace(int heads, int q_heads, int dim, int max_nodes, int device) {
  if (heads < 1 || q_heads < 1 || dim < 1 || max_nodes < 0 || max_nodes > SV_MAX_NODES) return 0;
  const size_t sms = sv::sms_of(device);
  return (sms + sms % 2) * sizeof(sv::Start) + 2 * sms * sv::unit_columns(q_heads / heads, max_nodes) * (dim + 2) * sizeof(float);
}

extern "C" sv_status spec_verify_attend(const sv_cache* cache, const void* q, int64_t q_row, int64_t q_head, void* out,
                                        int64_t out_row, int64_t out_head, int q_heads, float scale,
                                        const int32_t* page_table, int64_t table_stride, int table_cols,
                                        const int32_t* context, const int32_t* node_start, const int32_t* parent, int B,
                                        int total_nodes, int max_nodes, void* workspace, size_t workspace_bytes, int device,
                                        void* cuda_stream) {
  if (sv_status s = sv::check_cache(cache, 1); s != SV_OK) return s;
  if (sv_status s = sv::check_table(page_table, table_stride, table_cols, B); s != SV_OK) return s;
  if (q_heads < 1 || q_heads % cache->heads || !std::isfinite(scale)) return SV_EINVAL;
  if (std::fabs(scale) > 0x1p126f) return SV_EUNSUPPORTED;  // (in base 2 it is 1.44 times as large)
  if (B < 0 || total_nodes < 0 || max_nodes < 0) return SV_EINVAL;
  if (max_nodes > SV_MAX_NODES) return SV_EUNSUPPORTED;
  if (q_row < 0 || q_head < 0 || out_row < 0 || out_head < 0) return SV_EINVAL;
  for (const int64_t s : {q_row, q_head, out_row, out_head})
    if (s >= (int64_t{1} << 40)) return SV_EUNSUPPORTED;
  if (B == 0) return SV_OK;
  if (static_cast<int64_t>(total_nodes) + B > INT32_MAX || q_heads / cache->heads > (1 << 20)) return SV_EUNSUPPORTED;
  if (!q || !out || !context || !node_start) return SV_EINVAL;
  const int rows = total_nodes + B;
  // (the stride of a dimension of one is not used)
  if ((rows > 1 && q_row % 8) || (q_heads > 1 && q_head % 8) || reinterpret_cast<uintptr_t>(q) % 16 ||
      reinterpret_cast<uintptr_t>(out) % 2)
    return SV_EINVAL;
  for (const void* p : {static_cast<const void*>(context), static_cast<const void*>(node_start),
                        static_cast<const void*>(parent)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SV_EINVAL;
  if (!sv::rows_apart(out_head, out_row, q_heads, rows, cache->dim)) return SV_EINVAL;
  if (sv::sure_to_overlap({q, 2, cache->dim, q_head, q_heads, q_row, rows},
                          {out, 2, cache->dim, out_head, q_heads, out_row, rows}))
    return SV_EINVAL;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16) return SV_EINVAL;
  sv::DeviceGuard g(device);
  if (!g.ok) return SV_ECUDA;
  const int sms = sv::sms_of(device);
  if (sms < 1) return SV_ECUDA;
  if (workspace_bytes < spec_verify_attend_workspace(cache->heads, q_heads, cache->dim, max_nodes, device)) return SV_EINVAL;
  sv::AttendParams P = {};
  P.c = sv::view_of(*cache, page_table, table_stride, table_cols);
  P.q = static_cast<const __nv_bfloat16*>(q), P.out = static_cast<__nv_bfloat16*>(out);
  P.q_row = q_row, P.q_head = q_head, P.out_row = out_row, P.out_head = out_head;
  P.group = q_heads / cache->heads;
  P.scale = scale * 1.4426950408889634f;
  P.context = context, P.node_start = node_start, P.parent = parent;
  P.B = B, P.total = total_nodes, P.max_nodes = max_nodes;
  P.box_tokens = std::min(cache->page_tokens, sv::kTile);
  P.boxes = sv::kTile / P.box_tokens;
  P.page_scales = cache->heads * (cache->page_tokens / cache->block), P.in_page = static_cast<unsigned>(cache->page_tokens) - 1u;
  P.grid = sms;
  P.cuts = static_cast<sv::Start*>(workspace);
  P.parts = reinterpret_cast<float*>(P.cuts + sms + (sms & 1));
  sv::Maps maps;
  if (!sv::map_entries(&maps.k, *cache, cache->k, workspace, P.box_tokens) ||
      !sv::map_entries(&maps.v, *cache, cache->v, workspace, P.box_tokens))
    return SV_ECUDA;
  const int columns = sv::unit_columns(P.group, max_nodes);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int64_t used = static_cast<int64_t>(max_nodes + 1) * P.group;
  return cache->dim == 128 ? sv::launch_attend<128>(P, maps, columns, used, device, st)
                           : sv::launch_attend<64>(P, maps, columns, used, device, st);
}
