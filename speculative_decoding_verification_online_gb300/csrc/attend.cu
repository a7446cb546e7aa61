// Attention of drafted rows over a cache of 8-bit entries: spec_verify_attend.
//
//   out[r, h] = sum_p softmax_p(scale q[r, h] . K[p]) V[p],  p over the committed positions and the row's path
//
// Keys and values go from memory to the tensor cores as they are, in 8 bits.  A query of
// eight significant bits is the exact sum of two e4m3 numbers (times a power of two for
// its row), and a weight is rounded to two: hi = e4m3(w), lo = e4m3(w - hi), as good as
// a rounding to bf16.  So S = K (Qhi + Qlo)^T and O = V^T (Phi + Plo), two products each
// at twice the rate of bf16's, and nothing is converted but queries and weights.
//
// A key head's query rows (all rows of the step times the query heads of its group) are
// the columns: up to kN of them make a block.  Positions are rows, 128 to a tile: thread
// t of a warpgroup has position t of every column, so that a position's scale and
// visibility are the thread's own.  The softmax is per tile: weights times their value's
// scale stand against the tile's own largest such product (times 2^8, of the 448 that
// e4m3 holds), so that what is small against another tile's does not fall below e4m3's
// range; the tiles' sums are joined in fp32 registers.
//
// Work is cut evenly over the SMs, whatever the lengths: all tiles of all units (sequence, key
// head, two blocks of columns) in a row, a CTA taking the n-th part of them.  A unit that
// is cut leaves its parts in the workspace, and a second kernel joins them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "cache.cuh"
#include "entry.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

constexpr int kTile = 128;  // positions
constexpr int kGroupThreads = 128;
constexpr int kAttendThreads = 128 + 2 * kGroupThreads;
constexpr int kMaxStages = 8;
constexpr int kAttendSmem = 226 * 1024;
constexpr float kTop = 8.f;  // log2 of a tile's largest weight

struct AttendParams {
  CacheView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t q_row, q_head, out_row, out_head;
  int group;
  float scale;  // times log2(e)
  const int32_t *context, *node_start, *parent;
  int B, total, max_nodes;
  int stages, boxes, box_tokens;  // boxes of a tile
  int grid;                       // CTAs that share the tiles
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

template <int kN>
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
  s.pairs = (s.cols + 2 * kN - 1) / (2 * kN);
  s.units = static_cast<int64_t>(P.c.heads) * s.pairs;
  s.work = s.units * s.tiles;
  return s;
}

__device__ __forceinline__ int64_t cut(int64_t total, int i, int n) { return total / n * i + total % n * i / n; }

struct Start {
  int64_t total;
  int b;
  int64_t off;  // in sequence b's work
};

// Where tile `at(total)` of all lies; every thread of the CTA calls it.
template <int kN, typename F>
__device__ __forceinline__ void find_tile(const AttendParams& P, F&& at, Start* s, int64_t* warp_sums) {
  const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (P.B + threads - 1) / threads;
  const int lo = min(P.B, static_cast<int>(threadIdx.x) * per), hi = min(P.B, lo + per);
  int64_t mine = 0;
  for (int b = lo; b < hi; ++b) mine += sequence_of<kN>(P, b).work;
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
      const int64_t w = sequence_of<kN>(P, b).work;
      if (tile < base + w) {
        s->b = b, s->off = tile - base;
        break;
      }
      base += w;
    }
  }
  __syncthreads();
}

// A run of tiles of one unit.
struct Segment {
  Sequence s;
  int b, h, c0, t0, t1;  // c0: the first column
  bool two, whole_front, whole;  // two blocks of columns; from the unit's first tile on; all of the unit's tiles
};

template <int kN>
struct Walk {
  const AttendParams& P;
  int64_t pos, hi, off;
  int b;
  Sequence s;
  bool loaded = false;

  __device__ __forceinline__ Walk(const AttendParams& P, const Start& at, int64_t lo, int64_t hi)
      : P(P), pos(lo), hi(hi), off(at.off), b(at.b) {}

  __device__ __forceinline__ bool next(Segment& g) {
    if (pos >= hi) return false;
    while (!loaded || off >= s.work) {
      if (loaded) ++b, off = 0;
      if (b >= P.B) return false;
      s = sequence_of<kN>(P, b);
      loaded = true;
    }
    const int64_t unit = off / s.tiles;
    g.s = s, g.b = b;
    g.h = static_cast<int>(unit / s.pairs);
    g.c0 = static_cast<int>(unit % s.pairs) * 2 * kN;
    g.t0 = static_cast<int>(off - unit * s.tiles);
    const int64_t left = hi - pos, here = s.tiles - g.t0, n = left < here ? left : here;
    g.t1 = g.t0 + static_cast<int>(n);
    g.two = s.cols - g.c0 > kN;
    g.whole_front = g.t0 == 0;
    g.whole = g.t0 == 0 && g.t1 == s.tiles;
    pos += n, off += n;
    return true;
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

__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// kCols columns of this warp's 32 lanes
template <int kCols>
__device__ __forceinline__ void tc_load(uint32_t addr, float (&f)[kCols]) {
#pragma unroll
  for (int c = 0; c < kCols; c += 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=f"(f[c]), "=f"(f[c + 1]), "=f"(f[c + 2]), "=f"(f[c + 3]), "=f"(f[c + 4]), "=f"(f[c + 5]), "=f"(f[c + 6]),
          "=f"(f[c + 7]), "=f"(f[c + 8]), "=f"(f[c + 9]), "=f"(f[c + 10]), "=f"(f[c + 11]), "=f"(f[c + 12]),
          "=f"(f[c + 13]), "=f"(f[c + 14]), "=f"(f[c + 15])
        : "r"(addr + c)
        : "memory");
#pragma unroll
  for (int c = 0; c < kCols; c += 16)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(f[c]), "+f"(f[c + 1]), "+f"(f[c + 2]), "+f"(f[c + 3]), "+f"(f[c + 4]), "+f"(f[c + 5]),
                   "+f"(f[c + 6]), "+f"(f[c + 7]), "+f"(f[c + 8]), "+f"(f[c + 9]), "+f"(f[c + 10]), "+f"(f[c + 11]),
                   "+f"(f[c + 12]), "+f"(f[c + 13]), "+f"(f[c + 14]), "+f"(f[c + 15])
                 :
                 : "memory");
}

// Operands in shared memory (all of their offsets in units of 16 bytes).
// Tiles of K and V: rows of kD bytes, 128- or 64-byte swizzle, groups of 8 rows behind one another.  As they lie they are K-major
// for K (its rows are the rows of the product, kD its inner dimension), and for V, whose rows are the inner dimension,
// transposed.  Q's rows lie like K's.
template <int kD>
__device__ __forceinline__ uint64_t rows_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (1ull << 16) | (static_cast<uint64_t>(kD * 8 / 16) << 32) | (1ull << 46) |
         (kD == 128 ? 2ull << 61 : 4ull << 61);
}
// Weights: runs of 16 columns, 16 bytes for each position, a run's 128 positions behind one another; no swizzle.  Eight positions
// on: 128 bytes; a run on: 2048.
__device__ __forceinline__ uint64_t weights_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (8ull << 16) | (128ull << 32) | (1ull << 46);
}

__device__ __forceinline__ float power(float x) {  // 2^x; results below 2^-126 become 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Each column's largest, or sum, over a warp's lanes: halves of the columns change hands until a lane has its own.  Of 32
// columns lane i gets column i; of 16 column i / 2.
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

template <int kN>
struct AttendShared {
  static constexpr int kWords = kN > 32 ? kN / 32 : 1;  // of a block's visibility
  // of a position: the scale of K; a power of two c that is not below the scale of V over the tile's largest (but 2^-12 at
  // least) as log2 c and 1 / c; the rest of that scale, over c
  float4 factor[kMaxStages][kTile];
  uint32_t seen[kMaxStages][kTile][2 * kWords];
  float vmost[kMaxStages];
  int special[kMaxStages];
  float most[2][4][kN];                    // a warp's largest logits, and at last its sums
  float ref[2][kN];                        // what a tile's logits stand against
  float keep[2][kN], take[2][kN];          // factors of the sums so far and of the tile's
  float row[2][kN];                        // of a query row: its power of two, the softmax's scale
  float m[2][kN];
  float lsum[kN];
  uint32_t path[2][SV_MAX_NODES][2 * kWords];
  int parent[2][SV_MAX_NODES];
  uint64_t full[kMaxStages], ready[kMaxStages], empty[kMaxStages];
  uint64_t s_full[2], s_free[2], p_full[2], o_full[2], q_full;
  int64_t warp_sums[kAttendThreads / 32];
  Start start;
  uint32_t tmem;
  volatile int dead;
};

template <int kN, int kD>
struct Sizes {
  static constexpr int kTileBytes = kTile * kD, kStageBytes = 2 * kTileBytes;
  static constexpr int kQ = kN * kD, kWeights = kTile * kN;  // one of the two numbers of a block's entries
  static constexpr int kFixed = 1024 + 4 * kQ + 4 * kWeights;
  static constexpr int kFits = (kAttendSmem - 1024 - static_cast<int>(sizeof(AttendShared<kN>)) - kFixed) / kStageBytes;
  static constexpr int kStages = kFits < kMaxStages ? kFits : kMaxStages;
  static constexpr int kPart = 2 * kN * (kD + 2);  // floats of a part in the workspace
  static_assert(kStages >= 3);
};

__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ void groups_sync() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

// smallest power of two that brings values of up to `a` to 448 at most (2^-100 at least)
__device__ __forceinline__ float power_for(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 126;
  const int k = max(-100, (u & 0x7fffffu) <= 0x600000u ? e - 9 : e - 8);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

__device__ __forceinline__ bool holds_nan(uint4 e) {
  // 0x7f in the low seven bits of a byte
  const auto hit = [](uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
  return (hit(e.x) | hit(e.y) | hit(e.z) | hit(e.w)) != 0;
}

template <int kN, int kD>
__global__ void __launch_bounds__(kAttendThreads, 1) attend_kernel(const __grid_constant__ AttendParams P,
                                                                   const __grid_constant__ Maps maps) {
  using Z = Sizes<kN, kD>;
  using Shared = AttendShared<kN>;
  constexpr int kWords = Shared::kWords, kWordCols = kN < 32 ? kN : 32;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(16) Shared s;
  uint8_t* const base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  uint8_t* const tiles = base;                                   // stages: K, V
  uint8_t* const queries = tiles + P.stages * Z::kStageBytes;    // [block][hi, lo]
  uint8_t* const weights = queries + 4 * Z::kQ;                  // [warpgroup][hi, lo]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < P.stages; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.ready[i], 1), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(&s.s_full[i], 1), mbar_init(&s.s_free[i], 4), mbar_init(&s.p_full[i], 4), mbar_init(&s.o_full[i], 1);
    mbar_init(&s.q_full, 8);
    s.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s.tmem)), "n"(4 * kN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  wait_for_stream();
  int64_t lo = 0;
  find_tile<kN>(P, [&](int64_t total) { return cut(total, blockIdx.x, P.grid); }, &s.start, s.warp_sums);
  tc_before();
  __syncthreads();
  tc_after();
  const Start start = s.start;
  lo = cut(start.total, blockIdx.x, P.grid);
  const int64_t hi = cut(start.total, blockIdx.x + 1, P.grid);
  const uint32_t tmem = s.tmem;  // S of the two groups, then O
  Walk<kN> walk(P, start, lo, hi);
  Segment g;
  if (warp == 0) {
    // ---- tiles by TMA, a lane for each of a tile's boxes
    unsigned count = 0;
    while (walk.next(g)) {
      auto page_at = [&](int t) {
        const int64_t pos = static_cast<int64_t>(t) * kTile + lane * P.box_tokens;
        int page = -1;
        if (lane < P.boxes && !g.s.lost && t < g.t1 && pos < g.s.end) page = P.c.page_of(g.b, pos);
        return page < 0 ? max(1, P.c.pages) : page;  // (behind the last page: zeros)
      };
      int page = page_at(g.t0);
      for (int t = g.t0; t < g.t1; ++t, ++count) {
        const int st = count % P.stages;
        const int next = page_at(t + 1);
        if (count >= static_cast<unsigned>(P.stages)) mbar_wait(&s.empty[st], (count / P.stages - 1) & 1, &s.dead);
        if (lane == 0) mbar_expect(&s.full[st], Z::kStageBytes);
        __syncwarp();
        if (lane < P.boxes) {
          const int token = static_cast<int>((static_cast<int64_t>(t) * kTile + lane * P.box_tokens) & ((1 << P.c.page_log) - 1));
          const uint32_t to = smem_addr(tiles + st * Z::kStageBytes) + lane * P.box_tokens * kD;
          tma_load(&maps.k, to, &s.full[st], token, g.h, page);
          tma_load(&maps.v, to + Z::kTileBytes, &s.full[st], token, g.h, page);
        }
        page = next;
      }
    }
  } else if (warp == 1) {
    // ---- products
    constexpr unsigned kQk = (1u << 4) | (static_cast<unsigned>(kN / 8) << 17) | (8u << 24);
    constexpr unsigned kPv =
        (1u << 4) | (1u << 15) | (1u << 16) | (static_cast<unsigned>(kN / 8) << 17) | (static_cast<unsigned>(kD / 16) << 24);
    unsigned count = 0, segment = 0, done[2] = {0, 0}, asked[2] = {0, 0};
    while (walk.next(g)) {
      mbar_wait(&s.q_full, segment++ & 1, &s.dead);
      const int items = (g.t1 - g.t0) << (g.two ? 1 : 0);
      for (int i = 0; i <= items; ++i) {
        if (i < items) {
          const int w = i & 1, tile = g.two ? i / 2 : i;
          const unsigned n = count + tile, st = n % P.stages;
          if (!g.two || w == 0) {
            mbar_wait(&s.full[st], n / P.stages & 1, &s.dead);
            mbar_wait(&s.ready[st], n / P.stages & 1, &s.dead);
          }
          if (asked[w] > 0) mbar_wait(&s.s_free[w], (asked[w] - 1) & 1, &s.dead);
          ++asked[w];
          tc_after();
          const uint64_t k = rows_desc<kD>(smem_addr(tiles + st * Z::kStageBytes));
          const uint64_t q = rows_desc<kD>(smem_addr(queries + (g.two ? w : 0) * 2 * Z::kQ));
          if (elect_one()) {
#pragma unroll
            for (int piece = 0; piece < 2; ++piece)
#pragma unroll
              for (int d = 0; d < kD / 32; ++d)
                tc_mma(tmem + w * kN, k + 2 * d, q + piece * (Z::kQ / 16) + 2 * d, kQk, piece + d > 0);
            tc_commit(&s.s_full[w]);
          }
          __syncwarp();
        }
        if (i > 0) {
          const int j = i - 1, w = j & 1, tile = g.two ? j / 2 : j;
          const unsigned n = count + tile, st = n % P.stages;
          mbar_wait(&s.p_full[w], done[w]++ & 1, &s.dead);
          tc_after();
          const uint64_t v = rows_desc<kD>(smem_addr(tiles + st * Z::kStageBytes + Z::kTileBytes));
          const uint64_t p = weights_desc(smem_addr(weights + w * 2 * Z::kWeights));
          if (elect_one()) {
#pragma unroll
            for (int piece = 0; piece < 2; ++piece)
#pragma unroll
              for (int t = 0; t < kTile / 32; ++t)
                tc_mma(tmem + (2 + w) * kN, v + t * (32 * kD / 16), p + piece * (Z::kWeights / 16) + t * 32, kPv, piece + t > 0);
            tc_commit(&s.o_full[w]);
            if (!g.two || w == 1) tc_commit(&s.empty[st]);
          }
          __syncwarp();
        }
      }
      count += g.t1 - g.t0;
    }
  } else if (warp < 4) {
    // ---- scales and visibility of a tile's positions, by turns
    const int me = warp - 2;
    unsigned count = 0;
    while (walk.next(g)) {
      bool built = false, bad = false;
      for (int t = g.t0; t < g.t1; ++t, ++count) {
        if ((count & 1) != static_cast<unsigned>(me)) continue;
        const int st = count % P.stages;
        const int64_t p0 = static_cast<int64_t>(t) * kTile;
        const bool special = g.s.lost || p0 + kTile > g.s.context + 1;
        float kf[4], vf[4];
        bool none[4];  // no page
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t pos = p0 + lane + 32 * i;
          kf[i] = vf[i] = 0.f;
          none[i] = g.s.lost;
          if (!g.s.lost && pos < g.s.end) {
            const int page = P.c.page_of(g.b, pos);
            none[i] = page < 0;
            if (page >= 0) {
              const int64_t at = P.c.scale_at(page, g.h, pos);
              kf[i] = P.c.scales[0][at], vf[i] = P.c.scales[1][at];
            }
          }
        }
        float most = fmaxf(fmaxf(vf[0], vf[1]), fmaxf(vf[2], vf[3]));
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
        if (special && !built && !g.s.lost && P.parent) {
          // rows of the path of each node's column
          built = true;
          __syncwarp();
          for (int i = lane; i < g.s.nodes; i += 32) {
            const int up = P.parent[g.s.start + i];
            bad |= up < -1 || up >= i;
            s.parent[me][i] = up;
#pragma unroll
            for (int w = 0; w < 2 * kWords; ++w) s.path[me][i][w] = 0;
          }
          bad = __any_sync(~0u, bad);
          __syncwarp();
          const int last = min(g.s.nodes, (g.c0 + 2 * kN - 1) / P.group);
          for (int i = g.c0 / P.group + lane; !bad && i <= last; i += 32) {
            const int from = i * P.group - g.c0, to = from + P.group;
            for (int node = i - 1; node >= 0; node = s.parent[me][node])
#pragma unroll
              for (int w = 0; w < 2 * kWords; ++w) {
                const int a = max(0, from - w * kWordCols), e = min(kWordCols, to - w * kWordCols);
                if (e > a) atomicOr(&s.path[me][node][w], (e - a == 32 ? ~0u : ((1u << (e - a)) - 1u)) << a);
              }
          }
          __syncwarp();
        }
        if (count >= static_cast<unsigned>(P.stages)) mbar_wait(&s.empty[st], (count / P.stages - 1) & 1, &s.dead);
        if (special) mbar_wait(&s.full[st], count / P.stages & 1, &s.dead);
        uint8_t* const v = tiles + st * Z::kStageBytes + Z::kTileBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = lane + 32 * i;
          if (special) {
            const int64_t pos = p0 + at, node = pos - g.s.context - 1;
            uint32_t seen[2 * kWords];
#pragma unroll
            for (int w = 0; w < 2 * kWords; ++w) seen[w] = ~0u;
            if (!g.s.lost && node >= 0) {
              // What a position holds that not every row sees goes through the product of every row: nothing but numbers
              // may stand there.
              uint4* row = reinterpret_cast<uint4*>(v + at * kD);
              bool nan = false;
              if (pos < g.s.end)
                for (int c = 0; c < kD / 16; ++c) nan |= holds_nan(row[c]);
              if (nan || pos >= g.s.end)
                for (int c = 0; c < kD / 16; ++c) row[c] = make_uint4(0, 0, 0, 0);
              if (nan || bad) kf[i] = NAN;
              if (none[i]) {
              } else if (pos >= g.s.end) {
#pragma unroll
                for (int w = 0; w < 2 * kWords; ++w) seen[w] = 0;
              } else if (!bad && P.parent) {
#pragma unroll
                for (int w = 0; w < 2 * kWords; ++w) seen[w] = s.path[me][node][w];
              } else if (!bad) {
                const int from = static_cast<int>(node + 1) * P.group - g.c0;  // the first column that sees it
#pragma unroll
                for (int w = 0; w < 2 * kWords; ++w) {
                  const int a = from - w * kWordCols;
                  seen[w] = a <= 0 ? ~0u : a >= 32 ? 0u : ~0u << a;
                }
              }
            }
#pragma unroll
            for (int w = 0; w < 2 * kWords; ++w) s.seen[st][at][w] = seen[w];
          }
          const float ratio = most > 0.f ? vf[i] / most : vf[i];
          // ratio = f * 2^e, f in [1/2, 1): 2^e, or 2^(e - 1) where f is 1/2
          const uint32_t u = __float_as_uint(ratio);
          const int e = max(-12, min(0, static_cast<int>(u >> 23) - 126 - ((u & 0x7fffffu) == 0)));
          s.factor[st][at] = make_float4(none[i] ? NAN : kf[i], e, __uint_as_float((127 - e) << 23),
                                         ratio * __uint_as_float((127 - e) << 23));
        }
        if (lane == 0) s.vmost[st] = most > 0.f ? most : 1.f, s.special[st] = special;
        if (special) async_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.ready[st]);
      }
    }
  } else {
    // ---- softmax
    const int me = (warp - 4) / 4, quad = warp & 3, t = threadIdx.x - 128 - me * kGroupThreads;
    const uint32_t lanes = static_cast<uint32_t>(quad) << 21;  // 32 lanes of tensor memory each
    unsigned count = 0, items = 0;
    uint8_t* const mine = weights + me * 2 * Z::kWeights;
    float* const others = reinterpret_cast<float*>(weights);  // the second group's sums at a segment's end
    while (walk.next(g)) {
      // the queries, a warp for each row: two e4m3 numbers an entry, of the entry over its row's power of two
      constexpr int kPer = kD / 32;
      const int rows = g.two ? 2 * kN : kN;
      for (int r = warp - 4; r < rows; r += 8) {
        const int col = g.c0 + r;
        float q[kPer] = {};
        if (col < g.s.cols) {
          const int i = col / P.group;
          const __nv_bfloat16* p = P.q + (static_cast<int64_t>(g.s.start) + g.b + i) * P.q_row +
                                   (static_cast<int64_t>(g.h) * P.group + col - i * P.group) * P.q_head + lane * kPer;
          uint32_t u[kPer / 2];
          if constexpr (kPer == 4) {
            const uint2 e = *reinterpret_cast<const uint2*>(p);
            u[0] = e.x, u[1] = e.y;
          } else {
            u[0] = *reinterpret_cast<const uint32_t*>(p);
          }
#pragma unroll
          for (int k = 0; k < kPer / 2; ++k)
            q[2 * k] = __uint_as_float(u[k] << 16), q[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
        }
        float most = 0.f;
        bool fine = true;
#pragma unroll
        for (int k = 0; k < kPer; ++k) most = fmaxf(most, fabsf(q[k])), fine &= fabsf(q[k]) < INFINITY;
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
        fine = __all_sync(~0u, fine);
        const float unit = fine ? power_for(most) : 1.f, inverse = 1.f / unit;
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) {
          const float a = q[2 * k] * inverse, b = q[2 * k + 1] * inverse;
          const uint32_t h = e4m3x2(a, b);
          const float2 f = from_e4m3x2(h);
          hi |= h << (16 * k), lo |= e4m3x2(a - f.x, b - f.y) << (16 * k);
        }
        const int block = r / kN, row = r % kN, byte = lane * kPer, chunk = byte / 16;
        const int swizzled = kD == 128 ? chunk ^ (row & 7) : chunk ^ (row >> 1 & 3);
        uint8_t* const to = queries + block * 2 * Z::kQ + row * kD + swizzled * 16 + byte % 16;
        if constexpr (kPer == 4) {
          *reinterpret_cast<uint32_t*>(to) = hi, *reinterpret_cast<uint32_t*>(to + Z::kQ) = lo;
        } else {
          *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(hi);
          *reinterpret_cast<uint16_t*>(to + Z::kQ) = static_cast<uint16_t>(lo);
        }
        if (lane == 0) {
          const float f = fine ? unit * P.scale : NAN;
          s.row[block][row] = f;
        }
      }
      async_fence();
      groups_sync();  // the rows' factors are there for both groups
      if (lane == 0) mbar_arrive(&s.q_full);
      const float* const factors = s.row[g.two ? me : 0];
      float o[kN], l[kN < 32 ? 1 : kN / 32], m = -INFINITY;
#pragma unroll
      for (int c = 0; c < kN; ++c) o[c] = 0.f;
#pragma unroll
      for (int c = 0; c < (kN < 32 ? 1 : kN / 32); ++c) l[c] = 0.f;
      constexpr int kChunk = kN < 32 ? kN : 32;
      const int own = kN < 32 ? lane >> 1 : lane;  // this lane's column of a chunk
      for (int tile = g.two ? 0 : me; tile < g.t1 - g.t0; tile += g.two ? 1 : 2) {
        const unsigned n = count + tile, st = n % P.stages;
        mbar_wait(&s.ready[st], n / P.stages & 1, &s.dead);
        mbar_wait(&s.s_full[me], items & 1, &s.dead);
        tc_after();
        float x[kN];
        tc_load<kN>(tmem + lanes + me * kN, x);
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.s_free[me]);
        const float4 mul = s.factor[st][t];
#pragma unroll
        for (int c = 0; c < kN; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(factors + c);
          x[c] = fmaf(x[c] * f.x, mul.x, mul.y), x[c + 1] = fmaf(x[c + 1] * f.y, mul.x, mul.y);
          x[c + 2] = fmaf(x[c + 2] * f.z, mul.x, mul.y), x[c + 3] = fmaf(x[c + 3] * f.w, mul.x, mul.y);
        }
        if (s.special[st]) {
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            const uint32_t seen = s.seen[st][t][(g.two ? me : 0) * kWords + w];
#pragma unroll
            for (int c = 0; c < kWordCols; ++c)
              if (!(seen >> c & 1u)) x[w * kWordCols + c] = -INFINITY;
          }
        }
#pragma unroll
        for (int c = 0; c < kN; c += kChunk) s.most[me][quad][c + own] = over_lanes<kChunk, false>(x + c);
        group_sync(me);
        if (t < kN) {
          const float mt = fmaxf(fmaxf(s.most[me][0][t], s.most[me][1][t]), fmaxf(s.most[me][2][t], s.most[me][3][t]));
          const float to = fmaxf(m, mt);
          s.ref[me][t] = (mt == -INFINITY ? 0.f : mt) - kTop;
          s.keep[me][t] = m == to ? 1.f : power(m - to);
          s.take[me][t] = mt == -INFINITY ? 0.f : power(mt - to);
          m = to;
        }
        group_sync(me);
#pragma unroll
        for (int c = 0; c < kN; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&s.ref[me][c]);
          x[c] = power(x[c] - f.x), x[c + 1] = power(x[c + 1] - f.y), x[c + 2] = power(x[c + 2] - f.z),
          x[c + 3] = power(x[c + 3] - f.w);
        }
#pragma unroll
        for (int c = 0; c < kN; c += kChunk) {
          float p[kChunk];
#pragma unroll
          for (int k = 0; k < kChunk; ++k) p[k] = x[c + k] * mul.z;
          const float sum = over_lanes<kChunk, true>(p);
          l[c / kChunk] = l[c / kChunk] * s.keep[me][c + own] + sum * s.take[me][c + own];
        }
#pragma unroll
        for (int c = 0; c < kN; c += 16) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = x[c + 4 * k] * mul.w, b = x[c + 4 * k + 1] * mul.w, d = x[c + 4 * k + 2] * mul.w,
                        e = x[c + 4 * k + 3] * mul.w;
            const uint32_t h0 = e4m3x2(a, b), h1 = e4m3x2(d, e);
            const float2 f0 = from_e4m3x2(h0), f1 = from_e4m3x2(h1);
            hi[k] = h0 | h1 << 16;
            lo[k] = e4m3x2(a - f0.x, b - f0.y) | e4m3x2(d - f1.x, e - f1.y) << 16;
          }
          uint4* const to = reinterpret_cast<uint4*>(mine + c / 16 * (kTile * 16) + t * 16);
          to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          to[Z::kWeights / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        const float vmost = s.vmost[st];  // behind the arrival the stage may be filled again
        async_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[me]);
        mbar_wait(&s.o_full[me], items & 1, &s.dead);
        tc_after();
        ++items;
#pragma unroll
        for (int c = 0; c < kN; c += 16) {
          float u[16];
          tc_load<16>(tmem + lanes + (2 + me) * kN + c, u);
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            const float4 a = *reinterpret_cast<const float4*>(&s.keep[me][c + k]),
                         b = *reinterpret_cast<const float4*>(&s.take[me][c + k]);
            o[c + k] = o[c + k] * a.x + u[k] * (b.x * vmost), o[c + k + 1] = o[c + k + 1] * a.y + u[k + 1] * (b.y * vmost);
            o[c + k + 2] = o[c + k + 2] * a.z + u[k + 2] * (b.z * vmost);
            o[c + k + 3] = o[c + k + 3] * a.w + u[k + 3] * (b.w * vmost);
          }
        }
        tc_before();
      }
      count += g.t1 - g.t0;
      // ---- the segment's end.  Lane d of tensor memory is entry d: with 64 of them the first 16 lanes of each warp have one.
      const int d = kD == 128 ? t : quad * 16 + lane;
      const bool has = kD == 128 || lane < 16;
#pragma unroll
      for (int c = 0; c < kN; c += kChunk) s.most[me][quad][c + own] = l[c / kChunk];
      if (t < kN) s.m[me][t] = m;
      groups_sync();
      if (!g.two && me == 1) {
        if (has)
#pragma unroll
          for (int c = 0; c < kN; ++c) others[c * kD + d] = o[c];
      }
      if (t < kN && (g.two || me == 0)) {
        float sum = s.most[me][0][t] + s.most[me][1][t] + s.most[me][2][t] + s.most[me][3][t], to = m, f1 = 0.f;
        if (!g.two) {
          to = fmaxf(m, s.m[1][t]);
          f1 = s.m[1][t] == -INFINITY ? 0.f : power(s.m[1][t] - to);
          sum = sum * (m == to ? 1.f : power(m - to)) + f1 * (s.most[1][0][t] + s.most[1][1][t] + s.most[1][2][t] + s.most[1][3][t]);
        }
        // (in the first group's places of a segment of one block)
        s.keep[me][t] = m == to ? 1.f : power(m - to);
        s.take[me][t] = f1;
        s.ref[me][t] = sum;
        m = to;
      }
      if (!g.two)
        groups_sync();
      else
        group_sync(me);
      if (g.two || me == 0) {
        const int c0 = g.c0 + (g.two ? me * kN : 0), cols = min(kN, g.s.cols - c0);
        const bool ok = !s.dead;
        if (g.whole) {
          __nv_bfloat16* const to = P.out + (static_cast<int64_t>(g.s.start) + g.b) * P.out_row +
                                    static_cast<int64_t>(g.h) * P.group * P.out_head + d;
#pragma unroll
          for (int c = 0; c < kN; ++c) {
            float v = o[c] * s.keep[me][c];
            if (!g.two && has) v += others[c * kD + d] * s.take[me][c];
            v = ok ? v / s.ref[me][c] : NAN;
            const int i = (c0 + c) / P.group;
            if (has && c < cols) to[i * P.out_row + (c0 + c - i * P.group) * P.out_head] = __float2bfloat16(v);
          }
        } else {
          float* const to = P.parts + (2 * static_cast<int64_t>(blockIdx.x) + g.whole_front) * Z::kPart;
          const int first = g.two ? me * kN : 0;
#pragma unroll
          for (int c = 0; c < kN; ++c) {
            float v = o[c] * s.keep[me][c];
            if (!g.two && has) v += others[c * kD + d] * s.take[me][c];
            if (has && c < cols) to[(first + c) * kD + d] = v;
          }
          if (t < cols) {
            to[2 * kN * kD + first + t] = m;
            to[2 * kN * (kD + 1) + first + t] = ok ? s.ref[me][t] : NAN;
          }
        }
      }
      groups_sync();  // queries, weights and factors are free again
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

template <int kN, int kD>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttendParams P) {
  using Z = Sizes<kN, kD>;
  __shared__ Start start;
  __shared__ int64_t warp_sums[kJoinThreads / 32];
  wait_for_stream();
  // CTA i looks at the cut in front of the i + 1-st of the CTAs that shared the tiles
  const int at = blockIdx.x + 1;
  int64_t tile = 0;
  find_tile<kN>(P, [&](int64_t total) { return cut(total, at, P.grid); }, &start, warp_sums);
  tile = cut(start.total, at, P.grid);
  if (start.b >= P.B) return;
  const Sequence s = sequence_of<kN>(P, start.b);
  const int64_t unit = start.off / s.tiles, first = tile - (start.off - unit * s.tiles), last = first + s.tiles;
  // nothing is cut here, or an earlier cut is in this unit too
  if (tile == first || cut(start.total, at - 1, P.grid) > first) return;
  int parts = 1;
  while (at + parts - 1 < P.grid && cut(start.total, at + parts - 1, P.grid) < last) ++parts;
  const int h = static_cast<int>(unit / s.pairs), c0 = static_cast<int>(unit % s.pairs) * 2 * kN, cols = min(2 * kN, s.cols - c0);
  const int lane = threadIdx.x & 31;
  const int64_t before = static_cast<int64_t>(at) - 1;  // the CTA with the first part
  // a CTA without tiles has no part: its place is skipped
  auto part = [&](int k) { return P.parts + (2 * (before + k) + (k == 0)) * Z::kPart; };
  auto empty = [&](int k) {
    return cut(start.total, static_cast<int>(before) + k, P.grid) == cut(start.total, static_cast<int>(before) + k + 1, P.grid);
  };
  for (int c = blockIdx.y * (kJoinThreads / 32) + threadIdx.x / 32; c < cols; c += gridDim.y * (kJoinThreads / 32)) {
    float m = -INFINITY;
    for (int k = lane; k < parts; k += 32)
      if (!empty(k)) m = fmaxf(m, part(k)[2 * kN * kD + c]);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    float l = 0.f, v[kD / 32] = {};
    for (int k = 0; k < parts; ++k) {
      if (empty(k)) continue;
      const float* p = part(k);
      const float mk = p[2 * kN * kD + c], f = mk == m ? 1.f : power(mk - m);
      l += p[2 * kN * (kD + 1) + c] * f;
#pragma unroll
      for (int e = 0; e < kD / 32; ++e) v[e] += p[c * kD + lane + 32 * e] * f;
    }
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

// columns of a block: as few as hold a sequence's rows in one block, 64 at most
int block_columns(int group, int max_nodes) {
  const int64_t cols = static_cast<int64_t>(max_nodes + 1) * group;
  return cols <= 16 ? 16 : cols <= 32 ? 32 : 64;
}

template <int kN, int kD>
sv_status launch_attend(AttendParams P, const Maps& maps, int device, cudaStream_t st) {
  using Z = Sizes<kN, kD>;
  P.stages = Z::kStages;
  const int smem = Z::kFixed + Z::kStages * Z::kStageBytes;
  static std::atomic<bool> opted_in[64];
  if (device >= 64 || !opted_in[device].load()) {
    if (cudaFuncSetAttribute(attend_kernel<kN, kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return SV_ECUDA;
    if (device < 64) opted_in[device].store(true);
  }
  if (launch_waiting(attend_kernel<kN, kD>, P.grid, kAttendThreads, smem, 1, st, P, maps) != cudaSuccess) return SV_ECUDA;
  if (P.grid > 1 &&
      launch_waiting(join_kernel<kN, kD>, dim3(P.grid - 1, kN / 8), kJoinThreads, 0, 1, st, P) != cudaSuccess)
    return SV_ECUDA;
  return SV_OK;
}

template <int kD>
sv_status launch_attend(const AttendParams& P, const Maps& maps, int columns, int device, cudaStream_t st) {
  return columns == 16   ? launch_attend<16, kD>(P, maps, device, st)
         : columns == 32 ? launch_attend<32, kD>(P, maps, device, st)
                         : launch_attend<64, kD>(P, maps, device, st);
}

int sms_of(int device) {
  int sms = 0;
  return cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess ? sms : 0;
}

}  // namespace
}  // namespace sv

extern "C" size_t spec_verify_attend_workspace(int heads, int q_heads, int dim, int max_nodes, int device) {
  if (heads < 1 || q_heads < 1 || dim < 1 || max_nodes < 0 || max_nodes > SV_MAX_NODES) return 0;
  const int columns = sv::block_columns(q_heads / heads, max_nodes);
  return static_cast<size_t>(2 * sv::sms_of(device)) * 2 * columns * (dim + 2) * sizeof(float);
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
  if (B < 0 || total_nodes < 0 || max_nodes < 0) return SV_EINVAL;
  if (max_nodes > SV_MAX_NODES) return SV_EUNSUPPORTED;
  if (q_row < 0 || q_head < 0 || out_row < 0 || out_head < 0) return SV_EINVAL;
  for (const int64_t s : {q_row, q_head, out_row, out_head})
    if (s >= (int64_t{1} << 40)) return SV_EUNSUPPORTED;
  if (B == 0) return SV_OK;
  if (static_cast<int64_t>(total_nodes) + B > INT32_MAX || q_heads / cache->heads > (1 << 20)) return SV_EUNSUPPORTED;
  if (!q || !out || !context || !node_start) return SV_EINVAL;
  if (q_row % 8 || q_head % 8 || reinterpret_cast<uintptr_t>(q) % 16 || reinterpret_cast<uintptr_t>(out) % 2) return SV_EINVAL;
  for (const void* p : {static_cast<const void*>(context), static_cast<const void*>(node_start),
                        static_cast<const void*>(parent)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SV_EINVAL;
  const int rows = total_nodes + B;
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
  P.grid = sms;
  P.parts = static_cast<float*>(workspace);
  sv::Maps maps;
  if (!sv::map_entries(&maps.k, *cache, cache->k, workspace, P.box_tokens) ||
      !sv::map_entries(&maps.v, *cache, cache->v, workspace, P.box_tokens))
    return SV_ECUDA;
  const int columns = sv::block_columns(P.group, max_nodes);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return cache->dim == 128 ? sv::launch_attend<128>(P, maps, columns, device, st)
                           : sv::launch_attend<64>(P, maps, columns, device, st);
}
