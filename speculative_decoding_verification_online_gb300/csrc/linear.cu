// Grouped matrix products with an epilogue: spec_verify_linear.
//
//   y[g, m, n] = act(sum_k x[g, m, k] w[g, n, k] + bias[g, n]) + residual[g, m, n]
//
// The products run on the tensor cores (tcgen05).  Rows of x and w that start at
// multiples of 16 bytes come in by TMA.  Where one of the two does not, w still comes
// by TMA, in classes of rows that start at the same place in 16 bytes, and warps load
// x, shifted to match.
//
// What bounds it, measured on a GB300 (6.78 TB/s, 1.95 PFLOP/s bf16 measured with a
// copy and a library product):
//  * few tokens: reading w once.  M = 6, N = 151936, K = 2048: 99 us, 6.3 TB/s; five
//    heads of M = 64, N = K = 4096 with bias, SiLU and residual: 34.7 us, 5.0 TB/s
//    (one wave of tiles: its start and its end are not hidden).
//  * many tokens: the tensor cores and the power limit.  M = 2304, N = 32000, K =
//    4096: 298 us, 2.03 PFLOP/s alone, 340 to 354 us, 1.71 to 1.78, back to back;
//    M = 384, N = 128256, K = 4096 with a soft cap: 248 us, 1.62 PFLOP/s alone, 258 to
//    262 us repeated on the same inputs, 296 to 300 us, 1.36, back to back on others
//    (75 % of the cycles in products: 200 KB of stages in flight a SM do not cover what
//    w takes to come from HBM).
//  * rows at odd addresses: w's bytes where K is long (M = 77, N = 32001, K = 8001:
//    103 us, 5.0 TB/s; 83 us for K = 8000), the start and the end of a tile where it is
//    short (K = 1001: 27 us; 21 us for K = 1000; 42 us where warps load both operands).
//    M = 8, K = 2001: 28 us (66); M = 300, K = 1001: 63 us (137); M = 2304, N = 32000,
//    K = 4097: 763 us (1398), 0.79 PFLOP/s: there the loading warps' latency.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "entry.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

struct LinearParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  const void* bias;
  const void* res;
  void* y;
  int64_t x_row, x_group, w_row, w_group, b_group, r_row, r_group, y_row, y_group;
  int groups, M, N, K;
  int bias_bf16, res_bf16, y_bf16, act;
  float cap, inv_cap;
};

// An fp32 or bf16 entry as its bits; shifted up by wide(bf16) they are the fp32 value.  Several entries are loaded under
// one branch on the type: a branch for each would wait for each.
__device__ __forceinline__ uint32_t bits_f32(const void* p, int64_t i) { return static_cast<const uint32_t*>(p)[i]; }
__device__ __forceinline__ uint32_t bits_bf16(const void* p, int64_t i) { return static_cast<const uint16_t*>(p)[i]; }
__device__ __forceinline__ int wide(int bf16) { return bf16 ? 16 : 0; }

__device__ __forceinline__ float load_either(const void* p, int64_t i, int bf16) {
  return __uint_as_float((bf16 ? bits_bf16(p, i) : bits_f32(p, i)) << wide(bf16));
}

// entries i, i + step, .. of the first n of kCount, 0 behind them
template <int kCount>
__device__ __forceinline__ void load_entries(uint32_t (&r)[kCount], const void* p, int64_t i, int64_t step, int n, int bf16) {
  if (bf16) {
#pragma unroll
    for (int k = 0; k < kCount; ++k, i += step) r[k] = k < n ? bits_bf16(p, i) : 0u;
  } else {
#pragma unroll
    for (int k = 0; k < kCount; ++k, i += step) r[k] = k < n ? bits_f32(p, i) : 0u;
  }
}

// (1 + erf(z / sqrt 2)) / 2 for results of bf16.  The part beyond |z| is t p(t) exp(-z^2 / 2) with t = 1 / (1 + 0.3275911 |z| /
// sqrt 2) and a p of degree 4, off by 7.5e-8 (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26, halved), and
// by as much again with fp32's roundings.  GELU of 357 x 37248 bf16 results with bias and residual, K = 128: 33.7 us, 35.4 with
// erff.
__device__ __forceinline__ float normal_below(float z) {
  const float a = fabsf(z), t = __fdividef(1.f, fmaf(0.231641888f, a, 1.f));
  const float p = fmaf(fmaf(fmaf(fmaf(0.5307027145f, t, -0.7265760135f), t, 0.7107068705f), t, -0.142248368f), t, 0.127414796f);
  const float beyond = t * p * __expf(-0.5f * a * a);
  return z > 0.f ? 1.f - beyond : beyond;
}

// cap * tanh(z / cap) to about 8 half steps.  With x = z / cap: z times the series of tanh(x) / x below 1/4, so that z keeps
// its digits where the quotient falls below the normal floats, and cap (1 - 2 / (1 + exp 2x)) above.  Above 2^126 the
// reciprocal is below them and off by up to 2^-22.
__device__ __forceinline__ float soft_cap(float z, const LinearParams& P) {
  const float x = z * P.inv_cap, a = fabsf(x), q = a * a;
  const float low = z * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
  const float high = P.cap * (1.f - __fdividef(2.f, 1.f + __expf(2.f * a)));
  return a < 0.25f ? low : copysignf(high, z);
}

// fp32 results of GELU take erff: 0.6 to 0.7 half steps in the 2-norm for normal z, where the formula above has 1.4 to 2.1 (357 x
// 37248 fp32 results with bias and residual, K = 128: 34.3 us, 32.4 with the formula).
template <int kAct, bool kBf16>
__device__ __forceinline__ float activate(float z, const LinearParams& P) {
  if constexpr (kAct == SV_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (kAct == SV_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
  if constexpr (kAct == SV_ACT_GELU) return kBf16 ? z * normal_below(z) : 0.5f * z * (1.f + erff(z * 0.70710678f));
  // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
  if constexpr (kAct == SV_ACT_GELU_TANH) return __fdividef(z, 1.f + __expf(-1.59576912f * (z + 0.044715f * z * z * z)));
  if constexpr (kAct == SV_ACT_SOFTCAP) return soft_cap(z, P);
  return z;
}

// Runs of tokens are finished in straight code; with these activations runs of 32 are slower than runs of 16 (357 x 37248
// bf16 results, K = 128: GELU with bias and residual 39.2 -> 35.4 us, the soft cap 25.0 -> 23.4 us), the others are not
// (a residual alone: 24.6 -> 30.5 us with 16).
__host__ __device__ constexpr bool long_code(int act) {
  return act == SV_ACT_GELU || act == SV_ACT_GELU_TANH || act == SV_ACT_SOFTCAP;
}

// What a kernel is made for: sums of all of K for results of either type, or sums in segments (see below) for one type
enum Sums { kWhole = 0, kSegmentsF32 = 1, kSegmentsBf16 = 2 };

// f with the activation and y's type as constants: code that a call does not use is not fetched either
template <int kAct, int kSums, typename F>
__device__ __forceinline__ void with_type(int y_bf16, F&& f) {
  if (kSums == kSegmentsBf16 || (kSums == kWhole && y_bf16))
    f(std::integral_constant<int, kAct>(), std::bool_constant<kSums != kSegmentsF32>());
  else
    f(std::integral_constant<int, kAct>(), std::bool_constant<kSums == kSegmentsBf16>());
}

template <int kSums, typename F>
__device__ __forceinline__ void with_epilogue(int act, int y_bf16, F&& f) {
  switch (act) {
    case SV_ACT_RELU: with_type<SV_ACT_RELU, kSums>(y_bf16, f); break;
    case SV_ACT_SILU: with_type<SV_ACT_SILU, kSums>(y_bf16, f); break;
    case SV_ACT_GELU: with_type<SV_ACT_GELU, kSums>(y_bf16, f); break;
    case SV_ACT_GELU_TANH: with_type<SV_ACT_GELU_TANH, kSums>(y_bf16, f); break;
    case SV_ACT_SOFTCAP: with_type<SV_ACT_SOFTCAP, kSums>(y_bf16, f); break;
    default: with_type<SV_ACT_NONE, kSums>(y_bf16, f);
  }
}

__device__ __forceinline__ float load_bias(const LinearParams& P, int g, int64_t n) {
  return P.bias ? load_either(P.bias, g * P.b_group + n, P.bias_bf16) : 0.f;
}

__device__ __forceinline__ void prefetch_l2(const void* p, int64_t i, int bf16) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + i * (bf16 ? 2 : 4)));
}

// The sum's way out: the one rounding to bf16, where y is bf16, is the last step.
template <int kAct, bool kBf16>
__device__ __forceinline__ void finish_value(const LinearParams& P, int64_t at, float z, float bias, float res) {
  z = activate<kAct, kBf16>(z + bias, P) + res;
  if constexpr (kBf16)
    static_cast<__nv_bfloat16*>(P.y)[at] = __float2bfloat16(z);
  else
    static_cast<float*>(P.y)[at] = z;
}

// ------------------------------------------------------------ tensor cores
//
// Persistent CTAs, one per SM, each (or each pair) taking every n-th tile of y.  Warp 0
// fetches tiles of both operands by TMA into a ring of stages, 64 entries of
// K at a time (rows of 128 bytes, 128-byte swizzle), or warps 10 to 25 load x's;
// warp 1 multiplies them into tensor memory, 128 rows of one operand (A) by nt rows
// of the other (B); warps 2 to 9 take the sums out and finish them while the next
// tile is multiplied into the other half of the accumulators.
//
// Which operand is A:
//  * M > 128: w, 256 rows of it by a pair of CTAs (a cluster of two, on one
//    pair of SMs): each holds 128 rows of A and half the rows of B, and one
//    product instruction of the first CTA works on both.  A lane of tensor
//    memory is one n, so a warp's 32 lanes write 32 neighbours of y for each m,
//    straight from registers.
//  * M <= 128, or rows at odd addresses (128 tokens at a time): x.  The call is bound by reading w, and the width of a tile of
//    w is then free (any multiple of 16 up to 256), so that the tiles come out
//    even over the SMs.  Lanes are tokens here; sums pass through shared memory
//    so that neighbouring threads finish neighbouring n, however few tokens
//    there are.  Only the rows of x that exist are fetched: a product row that
//    belongs to no token multiplies whatever lies behind them in shared memory
//    and is never read.
//
// The tensor core cuts its sums off after each step of 16 entries of K, towards
// zero: after K = 2048 a sum is 2.1e-6 short, about in proportion to K.  (Sums of
// one sign: 1e-7 for each step, 6.3e-3 after K = 2^20.)  For fp32 results of K > 768
// and bf16 results of K > 32768 (kSegments) a sum is carried through the tensor core
// for at most 768 entries: two segments in the two accumulators where that is
// enough, added when a tile is finished; else segments of 512, which the epilogue's
// warps add up in tensor memory beside the two accumulators (for which a tile is
// then 160 wide at most).  bf16 results of shorter K are at most 2e-4 short, a
// twentieth of their own rounding, and few of them land on another bf16 value than
// an exact sum's (at K = 4096 1.4e-4 in the 2-norm; either kind is 1.66e-3 from the
// exact results).  So no wait for a sum is longer than 512 blocks of K, far below
// the limit at which waits give up.

constexpr int kMmaK = 64;        // entries of K a stage holds of each row: 128 bytes
constexpr int kRowBytes = 128;
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 8;
// Warps that load a stage of x together; groups of them, by turns.  Four groups of four against two of eight and two of
// four: M = 77, N = 32001, K = 2001 56, 59 and 69 us; M = 1000, N = 8001, K = 4097 178, 187 and 207 us; M = 8, N = 32001,
// K = 2001 33, 32 and 31 us.
constexpr int kLoadWarps = 4, kLoadGroups = 4;
constexpr int kMmaThreads = 32 * (2 + kEpiWarps);
constexpr int kStageCols = 64;   // columns of a tile that pass through shared memory at a time where x is A
constexpr int kMmaSmem = 226 * 1024;
constexpr int kLongF32 = 768, kLongBf16 = 32768;  // the longest K without segments

struct MmaParams {
  LinearParams L;
  int nt;                // rows of B in a tile
  int ra;                // rows of A that are fetched
  int stages, tmem_cols;
  int tiles_a, tiles_b;
  int sub;               // blocks of 64 entries of K in a stage
  int kblocks;           // stages that K takes
  int seg_blocks, segs;  // stages of a segment, segments
  int halves;            // two segments, which stay in their accumulators until the tile is finished
  int a_groups, b_groups;  // 0: the operand is shared by all groups
  unsigned tiles;
  unsigned idesc;
  int at_once;           // a tile's columns pass through shared memory at once, not kStageCols at a time
  unsigned staging;      // where the epilogue's staging starts in dynamic shared memory
  // where warps load x (see below)
  int w_mapped;          // 1: w comes by TMA, 0: the warps load it too
  int every, classes;    // so many rows of w are between two of a class; classes that have rows
  int group_classes;     // the same of groups
};

template <int kMaps>
struct Maps {
  CUtensorMap m[kMaps];
};
constexpr int kMostMaps = 64;  // eight classes of rows times eight of groups

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  unsigned e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_in(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// into this CTA's memory, its bytes counted by the barrier of the pair's first CTA
__device__ __forceinline__ void tma_load_pair(const CUtensorMap* map, uint32_t dst, uint32_t bar, int k, int row, int g) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(k), "r"(row), "r"(g)
      : "memory");
}

__device__ __forceinline__ void tma_load(const CUtensorMap* map, uint32_t dst, uint64_t* bar, int k, int row, int g) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(smem_addr(bar)), "r"(k), "r"(row), "r"(g)
      : "memory");
}

// rows of 128 bytes in groups of 8 (1024 bytes), 128-byte swizzle, K innermost
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

template <bool kPair>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, unsigned idesc, bool add) {
  if constexpr (kPair)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned>(add))
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned>(add))
        : "memory");
}

// an arrival at `bar` (of both CTAs of a pair) once the products issued so far are done
template <bool kPair>
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// kCols (16 or 32) columns of this warp's 32 lanes
template <int kCols>
__device__ __forceinline__ void tc_load(uint32_t addr, uint32_t (&r)[kCols]) {
#pragma unroll
  for (int c = 0; c < kCols; c += 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[c]), "=r"(r[c + 1]), "=r"(r[c + 2]), "=r"(r[c + 3]), "=r"(r[c + 4]), "=r"(r[c + 5]), "=r"(r[c + 6]),
          "=r"(r[c + 7]), "=r"(r[c + 8]), "=r"(r[c + 9]), "=r"(r[c + 10]), "=r"(r[c + 11]), "=r"(r[c + 12]),
          "=r"(r[c + 13]), "=r"(r[c + 14]), "=r"(r[c + 15])
        : "r"(addr + c)
        : "memory");
  // the registers pass through the wait, so that nothing reads them in front of it
#pragma unroll
  for (int c = 0; c < kCols; c += 16)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[c]), "+r"(r[c + 1]), "+r"(r[c + 2]), "+r"(r[c + 3]), "+r"(r[c + 4]), "+r"(r[c + 5]),
                   "+r"(r[c + 6]), "+r"(r[c + 7]), "+r"(r[c + 8]), "+r"(r[c + 9]), "+r"(r[c + 10]), "+r"(r[c + 11]),
                   "+r"(r[c + 12]), "+r"(r[c + 13]), "+r"(r[c + 14]), "+r"(r[c + 15])
                 :
                 : "memory");
}

// 16 columns back into tensor memory
__device__ __forceinline__ void tc_store(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

struct TileAt {
  int ta, tb, g, cls;
};

// Where warps load x, the tokens' tiles follow one another (they share w's), then the classes (they share y's sectors).
template <bool kLoad>
__device__ __forceinline__ TileAt tile_at(const MmaParams& P, unsigned t) {
  if constexpr (kLoad) {
    const unsigned ta = t % P.tiles_a, u = t / P.tiles_a, cls = u % P.classes, v = u / P.classes;
    return {static_cast<int>(ta), static_cast<int>(v % P.tiles_b), static_cast<int>(v / P.tiles_b), static_cast<int>(cls)};
  }
  const unsigned tb = t % P.tiles_b, rest = t / P.tiles_b;
  return {static_cast<int>(rest % P.tiles_a), static_cast<int>(tb), static_cast<int>(rest / P.tiles_a), 0};
}

// ---- rows at odd addresses
//
// TMA wants rows that start at multiples of 16 bytes.  If rows of w are s entries
// apart, every 8 / gcd(8, s)-th row starts at the same place in 16 bytes: those rows
// are a class, a matrix of its own, which has a map that begins at the multiple of 16
// bytes in front of its first row.  In the map a row stands `behind` (0 to 7) entries
// from its start; a sum over K does not mind if x's rows are moved behind by as much.
// A tile of y takes columns of one class; the classes of the same columns follow one
// another, so that the parts of a sector of y meet in L2.  What a map shows in front
// of a row belongs to another row, or to nobody (and may be a NaN, which a zero of x
// would not take out of a sum): the loading warps put zeros there, in the first stage
// of a tile (M = 77, N = 32001, K = 1001 29 us; 30 us with that stage of w loaded by
// the warps).  Behind a row's end the map has zeros.
// Groups of w that are not multiples of 16 bytes apart are classes in the same way.
//
// eight entries, zeros in place of the first 1 to 7
__device__ __forceinline__ uint4 without_front(uint4 e, int n) {
  e.x &= n > 1 ? 0u : 0xffff0000u;
  e.y &= n > 3 ? 0u : n > 2 ? 0xffff0000u : ~0u;
  e.z &= n > 5 ? 0u : n > 4 ? 0xffff0000u : ~0u;
  e.w &= n > 6 ? 0xffff0000u : ~0u;
  return e;
}

// Eight entries of a row from any address that bf16 entries have lie in one or two aligned blocks of 16 bytes.  Only blocks
// with an entry of the row are read: an allocation has all of such a block.
__device__ __forceinline__ uint4 load_if(const char* p, bool there) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n"
      " mov.u32 %3, 0;\n @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(static_cast<unsigned>(there))
      : "memory");
  return v;
}

// The entries from `shift` bytes into the blocks a and b on; zeros in place of those in front of `front` and from `valid` on.
__device__ __forceinline__ uint4 entries_of(const uint4& a, const uint4& b, int shift, int front, int valid) {
  const bool two = shift & 8, one = shift & 4;
  const uint32_t w0 = two ? a.z : a.x, w1 = two ? a.w : a.y, w2 = two ? b.x : a.z, w3 = two ? b.y : a.w,
                 w4 = two ? b.z : b.x, w5 = two ? b.w : b.y;
  const uint32_t v0 = one ? w1 : w0, v1 = one ? w2 : w1, v2 = one ? w3 : w2, v3 = one ? w4 : w3, v4 = one ? w5 : w4;
  const int bits = (shift & 2) * 8;
  uint4 r = make_uint4(__funnelshift_r(v0, v1, bits), __funnelshift_r(v1, v2, bits), __funnelshift_r(v2, v3, bits),
                       __funnelshift_r(v3, v4, bits));
  if (valid < 8) {
    r.x &= valid > 1 ? ~0u : valid > 0 ? 0xffffu : 0u;
    r.y &= valid > 3 ? ~0u : valid > 2 ? 0xffffu : 0u;
    r.z &= valid > 5 ? ~0u : valid > 4 ? 0xffffu : 0u;
    r.w &= valid > 7 ? ~0u : valid > 6 ? 0xffffu : 0u;
  }
  return front > 0 ? without_front(r, front) : r;
}

// A warp's share (warp `mine` of the loading ones) of `rows` rows of 64 entries from k on, as TMA would lay them down: 16
// bytes a lane, eight lanes a row.  p is where an entry 0 of the first row would be; entries in front of `lo` and from `hi`
// on are zeros, and so are rows from `there` on.  A lane's rows are kStep apart, a multiple of 8: they all start at the
// same place in 16 bytes.
__device__ __forceinline__ void load_rows(uint32_t dst, const __nv_bfloat16* p, int64_t stride, int rows, int64_t there,
                                          int k, int lo, int hi, int mine) {
  constexpr int kBatch = 4, kStep = 4 * kLoadWarps;
  static_assert(kStep % 8 == 0);
  const int lane = threadIdx.x & 31, c = lane % 8;
  const int front = max(0, lo - k - 8 * c), valid = max(0, min(8, hi - k - 8 * c));
  int r = 4 * mine + lane / 8;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p + r * stride + k + 8 * c);
  const int shift = static_cast<int>(at & 15);
  const char* block = reinterpret_cast<const char*>(at & ~uintptr_t{15});
  const int64_t step = kStep * 2 * stride;
  const bool in_a = valid > front && shift + 2 * front < 16, in_b = valid > front && shift + 2 * valid > 16;
  const int last = static_cast<int>(min(static_cast<int64_t>(rows), there));
  dst += r * kRowBytes + ((c ^ (r & 7)) << 4);
  for (; r < rows; r += kBatch * kStep, dst += kBatch * kStep * kRowBytes) {
    uint4 a[kBatch], b[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i, block += step) {
      a[i] = load_if(block, in_a && r + i * kStep < last);
      b[i] = load_if(block + 16, in_b && r + i * kStep < last);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const uint4 e = entries_of(a[i], b[i], shift, front, valid);
      if (r + i * kStep < rows)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + i * kStep * kRowBytes), "r"(e.x), "r"(e.y),
                     "r"(e.z), "r"(e.w)
                     : "memory");
    }
  }
}

// zeros in place of the first `n` (below 8) entries of row r
__device__ __forceinline__ void clear_front(uint32_t rows, int r, int n) {
  const uint32_t at = rows + r * kRowBytes + ((r & 7) << 4);
  uint4 e;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(e.x), "=r"(e.y), "=r"(e.z), "=r"(e.w)
               : "r"(at)
               : "memory");
  e = without_front(e, n);
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(e.x), "r"(e.y), "r"(e.z), "r"(e.w) : "memory");
}

// the first row of w of a tile, and how many entries it starts behind a multiple of 16 bytes
__device__ __forceinline__ const __nv_bfloat16* first_row(const MmaParams& P, const TileAt& at, int* behind) {
  const int64_t n = at.cls + static_cast<int64_t>(at.tb) * P.nt * P.every;
  const __nv_bfloat16* p = P.L.w + at.g * P.L.w_group + n * P.L.w_row;
  *behind = P.w_mapped ? static_cast<int>(reinterpret_cast<uintptr_t>(p) / 2 % 8) : 0;
  return p;
}

// kWeightsA: w is A, and the CTAs work in pairs.  kSums, kSegments: see above.  kLoad: rows at odd addresses.
template <bool kWeightsA, bool kLoad, int kSums>
__global__ void __launch_bounds__(kMmaThreads + (kLoad ? 32 * kLoadGroups * kLoadWarps : 0), 1)
    mma_kernel(const __grid_constant__ MmaParams P, const __grid_constant__ Maps<kLoad ? kMostMaps : 2> maps) {
  static_assert(!(kWeightsA && kLoad));
  constexpr bool kPair = kWeightsA, kSegments = kSums != kWhole;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
  __shared__ uint64_t fronts[kLoad ? kMaxStages : 1];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int dead;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned rank = kPair ? cluster_rank() : 0;
  const unsigned first = kPair ? blockIdx.x / 2 : blockIdx.x, step = kPair ? gridDim.x / 2 : gridDim.x;
  const int b_rows = kPair ? P.nt / 2 : P.nt;  // of B in this CTA
  const uint32_t base = (smem_addr(smem) + 1023) & ~1023u;
  const uint32_t a_bytes = P.ra * kRowBytes, sub_bytes = a_bytes + b_rows * kRowBytes, stage_bytes = P.sub * sub_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) mbar_init(&full[s], kLoad ? kLoadWarps + P.w_mapped : 1), mbar_init(&empty[s], 1);
    for (int s = 0; kLoad && s < P.stages; ++s) mbar_init(&fronts[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&acc_full[s], 1), mbar_init(&acc_empty[s], kPair ? 2 * kEpiWarps : kEpiWarps);
    mbar_init(&drained, 1);
    dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if constexpr (!kLoad) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.m[0]));
      asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.m[1]));
    }
  }
  if (warp == 1) {
    if constexpr (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)),
                   "r"(P.tmem_cols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)),
                   "r"(P.tmem_cols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (kPair) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  wait_for_stream();

  // Warps 0 and 1 go through their loops as whole warps, and one lane that elect
  // picks issues: with a branch on the lane instead the compiler takes the
  // operands for different in every lane, and an issue costs several times as much.
  if (kLoad && warp >= 2 + kEpiWarps) {
    // Groups of warps fill the stages by turns, so that the loads of one are on their way while others store.  (More
    // groups than stages could come to a stage two phases early, and a parity does not tell two phases from none.)
    const int mine = (warp - 2 - kEpiWarps) % kLoadWarps, group = (warp - 2 - kEpiWarps) / kLoadWarps;
    int turn = 0;
    unsigned s = 0, phase = 1, fronts_phase = 0;  // of each stage a bit
    for (unsigned t = first; t < P.tiles && !dead; t += step) {
      const TileAt at = tile_at<kLoad>(P, t);
      int behind;
      const __nv_bfloat16* w = first_row(P, at, &behind) - behind;
      const int64_t m0 = static_cast<int64_t>(at.ta) * 128;
      const __nv_bfloat16* x = P.L.x + at.g * P.L.x_group + m0 * P.L.x_row - behind;
      const int64_t w_rows = (P.L.N - at.cls + P.every - 1) / P.every - static_cast<int64_t>(at.tb) * P.nt;
      for (int kb = 0; kb < P.kblocks; ++kb) {
        if (turn == group) {
          if (!mbar_wait(&empty[s], phase, &dead)) break;
          const uint32_t dst = base + s * stage_bytes;
          load_rows(dst, x, P.L.x_row, P.ra, P.L.M - m0, kb * kMmaK, behind, behind + P.L.K, mine);
          if (!P.w_mapped) {
            load_rows(dst + a_bytes, w, P.every * P.L.w_row, P.nt, w_rows, kb * kMmaK, 0, P.L.K, mine);
          } else if (kb == 0 && behind > 0) {
            if (!mbar_wait(&fronts[s], fronts_phase >> s & 1, &dead)) break;
            for (int r = 32 * mine + lane; r < P.nt; r += 32 * kLoadWarps) clear_front(dst + a_bytes, r, behind);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
        }
        if (kb == 0 && behind > 0) fronts_phase ^= 1u << s;
        if (++turn == kLoadGroups) turn = 0;
        if (++s == static_cast<unsigned>(P.stages)) s = 0, phase ^= 1;
      }
    }
  } else if (kLoad && warp == 0) {
    // w's share of the stages; where it shows entries in front of w's rows, the loading warps wait for it
    unsigned s = 0, phase = 1, fill = 0;
    for (unsigned t = P.w_mapped ? first : P.tiles; t < P.tiles && !dead; t += step) {
      const TileAt at = tile_at<kLoad>(P, t);
      int behind;
      first_row(P, at, &behind);
      const CUtensorMap* map = &maps.m[at.g % P.group_classes * P.classes + at.cls];
      const int row = at.tb * P.nt, g = P.b_groups ? at.g / P.group_classes : 0;
      for (int kb = 0; kb < P.kblocks; ++kb) {
        if (!mbar_wait(&empty[s], phase, &dead)) break;
        if (elect_one()) {
          uint64_t* bar = kb == 0 && behind > 0 ? &fronts[s] : &full[s];
          if (bar != &full[s]) mbar_arrive(&full[s]);
          mbar_expect(bar, stage_bytes - a_bytes);
          tma_load(map, base + s * stage_bytes + a_bytes, bar, kb * kMmaK, row, g);
        }
        __syncwarp();
        ++fill;
        if (++s == static_cast<unsigned>(P.stages)) s = 0, phase ^= 1;
      }
    }
    if (dead) {
      int gave_up = 0;
      for (unsigned f = fill > static_cast<unsigned>(P.stages) ? fill - P.stages : 0; f < fill; ++f)
        mbar_wait(&full[f % P.stages], (f / P.stages) & 1, &gave_up);
    }
  } else if (warp == 0) {
    // stage and phase go round by counting: a division by the number of stages
    // costs more than everything else that a stage needs
    unsigned s = 0, phase = 1, fill = 0;
    const uint32_t leader = kPair ? in_cta(full, 0) : 0;
    for (unsigned t = first; t < P.tiles && !dead; t += step) {
      const TileAt at = tile_at<kLoad>(P, t);
      const int ga = P.a_groups ? at.g : 0, gb = P.b_groups ? at.g : 0;
      const int row_a = kPair ? at.ta * 256 + static_cast<int>(rank) * 128 : 0;
      const int row_b = at.tb * P.nt + (kPair ? static_cast<int>(rank) * b_rows : 0);
      for (int kb = 0, k = 0; kb < P.kblocks; ++kb, k += P.sub * kMmaK) {
        if (!mbar_wait(&empty[s], phase, &dead)) break;
        if (elect_one()) {
          uint32_t dst = base + s * stage_bytes;
          if constexpr (kPair) {
            const uint32_t bar = leader + s * 8;
            if (rank == 0) mbar_expect(&full[s], 2 * stage_bytes);
            for (int u = 0; u < P.sub; ++u, dst += sub_bytes) {
              tma_load_pair(&maps.m[0], dst, bar, k + u * kMmaK, row_a, ga);
              tma_load_pair(&maps.m[1], dst + a_bytes, bar, k + u * kMmaK, row_b, gb);
            }
          } else {
            mbar_expect(&full[s], stage_bytes);
            for (int u = 0; u < P.sub; ++u, dst += sub_bytes) {
              tma_load(&maps.m[0], dst, &full[s], k + u * kMmaK, 0, ga);
              tma_load(&maps.m[1], dst + a_bytes, &full[s], k + u * kMmaK, row_b, gb);
            }
          }
        }
        __syncwarp();
        ++fill;
        if (++s == static_cast<unsigned>(P.stages)) s = 0, phase ^= 1;
      }
    }
    if (dead && rank == 0) {
      // copies still in flight land before the CTA's memory goes
      int gave_up = 0;
      for (unsigned f = fill > static_cast<unsigned>(P.stages) ? fill - P.stages : 0; f < fill; ++f)
        mbar_wait(&full[f % P.stages], (f / P.stages) & 1, &gave_up);
    }
  } else if (warp == 1) {
    if (rank == 0 && P.kblocks > 0) {
      unsigned s = 0, phase = 0, n = 0;
      const uint64_t desc_a = smem_desc(base), desc_b = smem_desc(base + a_bytes);
      const unsigned desc_step = stage_bytes / 16;
      for (unsigned t = first; t < P.tiles && !dead; t += step) {
        for (int kb0 = 0; kb0 < P.kblocks && !dead; kb0 += P.seg_blocks, ++n) {
          const unsigned buf = n & 1;
          if (!mbar_wait(&acc_empty[buf], ((n >> 1) & 1) ^ 1, &dead)) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t d = tmem + buf * P.nt;
          const int end = kSegments ? min(P.kblocks, kb0 + P.seg_blocks) : P.kblocks;
          for (int kb = kb0; kb < end; ++kb) {
            if (!mbar_wait(&full[s], phase, &dead)) break;
            // What warps stored is now seen here; the tensor core reads it by another way.  The fence stands here because
            // in a loading warp it would wait for the loads on their way.
            if constexpr (kLoad) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (elect_one()) {
              uint64_t da = desc_a + s * desc_step, db = desc_b + s * desc_step;
              for (int u = 0; u < P.sub; ++u, da += sub_bytes / 16, db += sub_bytes / 16) {
                tc_mma<kPair>(d, da, db, P.idesc, kb > kb0 || u > 0);
#pragma unroll
                for (int k = 1; k < kMmaK / 16; ++k) tc_mma<kPair>(d, da + 2 * k, db + 2 * k, P.idesc, true);
              }
              tc_commit<kPair>(&empty[s]);
              if (kb == end - 1) tc_commit<kPair>(&acc_full[buf]);
            }
            __syncwarp();
            if (++s == static_cast<unsigned>(P.stages)) s = 0, phase ^= 1;
          }
        }
      }
      if (dead) {
        int gave_up = 0;
        if (elect_one()) tc_commit<kPair>(&drained);
        __syncwarp();
        mbar_wait(&drained, 0, &gave_up);
      }
    }
  } else {
    const int ew = warp - 2, quad = warp & 3, half = ew >> 2;
    const int et = threadIdx.x - 64;
    float* staging = reinterpret_cast<float*>(smem + P.staging);
    unsigned n = 0;
    auto sum = [&](bool ok, float v) { return !ok ? NAN : P.kblocks == 0 ? 0.f : v; };  // no entries: no product ran
    // columns of a tile that go together to one of the two warps of 32 lanes
    constexpr int kCols = kWeightsA && kSegments ? 16 : 32;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16), carried = lanes + 2 * P.nt;
    const bool idle = !kWeightsA && !kLoad && quad * 32 >= P.L.M;  // no token in these lanes
    auto wait_sums = [&]() {
      const bool ok = !dead && (P.kblocks == 0 || mbar_wait(&acc_full[n & 1], (n >> 1) & 1, &dead));
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      return ok;
    };
    auto release = [&](unsigned buf) {
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair)
          mbar_arrive_in(in_cta(&acc_empty[buf], 0));
        else
          mbar_arrive(&acc_empty[buf]);
      }
    };
    // 16 columns' sums: the last segment's and what the others have carried
    auto sums16 = [&](int c, uint32_t (&v)[16], bool add) {
      tc_load<16>(lanes + (n & 1) * P.nt + c, v);
      if (!add) return;
      uint32_t w[16];
      tc_load<16>((kSegments && P.halves ? lanes + (~n & 1) * P.nt : carried) + c, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
    };
    auto carry = [&]() {
      for (int seg = 0; seg + 1 < P.segs; ++seg, ++n) {
        if (wait_sums() && !idle && !P.halves) {
          __syncwarp();
#pragma unroll 1
          for (int c0 = half * kCols; c0 < P.nt; c0 += 2 * kCols)
#pragma unroll 1
            for (int c = c0; c < min(c0 + kCols, P.nt); c += 16) {
              uint32_t v[16];
              sums16(c, v, seg > 0);
              tc_store(carried + c, v);
            }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        if (!P.halves) release(n & 1);
      }
    };
    for (unsigned t = first; t < P.tiles; t += step) {
      const TileAt at = tile_at<kLoad>(P, t);
      if constexpr (kWeightsA) {
        const int64_t col = static_cast<int64_t>(at.ta) * 256 + rank * 128 + quad * 32 + lane;
        const bool in = col < P.L.N;
        const float bias = in ? load_bias(P.L, at.g, col) : 0.f;
        // 32 tokens at a time (16 where registers are few), the next ones' residuals on their way meanwhile.  nt is a
        // multiple of 16: where a last 16 of 32 columns is not the tile's, it is read (the allocation has it) and not
        // used.
        const int64_t m_tile = static_cast<int64_t>(at.tb) * P.nt;
        const int rows_here = in ? static_cast<int>(min(static_cast<int64_t>(P.nt), P.L.M - m_tile)) : 0;
        const int shift = wide(P.L.res_bf16);
        if constexpr (kSegments) carry();
        with_epilogue<kSums>(P.L.act, P.L.y_bf16, [&](auto act, auto y_bf16) {
          constexpr int kRun = long_code(act.value) ? 16 : kCols;
          uint32_t r_next[kRun] = {};
          auto residuals = [&](int c) {
            if (P.L.res)
              load_entries(r_next, P.L.res, at.g * P.L.r_group + (m_tile + c) * P.L.r_row + col, P.L.r_row, rows_here - c,
                           P.L.res_bf16);
          };
          residuals(half * kRun);
          const bool ok = wait_sums();
#pragma unroll 1
          for (int c = half * kRun; c < P.nt; c += 2 * kRun) {
            uint32_t v[kRun], r[kRun];
            __syncwarp();
            if constexpr (kSegments)
              sums16(c, v, P.segs > 1);
            else
              tc_load<kRun>(lanes + (n & 1) * P.nt + c, v);
#pragma unroll
            for (int i = 0; i < kRun; ++i) r[i] = r_next[i];
            residuals(c + 2 * kRun);
            int64_t to = at.g * P.L.y_group + (m_tile + c) * P.L.y_row + col;
            auto finish = [&](int i) {
              finish_value<act.value, y_bf16.value>(P.L, to, sum(ok, __uint_as_float(v[i])), bias,
                                                    __uint_as_float(r[i] << shift));
            };
            if (__all_sync(~0u, c + kRun <= rows_here)) {
#pragma unroll
              for (int i = 0; i < kRun; ++i, to += P.L.y_row) finish(i);
            } else {
#pragma unroll
              for (int i = 0; i < kRun; ++i, to += P.L.y_row)
                if (c + i < rows_here) finish(i);
            }
          }
        });
      } else {
        const int every = kLoad ? P.every : 1;
        const int64_t j0 = static_cast<int64_t>(at.tb) * P.nt, n0 = at.cls + j0 * every;
        const int64_t m_tile = kLoad ? at.ta * int64_t{128} : 0;
        const int cols = static_cast<int>(min(static_cast<int64_t>(P.nt), (P.L.N - at.cls + every - 1) / every - j0));
        const int tokens = kLoad ? static_cast<int>(min(int64_t{128}, P.L.M - m_tile)) : P.L.M;
        const int64_t y0 = at.g * P.L.y_group + m_tile * P.L.y_row + n0;
        const int64_t r_from = at.g * P.L.r_group + m_tile * P.L.r_row + n0;
        // Sums come kWidth columns at a time, and each thread finishes one column of every kRows-th token, kBatch of them at
        // a time.  Biases and residuals are asked into L2 while the products run; the first ones are in registers before the
        // sums come, and each chunk's before the chunk in front of it is finished.
        //  * Few tokens and tiles wide enough for all threads: a whole tile at once, without the barriers between chunks (M =
        //    5, N = 232072, K = 184 26.8 -> 22 us; M = 32, K = 192 with bias, GELU and residual 65 -> 49 us).
        //  * Residuals: sixteen at a time, to have them on their way (eight where sixteen would not stay in registers: 2
        //    groups of M = 77, N = 32001, K = 1001 in fp32, 70 -> 63 us).
        //  * Else four at a time where that is faster, in a quarter of the code (M = 5, N = 232072, K = 184 33.3 -> 26.8 us;
        //    with M = 128 52.6 us by sixteen, 56.2 by four).
        if (et % kStageCols * every % 16 == 0)
          for (int c0 = et % kStageCols; c0 < cols; c0 += kStageCols) {
            if (P.L.bias && et < kStageCols)
              prefetch_l2(P.L.bias, at.g * P.L.b_group + n0 + c0 * every, P.L.bias_bf16);
            for (int m = et / kStageCols; P.L.res && m < tokens; m += kEpiWarps * 32 / kStageCols)
              prefetch_l2(P.L.res, r_from + m * P.L.r_row + c0 * every, P.L.res_bf16);
          }
        if constexpr (kSegments) carry();
        bool ok = true;
        if (kLoad && cols <= 0) wait_sums();  // the last tile of a class with a row less
        auto finish_tile = [&](auto act, auto y_bf16, auto width, auto batch) {
          constexpr int kWidth = width.value, kRows = kEpiWarps * 32 / kWidth, kBatch = batch.value;
          const int c = et % kWidth, row = et / kWidth;
          uint32_t r[kBatch] = {}, r_next[kBatch] = {};
          float bias, bias_next = 0.f;
          const int shift = wide(P.L.res_bf16);
          auto residuals = [&](uint32_t (&to)[kBatch], int c0, int m0) {
            if (P.L.res)
              load_entries(to, P.L.res, r_from + m0 * P.L.r_row + (c0 + c) * every, kRows * P.L.r_row,
                           c0 + c < cols ? (tokens - m0 + kRows - 1) / kRows : 0, P.L.res_bf16);
          };
          auto biases = [&](int c0) { return c0 + c < cols ? load_bias(P.L, at.g, n0 + (c0 + c) * every) : 0.f; };
          residuals(r_next, 0, row);
          bias_next = biases(0);
#pragma unroll 1
          for (int c0 = 0; c0 < cols; c0 += kWidth) {
            const int rows = c0 + c < cols ? tokens : 0;
            if (c0 == 0) ok = wait_sums();
            if (!idle)
#pragma unroll 1
              for (int cc = c0 + half * (kWidth / 2); cc < min(c0 + (half + 1) * (kWidth / 2), P.nt); cc += 16) {
                uint32_t v[16];
                __syncwarp();
                sums16(cc, v, kSegments && P.segs > 1);
                if (quad * 32 + lane < tokens)
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    staging[(quad * 32 + lane) * (kWidth + 1) + cc - c0 + i] = sum(ok, __uint_as_float(v[i]));
              }
            asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
            bias = bias_next;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) r[i] = r_next[i];
            if (c0 + kWidth < cols) {
              residuals(r_next, c0 + kWidth, row);
              bias_next = biases(c0 + kWidth);
            }
#pragma unroll 1
            for (int m0 = row; m0 < tokens; m0 += kBatch * kRows) {
              if (m0 != row) residuals(r, c0, m0);
              float v[kBatch];
#pragma unroll
              for (int i = 0; i < kBatch; ++i)
                v[i] = m0 + i * kRows < rows ? staging[(m0 + i * kRows) * (kWidth + 1) + c] : 0.f;
              int64_t to = y0 + m0 * P.L.y_row + (c0 + c) * every;
#pragma unroll
              for (int i = 0; i < kBatch; ++i, to += kRows * P.L.y_row)
                if (m0 + i * kRows < rows)
                  finish_value<act.value, y_bf16.value>(P.L, to, v[i], bias, __uint_as_float(r[i] << shift));
            }
            asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
          }
        };
        with_epilogue<kSums>(P.L.act, P.L.y_bf16, [&](auto act, auto y_bf16) {
          using Chunk = std::integral_constant<int, kStageCols>;
          using Tile = std::integral_constant<int, kEpiWarps * 32>;
          using Four = std::integral_constant<int, 4>;
          using Eight = std::integral_constant<int, 8>;
          using Most = std::integral_constant<int, kLoad && kSegments ? 8 : 16>;
          if (P.at_once && (tokens <= 4 || !P.L.res))
            finish_tile(act, y_bf16, Tile(), Four());
          else if (P.at_once)
            finish_tile(act, y_bf16, Tile(), Eight());
          else if (tokens <= 16 || (!P.L.res && (kLoad || tokens <= 32)))
            finish_tile(act, y_bf16, Chunk(), Four());
          else
            finish_tile(act, y_bf16, Chunk(), Most());
        });
      }
      if (kSegments && P.halves) release(~n & 1);
      release(n & 1);
      ++n;
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (kPair) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  __syncwarp();
  if (warp == 1) {
    if constexpr (kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols) : "memory");
  }
}

// ------------------------------------------------------------ host

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

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

// A map of [groups, rows, K] bf16 entries in boxes of box_rows x kMmaK, where
// TMA can address it: the base and the strides multiples of 16 bytes.  *grouped:
// whether the groups are a dimension of it (a shared operand has one).
bool make_map(CUtensorMap* map, const void* base, int64_t K, int64_t rows, int64_t groups, int64_t row_stride,
              int64_t group_stride, int box_rows, int* grouped) {
  const EncodeTiled encode = encode_tiled();
  if (!encode || reinterpret_cast<uintptr_t>(base) % 16) return false;
  const cuuint64_t any = static_cast<cuuint64_t>((K * 2 + 15) / 16 * 16);
  if (rows > 1 && (row_stride == 0 || row_stride % 8)) return false;
  *grouped = groups > 1 && group_stride > 0;
  if (*grouped && group_stride % 8) return false;
  if (row_stride >= (int64_t{1} << 38) || group_stride >= (int64_t{1} << 38)) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(*grouped ? groups : 1)};
  const cuuint64_t strides[2] = {rows > 1 ? static_cast<cuuint64_t>(row_stride) * 2 : any,
                                 *grouped ? static_cast<cuuint64_t>(group_stride) * 2 : any};
  const cuuint32_t box[3] = {kMmaK, static_cast<cuuint32_t>(box_rows), 1}, step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The width of a tile: the one with the least time by this estimate.  A stage
// (64 entries of K) of 128 x nt products takes 2 nt cycles of an SM's tensor
// core, and the rows of 128 bytes that the SM fetches for it come in at about 46
// bytes a cycle; the SMs (or pairs of them) take their tiles in waves, and each
// wave pays for starting and ending.
int choose_width(bool pair, int most, int64_t rows_b, int64_t tiles_a, int rows_a, int64_t groups, int64_t kblocks,
                 int workers) {
  int best = 16;
  double least = 1e300;
  for (int nt = 16; nt <= most; nt += 16) {
    const int64_t tiles = (rows_b + nt - 1) / nt * tiles_a * groups;
    const int64_t waves = (tiles + workers - 1) / workers;
    const double stage = std::max(2.0 * nt, (rows_a + (pair ? nt / 2 : nt)) * 128 / 46.0);
    const double t = waves * (kblocks * stage + 1500.0);
    if (t < least * 0.999) least = t, best = nt;
  }
  return best;
}

// Maps of w's classes of rows for a tile of P.nt of them; false where its rows cannot be had so.
bool map_classes(MmaParams* P, Maps<kMostMaps>* maps) {
  const LinearParams& L = P->L;
  for (int gc = 0; gc < P->group_classes; ++gc)
    for (int c = 0; c < P->classes; ++c) {
      const __nv_bfloat16* p = L.w + gc * L.w_group + c * L.w_row;
      const int behind = static_cast<int>(reinterpret_cast<uintptr_t>(p) / 2 % 8);
      int grouped;
      if (!make_map(&maps->m[gc * P->classes + c], p - behind, L.K + behind, (L.N - c + P->every - 1) / P->every,
                    L.w_group > 0 ? (L.groups - gc + P->group_classes - 1) / P->group_classes : 1, P->every * L.w_row,
                    P->group_classes * L.w_group, P->nt, &grouped))
        return false;
    }
  return true;
}

// how many steps of `stride` entries come back to the same place in 16 bytes
int period(int64_t stride) { return stride % 8 == 0 ? 1 : stride % 4 == 0 ? 2 : stride % 2 == 0 ? 4 : 8; }

template <bool kWeightsA, bool kLoad, int kSums>
sv_status launch_mma(const LinearParams& L, int device, int sms, cudaStream_t st, bool map_w = true) {
  constexpr bool kPair = kWeightsA, kSegments = kSums != kWhole;
  MmaParams P = {};
  P.L = L;
  P.every = P.classes = P.group_classes = 1;
  int64_t blocks = (static_cast<int64_t>(L.K) + kMmaK - 1) / kMmaK;
  if (kLoad && map_w && L.K > 0) {
    P.w_mapped = 1;
    P.every = L.N > 1 ? period(L.w_row) : 1;
    P.classes = std::min(P.every, L.N);
    P.group_classes = L.groups > 1 ? std::min(period(L.w_group), L.groups) : 1;
    if (P.classes * P.group_classes > 1 || reinterpret_cast<uintptr_t>(L.w) % 16)
      blocks = (static_cast<int64_t>(L.K) + 7 + kMmaK - 1) / kMmaK;
  }
  const int tokens = kWeightsA ? L.M : std::min(L.M, 128);  // of a tile of x
  P.ra = kWeightsA ? 128 : (tokens + 7) / 8 * 8;
  const int64_t rows_a = kWeightsA ? L.N : L.M;
  const int64_t rows_b = kWeightsA ? L.M : (static_cast<int64_t>(L.N) + P.every - 1) / P.every;
  const int workers = kPair ? std::max(1, sms / 2) : sms;
  P.tiles_a = static_cast<int>((rows_a + (kPair ? 255 : 127)) / (kPair ? 256 : 128));
  P.halves = kSegments && blocks <= 2 * kLongF32 / kMmaK;
  const int64_t others = static_cast<int64_t>(P.tiles_a) * P.classes;
  P.nt = choose_width(kPair, kSegments && !P.halves ? 160 : 256, rows_b, others, P.ra, L.groups, blocks, workers);
  P.tiles_b = static_cast<int>((rows_b + P.nt - 1) / P.nt);
  const int64_t most_tiles = (int64_t{1} << 31) - 1;
  if (others * P.tiles_b > most_tiles / L.groups) {
    // classes of rows cut the columns into up to eight times as many tiles; without them there are fewer than 2^31 for any
    // y that memory holds (a tile's width is at least N as far as 256)
    if (P.classes > 1) return launch_mma<false, true, kSums>(L, device, sms, st, false);
    return SV_EUNSUPPORTED;
  }
  const int64_t tiles = others * P.tiles_b * L.groups;
  P.tiles = static_cast<unsigned>(tiles);
  const int b_rows = kPair ? P.nt / 2 : P.nt;
  Maps<kLoad ? kMostMaps : 2> maps;
  if constexpr (kLoad) {
    P.b_groups = L.w_group > 0;
    if (P.w_mapped && !map_classes(&P, &maps)) return launch_mma<false, true, kSums>(L, device, sms, st, false);
  } else {
    CUtensorMap& map_x = maps.m[kWeightsA ? 1 : 0];
    CUtensorMap& map_w = maps.m[kWeightsA ? 0 : 1];
    int gx = 0, gw = 0;
    if (!make_map(&map_x, L.x, L.K, L.M, L.groups, L.x_row, L.x_group, kWeightsA ? b_rows : P.ra, &gx) ||
        !make_map(&map_w, L.w, L.K, L.N, L.groups, L.w_row, L.w_group, kWeightsA ? 128 : b_rows, &gw))
      return launch_mma<false, true, kSums>(L, device, sms, st);
    P.a_groups = kWeightsA ? gw : gx;
    P.b_groups = kWeightsA ? gx : gw;
  }
  const int sub_bytes = (P.ra + b_rows) * kRowBytes;
  P.at_once = tokens <= 32 && P.nt > 128;
  const int staging = kWeightsA ? 0 : tokens * ((P.at_once ? kEpiWarps * 32 : kStageCols) + 1) * 4;
  // a product reads 128 rows of A from a stage's last block on: they stay inside the allocation
  const int slack = std::max(0, 128 * kRowBytes - sub_bytes);
  const int room = kMmaSmem - 1024 - staging - slack;
  // Two or four blocks of K to a stage, as far as four stages fit: waiting for a stage and releasing it costs the issuing
  // warp as much as the products of a block (N = 2048 in 4 groups, K = 2048, M = 1: 12.5 us with one, 9.1 us with four;
  // M = 384, N = 128256, K = 4096: 253 us with one, 241 us with two; three stages are too few: M = 256, N = 32000, K =
  // 4096 53.2 us with one block, 56.8 us with two).
  P.sub = 1;
  while (!kLoad && P.sub < 4 && P.sub < blocks && 2 * P.sub * sub_bytes * 4 <= room) P.sub *= 2;
  P.kblocks = static_cast<int>((blocks + P.sub - 1) / P.sub);
  P.seg_blocks = P.halves ? (P.kblocks + 1) / 2 : kSegments ? 8 / P.sub : std::max(1, P.kblocks);
  P.segs = std::max(1, (P.kblocks + P.seg_blocks - 1) / P.seg_blocks);
  const int stage_bytes = P.sub * sub_bytes;
  P.stages = std::min(kMaxStages, room / stage_bytes);
  if (kLoad && P.stages < kLoadGroups) return SV_EUNSUPPORTED;  // never: four stages of 128 + 256 rows fit
  P.staging = 1024 + P.stages * stage_bytes + slack;
  const int smem = static_cast<int>(P.staging) + staging;
  P.tmem_cols = 32;
  // two accumulators, read 32 columns at a time, or three regions of sums, read 16 at a time
  while (P.tmem_cols < (kSegments && !P.halves ? 3 * P.nt : P.nt + (P.nt + 31) / 32 * 32)) P.tmem_cols *= 2;
  // fp32 sums, bf16 operands, both K-major, N = nt, M = 128 or 256
  P.idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<unsigned>(P.nt / 8) << 17) | ((kPair ? 16u : 8u) << 24);
  // once a device
  static std::atomic<bool> opted_in[64];
  if (device >= 64 || !opted_in[device].load()) {
    if (cudaFuncSetAttribute(mma_kernel<kWeightsA, kLoad, kSums>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmaSmem) !=
        cudaSuccess)
      return SV_ECUDA;
    if (device < 64) opted_in[device].store(true);
  }
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, workers)) * (kPair ? 2 : 1);
  const unsigned threads = kMmaThreads + (kLoad ? 32 * kLoadGroups * kLoadWarps : 0);
  const cudaError_t e = launch_waiting(mma_kernel<kWeightsA, kLoad, kSums>, grid, threads, smem, kPair ? 2 : 1, st, P, maps);
  return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

bool valid_dtype(int d) { return d == SV_F32 || d == SV_BF16; }
bool aligned_to(const void* p, int d) { return reinterpret_cast<uintptr_t>(p) % (d == SV_BF16 ? 2 : 4) == 0; }

}  // namespace
}  // namespace sv

extern "C" sv_status spec_verify_linear(const void* x, int64_t x_row, int64_t x_group, const void* w, int64_t w_row,
                                        int64_t w_group, const void* bias, sv_dtype bias_dt, int64_t bias_group,
                                        const void* residual, sv_dtype residual_dt, int64_t residual_row,
                                        int64_t residual_group, void* y, sv_dtype y_dt, int64_t y_row,
                                        int64_t y_group, int groups, int M, int N, int K, sv_activation act,
                                        float cap, int device, void* cuda_stream) {
  if (groups < 0 || M < 0 || N < 0 || K < 0) return SV_EINVAL;
  if (!sv::valid_dtype(y_dt) || (bias && !sv::valid_dtype(bias_dt)) || (residual && !sv::valid_dtype(residual_dt)))
    return SV_EINVAL;
  if (act < SV_ACT_NONE || act > SV_ACT_SOFTCAP) return SV_EINVAL;
  if (act == SV_ACT_SOFTCAP && !(cap > 0.f && std::isfinite(cap) && std::isfinite(1.f / cap))) return SV_EINVAL;
  if (x_row < 0 || x_group < 0 || w_row < 0 || w_group < 0 || bias_group < 0 || residual_row < 0 ||
      residual_group < 0 || y_row < 0 || y_group < 0)
    return SV_EINVAL;
  for (const int64_t stride : {x_row, x_group, w_row, w_group, bias_group, residual_row, residual_group, y_row, y_group})
    if (stride >= (int64_t{1} << 40)) return SV_EUNSUPPORTED;
  if (std::max({groups, M, N, K}) > (1 << 30)) return SV_EUNSUPPORTED;
  if (groups == 0 || M == 0 || N == 0) return SV_OK;
  if (!y || (K > 0 && (!x || !w))) return SV_EINVAL;
  if (!sv::aligned_to(x, SV_BF16) || !sv::aligned_to(w, SV_BF16) || !sv::aligned_to(y, y_dt) ||
      (bias && !sv::aligned_to(bias, bias_dt)) || (residual && !sv::aligned_to(residual, residual_dt)))
    return SV_EINVAL;
  if (!sv::rows_apart(y_row, y_group, M, groups, N)) return SV_EINVAL;
  sv::DeviceGuard guard(device);
  if (!guard.ok) return SV_ECUDA;
  const int64_t rs = residual_dt == SV_BF16 ? 2 : 4;
  const sv::Extent ey = {y, y_dt == SV_BF16 ? 2 : 4, N, y_row, M, y_group, groups};
  const sv::Extent ex = {x, 2, K, x_row, M, x_group, groups}, ew = {w, 2, K, w_row, N, w_group, groups};
  const sv::Extent er = {residual, rs, N, residual_row, M, residual_group, groups};
  const sv::Extent eb = {bias, bias_dt == SV_BF16 ? 2 : 4, N, bias_group, groups, 0, 1};
  if (K > 0 && (sv::sure_to_overlap(ey, ex) || sv::sure_to_overlap(ey, ew))) return SV_EINVAL;
  if (bias && sv::sure_to_overlap(ey, eb)) return SV_EINVAL;
  const bool own_residual = residual == y && residual_dt == y_dt && (M == 1 || residual_row == y_row) &&
                            (groups == 1 || residual_group == y_group);
  if (residual && !own_residual && sv::sure_to_overlap(ey, er)) return SV_EINVAL;
  sv::LinearParams P = {};
  P.x = static_cast<const __nv_bfloat16*>(x);
  P.w = static_cast<const __nv_bfloat16*>(w);
  P.bias = bias;
  P.res = residual;
  P.y = y;
  P.x_row = x_row, P.x_group = x_group;
  P.w_row = w_row, P.w_group = w_group;
  P.b_group = bias_group;
  P.r_row = residual_row, P.r_group = residual_group;
  P.y_row = y_row, P.y_group = y_group;
  P.groups = groups, P.M = M, P.N = N, P.K = K;
  P.bias_bf16 = bias_dt == SV_BF16, P.res_bf16 = residual_dt == SV_BF16, P.y_bf16 = y_dt == SV_BF16;
  P.act = act;
  P.cap = cap;
  P.inv_cap = act == SV_ACT_SOFTCAP ? 1.f / cap : 0.f;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return SV_ECUDA;
  if (K == 0) return sv::launch_mma<false, true, sv::kWhole>(P, device, sms, st);
  if (y_dt == SV_F32 && K > sv::kLongF32)
    return M > 128 ? sv::launch_mma<true, false, sv::kSegmentsF32>(P, device, sms, st)
                   : sv::launch_mma<false, false, sv::kSegmentsF32>(P, device, sms, st);
  if (y_dt == SV_BF16 && K > sv::kLongBf16)
    return M > 128 ? sv::launch_mma<true, false, sv::kSegmentsBf16>(P, device, sms, st)
                   : sv::launch_mma<false, false, sv::kSegmentsBf16>(P, device, sms, st);
  return M > 128 ? sv::launch_mma<true, false, sv::kWhole>(P, device, sms, st)
                 : sv::launch_mma<false, false, sv::kWhole>(P, device, sms, st);
}
