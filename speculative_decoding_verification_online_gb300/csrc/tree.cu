// Verification of drafted trees against probabilities: spec_verify_tree.
//
// At a node of the accepted path with target row p and draft row q, its
// children x_1, x_2, ... are offered in turn.  What is left of p after i
// refusals is, up to its mass,
//   rest_i = (p - c_i q)+,   c_0 = 0,   Z_0 = 1,   Z_i = sum rest_i,
// for a refusal of a proposal drawn from q / w_i (w_i = 1 with replacement,
// 1 minus the offered mass without) leaves
//   (rest_i / Z_i - q / w_i)+  ~  (rest_i - (Z_i / w_i) q)+  =  (p - (c_i + Z_i / w_i) q)+
// (where rest_i is 0, c_i q >= p already).  So one number per node carries the
// whole recursion, and a refusal costs one sum over the row pair.
//
// A pick among V tokens hangs on the last digits of its prefix sums: with
// sums good to 1e-7 one pick in a hundred would land beside the token that
// exact sums give.  fp64 has two lanes an SM and clock here (a warp's instruction
// takes its partition 64 clocks, and a walk and a pick in fp64 took 4 and 8 us), so
// everything is carried as pairs of floats: error-free sums and products, about 48
// bits.
//
// A sequence is a cluster of up to eight CTAs, each with a part of the row; every
// CTA's first warp takes the same walk, and a sum over a row is one exchange of
// partial sums through the cluster's shared memory.
//
// Measured on a GB300: one chain of four drafts over 32000 tokens 7.1 us, of which
// a pass over the row pair takes 2 and the dependent loads in front of the walk 1.6;
// 64 chains over 128256 tokens 15.8 us, their first pass at 8 TB/s from HBM and L2;
// 32 trees of up to 21 drafts over 151936 tokens 30.8 us, bound by the sequence with
// the most refusals (about 5 us each: a pass of 1.2 MB by eight SMs, an exchange, a
// step of the walk).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "entry.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kTreeThreads = 512;
constexpr int kTreeWarps = kTreeThreads / 32;
constexpr int kTreeCluster = 8;  // CTAs of a sequence at most
constexpr int kTreeChunk = 512;  // entries of a row whose weight is kept as one sum: 16 a lane

struct TreeParams {
  const float* p;
  const float* q;
  int64_t p_stride, q_stride;
  const int32_t *node_start, *tokens, *parent, *draft_row;
  const float *u_accept, *u_pick;
  int draft_rows, total_nodes, max_nodes, max_depth, V, nchunk, replacement;
  int32_t *accepted_len, *out_tokens, *path;
  float* accept_prob;
  int8_t* flags;
  unsigned long long* counters;
};

struct TreeShared {
  int32_t tok[SV_MAX_NODES], par[SV_MAX_NODES], drow[SV_MAX_NODES + 1];
  int32_t first[SV_MAX_NODES + 1], next[SV_MAX_NODES];  // children of node i - 1; the sibling after node i
  float px[SV_MAX_NODES], qx[SV_MAX_NODES], u[SV_MAX_NODES], alpha[SV_MAX_NODES];
  int32_t refused[SV_MAX_NODES];  // distinct tokens refused at a node without a draft row
  int8_t flag[SV_MAX_NODES], again[SV_MAX_NODES];
  // the CTAs' sums of a pass, by its parity: a CTA writes a place again only after every other one has passed the
  // exchange between
  float2 slot[2][kTreeCluster];
  uint64_t arrived[2];
  volatile int dead;
  // what the first warp asks of the others
  const float* row_p;
  const float* row_q;  // null: c is 0
  float c, cl;
  int n_refused, work;
};

enum { kTreeSum = 0, kTreePick = 1, kTreeEnd = 2 };

// s + l, l what s does not hold
struct Pair {
  float s, l;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, z = t - s;
    l += (s - (t - z)) + (x - z);
    s = t;
  }
  __device__ __forceinline__ void add(const Pair& o) {
    add(o.s);
    l += o.l;
  }
  __device__ __forceinline__ float value() const { return s + l; }
  // s the float nearest to s + l
  __device__ __forceinline__ Pair settled() const {
    const float t = s + l;
    return {t, l - (t - s)};
  }
};

__device__ __forceinline__ Pair times(const Pair& a, const Pair& b) {
  const float h = __fmul_rn(a.s, b.s);
  return Pair{h, fmaf(a.s, b.s, -h) + fmaf(a.s, b.l, a.l * b.s)}.settled();
}

__device__ __forceinline__ bool above(const Pair& a, const Pair& b) { return (a.s - b.s) + (a.l - b.l) > 0.f; }
__device__ __forceinline__ bool at_most(const Pair& a, const Pair& b) { return (a.s - b.s) + (a.l - b.l) <= 0.f; }

// a / b, b not 0
__device__ __forceinline__ Pair over(const Pair& a, const Pair& b) {
  const float x = a.s / b.s;
  const Pair back = times(Pair{x, 0.f}, b);
  return Pair{x, ((a.s - back.s) + (a.l - back.l)) / b.s}.settled();
}

// (p - (c + cl) q)+; a NaN stays
__device__ __forceinline__ Pair rest_of(float p, float q, float c, float cl) {
  const float h = __fmul_rn(c, q);  // not to be fused into the difference below
  const float hl = fmaf(cl, q, fmaf(c, q, -h));
  const float d = p - h, z = d - p;
  const float dl = ((p - (d - z)) - (h + z)) - hl;
  return d + dl <= 0.f ? Pair{0.f, 0.f} : Pair{d, dl};
}

// Two floats in a 64-bit register: one instruction for both, each rounded by itself.
using Two = unsigned long long;

__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(Two t) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(t));
  return f;
}
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
// b - a: a product with -1 is exact
__device__ __forceinline__ Two minus2(Two b, Two a) { return fma2(a, two(-1.f, -1.f), b); }

// two running sums
struct Pairs {
  Two s, l;
  __device__ __forceinline__ void add(Two x) {
    const Two t = add2(s, x), z = minus2(t, s);
    l = add2(l, add2(minus2(s, minus2(t, z)), minus2(x, z)));
    s = t;
  }
  __device__ __forceinline__ Pair total() const {
    const float2 a = both(s), b = both(l);
    Pair p = {a.x, b.x};
    p.add(Pair{a.y, b.y});
    return p;
  }
};

// rest_of for two entries, onto the sums.  kOne: c + cl is 1
template <bool kOne>
__device__ __forceinline__ void add_rests(Pairs& sum, Two p, Two q, Two c, Two minus_c, Two cl) {
  const Two nh = kOne ? minus2(two(0.f, 0.f), q) : mul2(minus_c, q);  // - c q, rounded
  const Two d = add2(p, nh), z = minus2(d, p);
  Two dl = minus2(minus2(p, minus2(d, z)), minus2(z, nh));
  if (!kOne) dl = minus2(dl, fma2(cl, q, fma2(c, q, nh)));
  const float2 r = both(add2(d, dl)), a = both(d), b = both(dl);
  const bool x = r.x <= 0.f, y = r.y <= 0.f;  // not so for a NaN, which stays
  sum.add(two(x ? 0.f : a.x, y ? 0.f : a.y));
  sum.l = add2(sum.l, two(x ? 0.f : b.x, y ? 0.f : b.y));
}

__device__ __forceinline__ Pair warp_total(Pair x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x.add(Pair{__shfl_xor_sync(~0u, x.s, o), __shfl_xor_sync(~0u, x.l, o)});
  return x;
}

// inclusive sums over the lanes
__device__ __forceinline__ Pair scan(Pair x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair up = {__shfl_up_sync(~0u, x.s, o), __shfl_up_sync(~0u, x.l, o)};
    if (lane >= o) x.add(up);
  }
  return x.settled();
}

__device__ __forceinline__ Pair from_lane(const Pair& x, int lane) {
  return {__shfl_sync(~0u, x.s, lane), __shfl_sync(~0u, x.l, lane)};
}

__device__ __forceinline__ Pair rest_at(const TreeShared& s, int v) {
  for (int i = 0; i < s.n_refused; ++i)
    if (s.refused[i] == v) return {0.f, 0.f};
  const float p = s.row_p[v];
  return s.row_q ? rest_of(p, s.row_q[v], s.c, s.cl) : Pair{fmaxf(p, 0.f), 0.f};
}

// four neighbouring entries of a row; nothing beyond its end
template <bool kVec>
__device__ __forceinline__ float4 load4(const float* row, int v, int V) {
  if constexpr (kVec) {
    if (v + 4 <= V) return *reinterpret_cast<const float4*>(row + v);
  } else if (v + 4 <= V) {
    return make_float4(row[v], row[v + 1], row[v + 2], row[v + 3]);
  }
  return make_float4(v < V ? row[v] : 0.f, v + 1 < V ? row[v + 1] : 0.f, v + 2 < V ? row[v + 2] : 0.f, 0.f);
}

// the weight of each of this CTA's chunks into chunk_sum: every warp
template <bool kVec>
__device__ __forceinline__ void chunk_sums(const TreeShared& s, float2* chunk_sum, int V, int first, int last) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float c = s.c, cl = s.cl;
  for (int ch = first + warp; ch < last; ch += kTreeWarps) {
    Pairs sum[2] = {};
    const int v0 = ch * kTreeChunk + lane * 4;
    float4 p[4], q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = load4<kVec>(s.row_p, v0 + j * 128, V);
    if (s.row_q) {
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = load4<kVec>(s.row_q, v0 + j * 128, V);
      const Two c2 = two(c, c), minus_c2 = two(-c, -c), cl2 = two(cl, cl);
      if (c == 1.f && cl == 0.f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          add_rests<true>(sum[0], two(p[j].x, p[j].y), two(q[j].x, q[j].y), c2, minus_c2, cl2);
          add_rests<true>(sum[1], two(p[j].z, p[j].w), two(q[j].z, q[j].w), c2, minus_c2, cl2);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          add_rests<false>(sum[0], two(p[j].x, p[j].y), two(q[j].x, q[j].y), c2, minus_c2, cl2);
          add_rests<false>(sum[1], two(p[j].z, p[j].w), two(q[j].z, q[j].w), c2, minus_c2, cl2);
        }
      }
    } else {
      bool hit = false;
      for (int i = 0; i < s.n_refused; ++i) hit |= s.refused[i] / kTreeChunk == ch;
      if (hit)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          for (int i = 0; i < s.n_refused; ++i) {
            const int at = s.refused[i] - (v0 + j * 128);
            if (at == 0) p[j].x = 0.f;
            if (at == 1) p[j].y = 0.f;
            if (at == 2) p[j].z = 0.f;
            if (at == 3) p[j].w = 0.f;
          }
      // a NaN or an infinity stays: p - p is 0 for every other p
      auto weight = [](float x) { return fmaxf(x, 0.f) + (x - x); };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[0].add(two(weight(p[j].x), weight(p[j].y)));
        sum[1].add(two(weight(p[j].z), weight(p[j].w)));
      }
    }
    Pair mine = sum[0].total();
    mine.add(sum[1].total());
    const Pair t = warp_total(mine).settled();
    if (lane == 0) chunk_sum[ch - first] = make_float2(t.s, t.l);
  }
}

// The first lane whose weight carries the sums past y; the last lane with weight where `any` and none does; else -1.
// *before becomes the sum in front of that lane.
__device__ __forceinline__ int lane_past(const Pair& w, const Pair& y, bool any, Pair* before) {
  Pair incl = scan(w);
  incl.add(*before);
  incl = incl.settled();
  const bool some = w.value() > 0.f;
  const unsigned past = __ballot_sync(~0u, some && above(incl, y)), heavy = __ballot_sync(~0u, some);
  const int at = past ? __ffs(past) - 1 : any && heavy ? 31 - __clz(heavy) : -1;
  const Pair up = from_lane(incl, at < 0 ? 31 : at ? at - 1 : 0);
  if (at != 0) *before = up;
  return at;
}

// The smallest v of this CTA's chunks whose inclusive prefix sum exceeds y, or the last v with weight when rounding
// leaves none (or y is infinite): the first warp.
template <bool kVec>
__device__ int pick(const TreeShared& s, const float2* chunk_sum, int V, int first, int last, Pair y) {
  const int lane = threadIdx.x & 31;
  Pair before = {0.f, 0.f};
  int ch = -1, heavy = first;
  for (int i0 = first; i0 < last && ch < 0; i0 += 32) {
    const float2 f = i0 + lane < last ? chunk_sum[i0 + lane - first] : make_float2(0.f, 0.f);
    const unsigned some = __ballot_sync(~0u, f.x + f.y > 0.f);
    if (some) heavy = i0 + 31 - __clz(some);
    const int at = lane_past(Pair{f.x, f.y}, y, false, &before);
    if (at >= 0) ch = i0 + at;
  }
  if (ch < 0) {
    ch = heavy;
    y = Pair{INFINITY, 0.f};
  }
  // runs of 16 neighbours a lane, then the 16 of one run
  constexpr int kRun = kTreeChunk / 32;
  const int v0 = ch * kTreeChunk + lane * kRun;
  Pair mine = {0.f, 0.f};
  float4 p[kRun / 4], q[kRun / 4];
#pragma unroll
  for (int j = 0; j < kRun / 4; ++j) p[j] = load4<kVec>(s.row_p, v0 + 4 * j, V);
  if (s.row_q) {
#pragma unroll
    for (int j = 0; j < kRun / 4; ++j) q[j] = load4<kVec>(s.row_q, v0 + 4 * j, V);
    Pairs sum[2] = {};
    const Two c2 = two(s.c, s.c), minus_c2 = two(-s.c, -s.c), cl2 = two(s.cl, s.cl);
#pragma unroll
    for (int j = 0; j < kRun / 4; ++j) {
      add_rests<false>(sum[0], two(p[j].x, p[j].y), two(q[j].x, q[j].y), c2, minus_c2, cl2);
      add_rests<false>(sum[1], two(p[j].z, p[j].w), two(q[j].z, q[j].w), c2, minus_c2, cl2);
    }
    mine = sum[0].total();
    mine.add(sum[1].total());
  } else if (s.n_refused == 0) {
#pragma unroll
    for (int j = 0; j < kRun / 4; ++j) {
      mine.add(fmaxf(p[j].x, 0.f));
      mine.add(fmaxf(p[j].y, 0.f));
      mine.add(fmaxf(p[j].z, 0.f));
      mine.add(fmaxf(p[j].w, 0.f));
    }
  } else {
    for (int i = 0; i < kRun; ++i)
      if (v0 + i < V) mine.add(rest_at(s, v0 + i));
  }
  const int run = lane_past(mine.settled(), y, true, &before);
  const int at = ch * kTreeChunk + run * kRun + lane;
  const Pair w = lane < kRun && at < V ? rest_at(s, at) : Pair{0.f, 0.f};
  return ch * kTreeChunk + run * kRun + lane_past(w, y, true, &before);
}

template <bool kVec>
__global__ void __launch_bounds__(kTreeThreads, 2) tree_kernel(const __grid_constant__ TreeParams P) {
  extern __shared__ float2 chunk_sum[];
  __shared__ TreeShared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  if (threadIdx.x == 0) {
    mbar_init(&s.arrived[0], 1);
    mbar_init(&s.arrived[1], 1);
    s.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster.barrier_arrive();  // every CTA of the cluster runs before any writes into another
  wait_for_stream();
  const int b = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31;
  const int first = static_cast<int>(static_cast<int64_t>(P.nchunk) * rank / ctas);
  const int last = static_cast<int>(static_cast<int64_t>(P.nchunk) * (rank + 1) / ctas);
  const int start = P.node_start[b], end = P.node_start[b + 1];
  const bool inside = start >= 0 && end >= start && end <= P.total_nodes;
  const bool range = inside && end - start <= P.max_nodes;
  const int n = range ? end - start : 0;
  const int64_t root = static_cast<int64_t>(start) + b;
  int bad = !range;
  for (int i = tid; range && i <= n; i += kTreeThreads) {
    s.drow[i] = P.draft_row[root + i];
    s.first[i] = SV_MAX_NODES;
    bad |= s.drow[i] < -1 || s.drow[i] >= P.draft_rows;
    if (i == n) break;
    s.tok[i] = P.tokens[start + i];
    s.par[i] = P.parent[start + i];
    s.u[i] = P.u_accept[start + i];
    s.flag[i] = SV_FLAG_UNREACHED;
    s.alpha[i] = 0.f;
    bad |= s.tok[i] < 0 || s.tok[i] >= P.V || s.par[i] < -1 || s.par[i] >= i;
  }
  bad = __syncthreads_or(bad);
  if (!bad) {
    for (int i = tid; i < n; i += kTreeThreads) {
      const int par = s.par[i], tok = s.tok[i], d = s.drow[par + 1];
      s.px[i] = P.p[(root + 1 + par) * P.p_stride + tok];
      s.qx[i] = d < 0 ? 1.f : P.q[d * P.q_stride + tok];
      atomicMin(&s.first[par + 1], i);
      int next = SV_MAX_NODES, again = 0;
      for (int j = 0; j < n; ++j)
        if (s.par[j] == par) {
          if (j > i) next = min(next, j);
          if (j < i && s.tok[j] == tok) again = 1;
        }
      s.next[i] = next;
      s.again[i] = static_cast<int8_t>(again);
      if (n > P.max_depth) {
        int depth = 1;
        for (int a = par; a >= 0; a = s.par[a]) ++depth;
        bad |= depth > P.max_depth;
      }
    }
    bad = __syncthreads_or(bad);
  }

  cluster.barrier_wait();

  // The walk: the first warp of every CTA takes the same steps, and stops where a sum over a row is needed.
  int cur = -1, child = bad ? SV_MAX_NODES : s.first[0];
  int len = 0, refused = 0, tested = 0, offered = 0, degenerate = 0, pass = 0;  // offered: children of cur
  const Pair zero = {0.f, 0.f}, one = {1.f, 0.f};
  Pair c = zero, Z = one, mass = zero;
  bool summed = false, closing = false;  // chunk_sum is that of cur and c; the sum for the pick is under way
  if (n == 0) child = SV_MAX_NODES;
  for (;;) {
    if (tid < 32) {
      int work = bad ? kTreeEnd : -1;
      bool bare = bad || s.drow[cur + 1] < 0;
      if (work < 0 && pass > 0) {
        // what the last pass was for
        Z = zero;
        for (int r = 0; r < ctas; ++r) Z.add(Pair{s.slot[(pass - 1) & 1][r].x, s.slot[(pass - 1) & 1][r].y});
        Z = Z.settled();
        if (!(Z.value() >= 0.f && Z.value() < INFINITY)) bad = 1, work = kTreeEnd;
        if (closing && work < 0) {
          if (Z.value() > 0.f) {
            work = kTreePick;
          } else if (degenerate) {
            bad = 1, work = kTreeEnd;  // the node's own row has no mass
          } else {
            degenerate = 1;
            if (lane == 0) s.row_q = nullptr, s.n_refused = 0;
            work = kTreeSum;
          }
        }
      }
      while (work < 0) {
        if (child >= SV_MAX_NODES) {
          // no child is left: the token comes from what is left of this row
          closing = true;
          if (summed && Z.value() > 0.f) {
            work = kTreePick;
          } else {
            if (summed) degenerate = 1;
            if (lane == 0) {
              s.row_p = P.p + (root + 1 + cur) * P.p_stride;
              s.row_q = nullptr;
              int k = 0;
              if (bare)
                for (int i = s.first[cur + 1]; i < SV_MAX_NODES && n > 0; i = s.next[i])
                  if (!s.again[i]) s.refused[k++] = s.tok[i];
              s.n_refused = k;
            }
            work = kTreeSum;
          }
          break;
        }
        const int i = child;
        float qx = s.qx[i];
        const float px = s.px[i], u = s.u[i];
        if (!(px >= 0.f && px < INFINITY && qx >= 0.f && qx < INFINITY)) {
          bad = 1, work = kTreeEnd;
          break;
        }
        bool yes;
        float alpha;
        Pair r, w = one;
        if (offered == 0 && (bare || P.replacement || qx <= 1.f) && px >= 1e-30f) {
          // a first child: rest is p and Z is 1, and the sign of u q - p is exact in one fused step
          r = Pair{px, 0.f};
          yes = fmaf(u, qx, -px) <= 0.f;
          alpha = qx > px ? px / qx : 1.f;
        } else {
          r = bare ? Pair{s.again[i] ? 0.f : px, 0.f} : rest_of(px, qx, c.s, c.l);
          // a sibling offered before has no place in what is left of the proposal
          if (!bare && !P.replacement && s.again[i]) qx = 0.f;
          if (!bare && !P.replacement) {
            w.add(-mass.s);
            w.l -= mass.l;
            w = w.value() > qx ? w.settled() : Pair{qx, 0.f};
          }
          const Pair most = times(Z, Pair{qx, 0.f}), rw = times(r, w);
          yes = r.value() > 0.f && at_most(times(most, Pair{u, 0.f}), rw);
          alpha = most.value() > 0.f ? (above(most, rw) ? over(rw, most).value() : 1.f) : (r.value() > 0.f ? 1.f : 0.f);
        }
        if (lane == 0 && rank == 0) {
          s.alpha[i] = alpha;
          s.flag[i] = yes ? SV_FLAG_ACCEPT : SV_FLAG_REJECT;
          if (yes) {
            if (P.path) P.path[static_cast<int64_t>(b) * P.max_depth + len] = i;
            P.out_tokens[static_cast<int64_t>(b) * (P.max_depth + 1) + len] = s.tok[i];
          }
        }
        ++tested;
        ++offered;
        if (yes) {
          ++len;
          cur = i, child = s.first[i + 1];
          c = zero, Z = one, mass = zero, offered = 0, summed = false;
          bare = s.drow[cur + 1] < 0;
          continue;
        }
        ++refused;
        mass.add(qx);
        child = s.next[i];
        if (bare) {
          Z.add(-r.s);
          Z = Z.settled();
        } else if (Z.value() > 0.f || !summed) {
          if (w.s == 1.f && w.l == 0.f) {
            c.add(Z);
          } else if (w.value() > 0.f) {
            c.add(over(Z, w));
          }
          c = c.s < 1e30f ? c.settled() : Pair{1e30f, 0.f};
          summed = true;
          if (lane == 0) {
            s.row_p = P.p + (root + 1 + cur) * P.p_stride;
            s.row_q = P.q + s.drow[cur + 1] * P.q_stride;
            s.c = c.s, s.cl = c.l;
            s.n_refused = 0;
          }
          work = kTreeSum;
        }
      }
      if (lane == 0) s.work = work;
    }
    __syncthreads();
    if (s.work != kTreeSum) break;
    chunk_sums<kVec>(s, chunk_sum, P.V, first, last);
    __syncthreads();
    if (tid < 32) {
      Pair t = zero;
      for (int i = lane; i < last - first; i += 32) t.add(Pair{chunk_sum[i].x, chunk_sum[i].y});
      t = warp_total(t).settled();
      // The sum goes into every CTA's memory, and the write itself counts there: a cluster barrier would hold up all
      // threads, and first wait for their stores.
      if (lane == 0) mbar_expect(&s.arrived[pass & 1], ctas * sizeof(float2));
      if (lane < ctas)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                         in_cta(&s.slot[pass & 1][rank], lane)),
                     "f"(t.s), "f"(t.l), "r"(in_cta(&s.arrived[pass & 1], lane))
                     : "memory");
      if (!__all_sync(~0u, mbar_wait(&s.arrived[pass & 1], pass >> 1 & 1, &s.dead))) bad = 1;
    }
    ++pass;
  }

  if (tid < 32 && s.work == kTreePick) {
    // the CTA whose part of the row holds u * Z
    const float2 f = lane < ctas ? s.slot[(pass - 1) & 1][lane] : make_float2(0.f, 0.f);
    Pair y = times(Z, Pair{P.u_pick[b], 0.f}), before = zero;
    const unsigned some = __ballot_sync(~0u, f.x + f.y > 0.f);
    int owner = lane_past(Pair{f.x, f.y}, y, false, &before);
    if (owner < 0) {
      owner = 31 - __clz(some);
      y = Pair{INFINITY, 0.f};
    } else {
      y.add(-before.s);
      y.l -= before.l;
      y = y.settled();
    }
    if (owner == rank) {
      const int v = pick<kVec>(s, chunk_sum, P.V, first, last, y);
      if (lane == 0) P.out_tokens[static_cast<int64_t>(b) * (P.max_depth + 1) + len] = v;
    }
  }
  // A CTA whose wait gave up stays behind, and then leaves the results of a sequence that failed, whatever others left.
  if (s.dead) stay_behind();
  else if (rank != 0) return;
  // rank 0 leaves the rest; its first warp knows how the walk went
  __shared__ int s_len, s_bad;
  if (tid == 0) {
    s_len = len, s_bad = bad;
    P.accepted_len[b] = bad ? -1 : len;
    if (P.counters && rank == 0) {
      if (bad) {
        atomicAdd(P.counters + SV_CNT_INVALID, 1ull);
      } else {
        if (tested) atomicAdd(P.counters + SV_CNT_TESTED, static_cast<unsigned long long>(tested));
        if (len) atomicAdd(P.counters + SV_CNT_ACCEPTED, static_cast<unsigned long long>(len));
        if (refused) atomicAdd(P.counters + SV_CNT_REJECTED, static_cast<unsigned long long>(refused));
        if (degenerate) atomicAdd(P.counters + SV_CNT_DEGENERATE, 1ull);
        if (offered == 0) atomicAdd(P.counters + SV_CNT_BONUS, 1ull);
      }
    }
  }
  __syncthreads();
  len = s_len, bad = s_bad;
  const int from = bad ? 0 : len;
  for (int i = tid; i <= P.max_depth; i += kTreeThreads) {
    if (i > len || bad) P.out_tokens[static_cast<int64_t>(b) * (P.max_depth + 1) + i] = -1;
    if (P.path && i >= from && i < P.max_depth) P.path[static_cast<int64_t>(b) * P.max_depth + i] = -1;
  }
  for (int i = tid; i < (inside ? end - start : 0); i += kTreeThreads) {
    if (P.accept_prob) P.accept_prob[start + i] = bad ? 0.f : s.alpha[i];
    if (P.flags) P.flags[start + i] = bad ? static_cast<int8_t>(SV_FLAG_INVALID) : s.flag[i];
  }
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_verify_tree(const float* target_probs, int64_t target_stride, const float* draft_probs,
                                      int64_t draft_stride, int draft_rows, const int32_t* node_start,
                                      const int32_t* node_tokens, const int32_t* parent, const int32_t* draft_row,
                                      const float* u_accept, const float* u_pick, int B, int total_nodes,
                                      int max_nodes, int max_depth, int V, sv_siblings siblings,
                                      int32_t* accepted_len, int32_t* tokens, int32_t* path, float* accept_prob,
                                      int8_t* flags, uint64_t* counters, int device, void* cuda_stream) {
  if (B < 0 || total_nodes < 0 || max_nodes < 0 || max_depth < 0 || draft_rows < 0 || V < 1) return SV_EINVAL;
  if (siblings != SV_WITH_REPLACEMENT && siblings != SV_WITHOUT_REPLACEMENT) return SV_EINVAL;
  if (V > SV_MAX_V || max_nodes > SV_MAX_NODES) return SV_EUNSUPPORTED;
  if (max_depth > max_nodes) return SV_EINVAL;
  if (B == 0) return SV_OK;
  if (!target_probs || !node_start || !draft_row || !u_pick || !accepted_len || !tokens) return SV_EINVAL;
  if (total_nodes > 0 && (!node_tokens || !parent || !u_accept)) return SV_EINVAL;
  if (draft_rows > 0 && !draft_probs) return SV_EINVAL;
  if (target_stride < 0 || draft_stride < 0) return SV_EINVAL;
  for (const void* a : {static_cast<const void*>(target_probs), static_cast<const void*>(draft_probs),
                        static_cast<const void*>(node_start), static_cast<const void*>(node_tokens),
                        static_cast<const void*>(parent), static_cast<const void*>(draft_row),
                        static_cast<const void*>(u_accept), static_cast<const void*>(u_pick),
                        static_cast<const void*>(accepted_len), static_cast<const void*>(tokens),
                        static_cast<const void*>(path), static_cast<const void*>(accept_prob)})
    if (reinterpret_cast<uintptr_t>(a) % 4) return SV_EINVAL;
  if (reinterpret_cast<uintptr_t>(counters) % 8) return SV_EINVAL;
  sv::DeviceGuard g(device);
  if (!g.ok) return SV_ECUDA;
  sv::TreeParams P = {};
  P.p = target_probs, P.q = draft_probs;
  P.p_stride = target_stride, P.q_stride = draft_stride;
  P.node_start = node_start, P.tokens = node_tokens, P.parent = parent, P.draft_row = draft_row;
  P.u_accept = u_accept, P.u_pick = u_pick;
  P.draft_rows = draft_rows, P.total_nodes = total_nodes, P.max_nodes = max_nodes, P.max_depth = max_depth;
  P.V = V, P.nchunk = (V + sv::kTreeChunk - 1) / sv::kTreeChunk;
  P.replacement = siblings == SV_WITH_REPLACEMENT;
  P.accepted_len = accepted_len, P.out_tokens = tokens, P.path = path;
  P.accept_prob = accept_prob, P.flags = flags;
  P.counters = reinterpret_cast<unsigned long long*>(counters);
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return SV_ECUDA;
  // As many CTAs a sequence as two per SM allow, each with a chunk for every other warp at least.  Half as many, as chosen and
  // twice as many, chains of four drafts: B = 1, V = 32000 8.2, 7.1, 6.8 us; B = 64, V = 128256 18.6, 16.2, 20.8 us; B = 100
  // 31.4, 26.4, 29.4 us; B = 152 35.9, 30.9, 43.3 us; above 152 sequences one CTA each, or two: B = 160 45.4, 44.8 us, B = 256
  // 48.2, 54.4 us.
  int ctas = 1;
  while (ctas < sv::kTreeCluster && static_cast<int64_t>(B) * ctas * 2 <= 2ll * sms &&
         ctas * sv::kTreeWarps < P.nchunk)
    ctas *= 2;
  if (static_cast<int64_t>(B) * ctas > 0x7fffffff) return SV_EUNSUPPORTED;
  const bool vec = reinterpret_cast<uintptr_t>(target_probs) % 16 == 0 && reinterpret_cast<uintptr_t>(draft_probs) % 16 == 0 &&
                   target_stride % 4 == 0 && draft_stride % 4 == 0;
  const size_t smem = (static_cast<size_t>(P.nchunk) + ctas - 1) / ctas * sizeof(float2) + sizeof(float2);
  const auto kernel = vec ? sv::tree_kernel<true> : sv::tree_kernel<false>;
  if (smem > (32u << 10) &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 << 10) != cudaSuccess)
    return SV_ECUDA;
  return sv::launch_waiting(kernel, static_cast<unsigned>(B * ctas), sv::kTreeThreads, smem, ctas,
                            static_cast<cudaStream_t>(cuda_stream), P) == cudaSuccess
             ? SV_OK
             : SV_ECUDA;
}
