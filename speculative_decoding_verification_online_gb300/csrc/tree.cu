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
// exact sums give.  fp64 has two lanes an SM and clock here, so the row sums are
// carried as pairs of floats (error-free sums and products, about 48 bits); one
// warp does the few scalar steps in fp64.
//
// A sequence is a cluster of up to eight CTAs, each with a part of the row; every
// CTA's first warp takes the same walk, and a sum over a row is one exchange of
// partial sums through the cluster's shared memory.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
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
  double slot[2][kTreeCluster];  // the CTAs' sums of a pass, by its parity
  // what the first warp asks of the others
  const float* row_p;
  const float* row_q;  // null: c is 0
  double c;
  int n_refused, work;
};

enum { kTreeSum = 0, kTreePick = 1, kTreeEnd = 2 };

// s + l, s the nearest float: sums of floats without losing what does not fit
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
};

// (p - (c + cl) q)+ onto a sum; a NaN stays
__device__ __forceinline__ void add_rest(Pair& sum, float p, float q, float c, float cl) {
  const float h = __fmul_rn(c, q);  // not to be fused into the difference below
  const float hl = fmaf(cl, q, fmaf(c, q, -h));
  const float d = p - h, z = d - p;
  const float dl = ((p - (d - z)) - (h + z)) - hl;
  if (!(d + dl <= 0.f)) {
    sum.add(d);
    sum.l += dl;
  }
}

__device__ __forceinline__ Pair warp_total(Pair x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x.add(Pair{__shfl_xor_sync(~0u, x.s, o), __shfl_xor_sync(~0u, x.l, o)});
  return x;
}

__device__ __forceinline__ double rest_at(const TreeShared& s, int v) {
  for (int i = 0; i < s.n_refused; ++i)
    if (s.refused[i] == v) return 0.0;
  const double p = s.row_p[v];
  const double r = s.row_q ? fma(-s.c, static_cast<double>(s.row_q[v]), p) : p;
  return r < 0.0 ? 0.0 : r;
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
__device__ __forceinline__ void chunk_sums(const TreeShared& s, double* chunk_sum, int V, int first, int last) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float c = static_cast<float>(s.c), cl = static_cast<float>(s.c - static_cast<double>(c));
  for (int ch = first + warp; ch < last; ch += kTreeWarps) {
    Pair sum[4] = {};
    const int v0 = ch * kTreeChunk + lane * 4;
    float4 p[4], q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = load4<kVec>(s.row_p, v0 + j * 128, V);
    if (s.row_q) {
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = load4<kVec>(s.row_q, v0 + j * 128, V);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        add_rest(sum[0], p[j].x, q[j].x, c, cl);
        add_rest(sum[1], p[j].y, q[j].y, c, cl);
        add_rest(sum[2], p[j].z, q[j].z, c, cl);
        add_rest(sum[3], p[j].w, q[j].w, c, cl);
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
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[0].add(fmaxf(p[j].x, 0.f) + (p[j].x - p[j].x));  // a NaN or an infinity stays
        sum[1].add(fmaxf(p[j].y, 0.f) + (p[j].y - p[j].y));
        sum[2].add(fmaxf(p[j].z, 0.f) + (p[j].z - p[j].z));
        sum[3].add(fmaxf(p[j].w, 0.f) + (p[j].w - p[j].w));
      }
    }
    sum[0].add(sum[1]);
    sum[2].add(sum[3]);
    sum[0].add(sum[2]);
    const Pair t = warp_total(sum[0]);
    if (lane == 0) chunk_sum[ch - first] = static_cast<double>(t.s) + static_cast<double>(t.l);
  }
}

__device__ __forceinline__ double scan(double x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += up;
  }
  return x;
}

// The smallest v of this CTA's chunks whose inclusive prefix sum exceeds y, or the last v with weight when rounding
// leaves none: the first warp.
__device__ int pick(const TreeShared& s, const double* chunk_sum, int V, int first, int last, double y) {
  const int lane = threadIdx.x & 31;
  double before = 0.0;
  int ch = -1, heavy = first;
  for (int i0 = first; i0 < last && ch < 0; i0 += 32) {
    const int i = i0 + lane;
    const double w = i < last ? chunk_sum[i - first] : 0.0;
    const double incl = before + scan(w);
    const unsigned past = __ballot_sync(~0u, w > 0.0 && incl > y), some = __ballot_sync(~0u, w > 0.0);
    if (some) heavy = i0 + 31 - __clz(some);
    if (past) {
      ch = i0 + __ffs(past) - 1;
      before = __shfl_sync(~0u, incl - w, __ffs(past) - 1);
    } else {
      before = __shfl_sync(~0u, incl, 31);
    }
  }
  if (ch < 0) {
    ch = heavy;
    y = INFINITY;
  }
  // 16 neighbours a lane
  constexpr int kRun = kTreeChunk / 32;
  const int v0 = ch * kTreeChunk + lane * kRun;
  double w[kRun], mine = 0.0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) w[i] = v0 + i < V ? rest_at(s, v0 + i) : 0.0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) mine += w[i];
  const double incl = before + scan(mine);
  const unsigned past = __ballot_sync(~0u, mine > 0.0 && incl > y), some = __ballot_sync(~0u, mine > 0.0);
  const int owner = past ? __ffs(past) - 1 : 31 - __clz(some);
  int v = -1;
  if (lane == owner) {
    double sum = incl - mine;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      sum += w[i];
      if (w[i] > 0.0 && (v < 0 || !past)) v = v0 + i;
      if (past && w[i] > 0.0 && sum <= y) v = -1;
    }
    if (v < 0)  // rounding: the lane's last weight
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        if (w[i] > 0.0) v = v0 + i;
  }
  return __shfl_sync(~0u, v, owner);
}

template <bool kVec>
__global__ void __launch_bounds__(kTreeThreads, 2) tree_kernel(const __grid_constant__ TreeParams P) {
  extern __shared__ double chunk_sum[];
  __shared__ TreeShared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
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
  double c = 0.0, Z = 1.0, mass = 0.0;
  bool summed = false, closing = false;  // chunk_sum is that of cur and c; the sum for the pick is under way
  if (n == 0) child = SV_MAX_NODES;
  for (;;) {
    if (tid < 32) {
      int work = bad ? kTreeEnd : -1;
      bool bare = bad || s.drow[cur + 1] < 0;
      if (work < 0 && pass > 0) {
        // what the last pass was for
        double t = 0.0;
        for (int r = 0; r < ctas; ++r) t += s.slot[(pass - 1) & 1][r];
        Z = t;
        if (!(t >= 0.0 && t < INFINITY)) bad = 1, work = kTreeEnd;
        if (closing && work < 0) {
          if (t > 0.0) {
            work = kTreePick;
          } else if (degenerate) {
            bad = 1, work = kTreeEnd;  // the node's own row has no mass
          } else {
            degenerate = 1;
            c = 0.0;
            if (lane == 0) s.row_q = nullptr, s.c = 0.0, s.n_refused = 0;
            work = kTreeSum;
          }
        }
      }
      while (work < 0) {
        if (child >= SV_MAX_NODES) {
          // no child is left: the token comes from what is left of this row
          closing = true;
          if (summed && Z > 0.0) {
            work = kTreePick;
          } else {
            if (summed) degenerate = 1, c = 0.0;
            if (lane == 0) {
              s.row_p = P.p + (root + 1 + cur) * P.p_stride;
              s.row_q = nullptr;
              s.c = 0.0;
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
        const double qx = s.qx[i], px = s.px[i];
        if (!(px >= 0.0 && px < INFINITY && qx >= 0.0 && qx < INFINITY)) {
          bad = 1, work = kTreeEnd;
          break;
        }
        double r = bare ? (s.again[i] ? 0.0 : px) : fma(-c, qx, px);
        if (r < 0.0) r = 0.0;
        const double w = bare || P.replacement ? 1.0 : fmax(1.0 - mass, qx);
        const double most = qx * Z;
        const bool yes = r > 0.0 && s.u[i] * most <= r * w;
        if (lane == 0 && rank == 0) {
          s.alpha[i] = most > 0.0 ? static_cast<float>(fmin(1.0, r * w / most)) : (r > 0.0 ? 1.f : 0.f);
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
          c = 0.0, Z = 1.0, mass = 0.0, offered = 0, summed = false;
          bare = s.drow[cur + 1] < 0;
          continue;
        }
        ++refused;
        mass += qx;
        child = s.next[i];
        if (bare) {
          Z -= r;
        } else if (Z > 0.0 || !summed) {
          if (w > 0.0) c = fmin(c + Z / w, 1e30);
          summed = true;
          if (lane == 0) {
            s.row_p = P.p + (root + 1 + cur) * P.p_stride;
            s.row_q = P.q + s.drow[cur + 1] * P.q_stride;
            s.c = c;
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
      double t = 0.0;
      for (int i = lane; i < last - first; i += 32) t += chunk_sum[i];
      for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
      if (lane < ctas) *cluster.map_shared_rank(&s.slot[pass & 1][rank], lane) = t;
    }
    ++pass;
    cluster.sync();
  }

  if (tid < 32 && s.work == kTreePick) {
    // the CTA whose part of the row holds u * Z
    const double* sums = s.slot[(pass - 1) & 1];
    const double y = static_cast<double>(P.u_pick[b]) * Z;
    double before = 0.0, mine_before = 0.0;
    int owner = -1, heavy = 0;
    for (int r = 0; r < ctas; ++r) {
      if (r == rank) mine_before = before;
      if (sums[r] > 0.0) heavy = r;
      if (owner < 0 && sums[r] > 0.0 && before + sums[r] > y) owner = r;
      before += sums[r];
    }
    const bool none = owner < 0;
    if (none) owner = heavy;
    if (owner == rank) {
      const int v = pick(s, chunk_sum, P.V, first, last, none ? INFINITY : y - mine_before);
      if (lane == 0) P.out_tokens[static_cast<int64_t>(b) * (P.max_depth + 1) + len] = v;
    }
  }
  if (rank != 0) return;
  // rank 0 leaves the rest; its first warp knows how the walk went
  __shared__ int s_len, s_bad;
  if (tid == 0) {
    s_len = len, s_bad = bad;
    P.accepted_len[b] = bad ? -1 : len;
    if (P.counters) {
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
  // as many CTAs a sequence as two per SM allow, each with a chunk for every other warp at least
  int ctas = 1;
  while (ctas < sv::kTreeCluster && static_cast<int64_t>(B) * ctas * 2 <= 2ll * sms &&
         ctas * sv::kTreeWarps < P.nchunk)
    ctas *= 2;
  if (getenv("TREEC")) ctas = atoi(getenv("TREEC"));
  if (static_cast<int64_t>(B) * ctas > 0x7fffffff) return SV_EUNSUPPORTED;
  const bool vec = reinterpret_cast<uintptr_t>(target_probs) % 16 == 0 && reinterpret_cast<uintptr_t>(draft_probs) % 16 == 0 &&
                   target_stride % 4 == 0 && draft_stride % 4 == 0;
  const size_t smem = (static_cast<size_t>(P.nchunk) + ctas - 1) / ctas * sizeof(double) + sizeof(double);
  const auto kernel = vec ? sv::tree_kernel<true> : sv::tree_kernel<false>;
  if (smem > (32u << 10) &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 << 10) != cudaSuccess)
    return SV_ECUDA;
  return sv::launch_waiting(kernel, static_cast<unsigned>(B * ctas), sv::kTreeThreads, smem, ctas,
                            static_cast<cudaStream_t>(cuda_stream), P) == cudaSuccess
             ? SV_OK
             : SV_ECUDA;
}
