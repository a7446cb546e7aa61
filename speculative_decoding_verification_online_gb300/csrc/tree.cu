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
// exact sums give.  Weights and sums are held in 64 bits.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "device_guard.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

constexpr int kTreeThreads = 512;
constexpr int kTreeWarps = kTreeThreads / 32;
constexpr int kTreeChunk = 1024;  // entries of a row whose weight is kept as one sum

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
  float px[SV_MAX_NODES], qx[SV_MAX_NODES], u[SV_MAX_NODES];
  int8_t flag[SV_MAX_NODES];
  float alpha[SV_MAX_NODES];
  double warp_sum[kTreeWarps];
  double total;
  int pick;
};

// the tokens refused at a node without a draft row
struct Refused {
  const TreeShared& s;
  int n, cur;
  __device__ bool holds(int v) const {
    for (int i = 0; i < n; ++i)
      if (s.par[i] == cur && s.tok[i] == v && s.flag[i] == SV_FLAG_REJECT) return true;
    return false;
  }
};

struct Rest {
  const float* p;
  const float* q;  // null: no draft row, or c is 0
  double c;
  __device__ double operator()(int v) const {
    const double r = q ? static_cast<double>(p[v]) - c * static_cast<double>(q[v]) : static_cast<double>(p[v]);
    return r < 0.0 ? 0.0 : r;  // a NaN stays
  }
};

__device__ __forceinline__ double warp_total(double x) {
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// the weight of every chunk into chunk_sum, their total returned to every thread
__device__ double row_sums(TreeShared& s, double* chunk_sum, const Rest& rest, const Refused* refused, int V,
                           int nchunk) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double mine = 0.0;
  for (int ch = warp; ch < nchunk; ch += kTreeWarps) {
    const int lo = ch * kTreeChunk, hi = min(lo + kTreeChunk, V);
    double sum = 0.0;
    for (int v = lo + lane; v < hi; v += 32) sum += refused && refused->holds(v) ? 0.0 : rest(v);
    sum = warp_total(sum);
    if (lane == 0) chunk_sum[ch] = sum;
    mine += sum;
  }
  if (lane == 0) s.warp_sum[warp] = mine;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < kTreeWarps; ++w) t += s.warp_sum[w];
  __syncthreads();
  return t;
}

// the smallest v whose inclusive prefix sum exceeds y (the last v with weight
// when rounding leaves none): warp 0
__device__ int pick(const double* chunk_sum, const Rest& rest, const Refused* refused, int V, int nchunk, double y) {
  const int lane = threadIdx.x & 31;
  double before = 0.0;
  int ch = -1, last = 0;
  for (int i = 0; i < nchunk; ++i) {
    const double sum = chunk_sum[i];
    if (sum > 0.0) last = i;
    if (before + sum > y) {
      ch = i;
      break;
    }
    before += sum;
  }
  if (ch < 0) {
    // every chunk's sum is at or below y: the last weight of the last chunk that has one
    ch = last;
    before = 0.0;
    y = INFINITY;
  }
  const int lo = ch * kTreeChunk, hi = min(lo + kTreeChunk, V);
  int found = -1, last_v = -1;
  for (int v0 = lo; v0 < hi && found < 0; v0 += 32) {
    const int v = v0 + lane;
    const double w = v < hi && !(refused && refused->holds(v)) ? rest(v) : 0.0;
    double incl = w;
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned past = __ballot_sync(~0u, w > 0.0 && before + incl > y), some = __ballot_sync(~0u, w > 0.0);
    if (past) found = v0 + __ffs(past) - 1;
    if (some) last_v = v0 + 31 - __clz(some);
    before += __shfl_sync(~0u, incl, 31);
  }
  return found >= 0 ? found : last_v;
}

__global__ void __launch_bounds__(kTreeThreads) tree_kernel(TreeParams P) {
  extern __shared__ double chunk_sum[];
  __shared__ TreeShared s;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int start = P.node_start[b], end = P.node_start[b + 1];
  const bool inside = start >= 0 && end >= start && end <= P.total_nodes;
  const bool range = inside && end - start <= P.max_nodes;
  const int n = range ? end - start : 0;
  const int64_t root = static_cast<int64_t>(start) + b;
  int bad = !range;
  for (int i = tid; i < n; i += kTreeThreads) {
    s.tok[i] = P.tokens[start + i];
    s.par[i] = P.parent[start + i];
    s.u[i] = P.u_accept[start + i];
    s.flag[i] = SV_FLAG_UNREACHED;
    s.alpha[i] = 0.f;
    bad |= s.tok[i] < 0 || s.tok[i] >= P.V || s.par[i] < -1 || s.par[i] >= i;
  }
  for (int i = tid; range && i <= n; i += kTreeThreads) {
    s.drow[i] = P.draft_row[root + i];
    bad |= s.drow[i] < -1 || s.drow[i] >= P.draft_rows;
  }
  bad = __syncthreads_or(bad);
  if (!bad) {
    for (int i = tid; i < n; i += kTreeThreads) {
      int depth = 1;
      for (int a = s.par[i]; a >= 0; a = s.par[a]) ++depth;
      bad |= depth > P.max_depth;
      const int d = s.drow[s.par[i] + 1];
      s.px[i] = P.p[(root + 1 + s.par[i]) * P.p_stride + s.tok[i]];
      s.qx[i] = d < 0 ? 1.f : P.q[d * P.q_stride + s.tok[i]];
    }
    bad = __syncthreads_or(bad);
  }

  // the walk: every thread takes the same steps; thread 0 writes what they leave
  int cur = -1, len = 0, refused = 0, tested = 0, offered = 0;  // offered: at cur
  double c = 0.0, Z = 1.0, mass = 0.0;
  for (int i = 0; i < n && !bad; ++i) {
    if (s.par[i] != cur) continue;
    const bool bare = s.drow[cur + 1] < 0;
    const double qx = s.qx[i], px = s.px[i];
    if (!(px >= 0.0 && px < INFINITY && qx >= 0.0 && qx < INFINITY)) {
      bad = 1;
      break;
    }
    double r = bare ? px : fma(-c, qx, px);
    if (bare)
      for (int j = 0; j < i; ++j)
        if (s.par[j] == cur && s.tok[j] == s.tok[i]) r = 0.0;  // offered here before, so refused
    if (r < 0.0) r = 0.0;
    const double w = bare || P.replacement ? 1.0 : fmax(1.0 - mass, qx);
    const double most = qx * Z;
    const bool yes = r > 0.0 && s.u[i] * most <= r * w;
    if (tid == 0) {
      s.alpha[i] = most > 0.0 ? static_cast<float>(fmin(1.0, r * w / most)) : (r > 0.0 ? 1.f : 0.f);
      s.flag[i] = yes ? SV_FLAG_ACCEPT : SV_FLAG_REJECT;
    }
    ++tested;
    ++offered;
    if (yes) {
      if (tid == 0 && P.path) P.path[static_cast<int64_t>(b) * P.max_depth + len] = i;
      if (tid == 0) P.out_tokens[static_cast<int64_t>(b) * (P.max_depth + 1) + len] = s.tok[i];
      ++len;
      cur = i, c = 0.0, Z = 1.0, mass = 0.0, offered = 0;
      continue;
    }
    ++refused;
    mass += qx;
    if (bare) {
      Z -= r;
    } else {
      if (w > 0.0) c = fmin(c + Z / w, 1e30);
      const Rest rest = {P.p + (root + 1 + cur) * P.p_stride, P.q + s.drow[cur + 1] * P.q_stride, c};
      Z = row_sums(s, chunk_sum, rest, nullptr, P.V, P.nchunk);
      if (!(Z < INFINITY)) bad = 1;
    }
  }
  __syncthreads();

  int degenerate = 0;
  if (!bad) {
    const float* p = P.p + (root + 1 + cur) * P.p_stride;
    const bool bare = s.drow[cur + 1] < 0;
    const Refused here = {s, n, cur};
    const Refused* ref = bare ? &here : nullptr;
    Rest rest = {p, bare || c == 0.0 ? nullptr : P.q + s.drow[cur + 1] * P.q_stride, c};
    double total = row_sums(s, chunk_sum, rest, ref, P.V, P.nchunk);
    if (total == 0.0) {
      // nothing is left: the node's own row
      degenerate = 1;
      rest.q = nullptr;
      ref = nullptr;
      total = row_sums(s, chunk_sum, rest, ref, P.V, P.nchunk);
    }
    if (!(total > 0.0 && total < INFINITY)) bad = 1;
    if (!bad && tid < 32) {
      const int v = pick(chunk_sum, rest, ref, P.V, P.nchunk, static_cast<double>(P.u_pick[b]) * total);
      if (tid == 0) P.out_tokens[static_cast<int64_t>(b) * (P.max_depth + 1) + len] = v;
    }
  }
  __syncthreads();
  const int from = bad ? 0 : len;
  for (int i = tid; i <= P.max_depth; i += kTreeThreads) {
    if (i > len || bad) P.out_tokens[static_cast<int64_t>(b) * (P.max_depth + 1) + i] = -1;
    if (P.path && i >= from && i < P.max_depth) P.path[static_cast<int64_t>(b) * P.max_depth + i] = -1;
  }
  for (int i = tid; i < (inside ? end - start : 0); i += kTreeThreads) {
    if (P.accept_prob) P.accept_prob[start + i] = bad ? 0.f : s.alpha[i];
    if (P.flags) P.flags[start + i] = bad ? static_cast<int8_t>(SV_FLAG_INVALID) : s.flag[i];
  }
  if (tid == 0) {
    P.accepted_len[b] = bad ? -1 : len;
    if (P.counters) {
      if (bad) {
        atomicAdd(P.counters + SV_CNT_INVALID, 1ull);
      } else {
        atomicAdd(P.counters + SV_CNT_TESTED, static_cast<unsigned long long>(tested));
        atomicAdd(P.counters + SV_CNT_ACCEPTED, static_cast<unsigned long long>(len));
        atomicAdd(P.counters + SV_CNT_REJECTED, static_cast<unsigned long long>(refused));
        if (degenerate) atomicAdd(P.counters + SV_CNT_DEGENERATE, 1ull);
        if (offered == 0) atomicAdd(P.counters + SV_CNT_BONUS, 1ull);
      }
    }
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
  sv::tree_kernel<<<B, sv::kTreeThreads, P.nchunk * sizeof(double), static_cast<cudaStream_t>(cuda_stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ECUDA;
}
