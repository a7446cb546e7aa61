// Penalties, biases and masks on logits rows: spec_verify_penalties.
//
//   z = seen ? (l > 0 ? l / rep : l rep) : l;  z -= freq n + (n > 0 ? pres : 0);  z += bias;  masked: -inf
//
// n counts a token in the sequence's history and among the row's own drafted path.
//
// A CTA takes a range of the vocabulary for one sequence.  It counts the history's
// tokens of its range in shared memory once for all of the sequence's rows, and makes
// a list of the tokens that occur: only they (and the path's) change, so that in place
// and without a mask nothing else of a row is touched.  Into another tensor, or under
// a mask, a row is first copied in straight 16-byte vectors and its listed tokens are
// put right after that.  Counts are integers: the result does not depend on the order
// of the atomics.
//
// In place it is a chain of waits: five rows of 32000 tokens after a history of 256 take 5.4 us, 64
// sequences of six rows of 128256 after up to 4096 tokens 15.7 us (counting, then a load and a store for
// each listed token and row, in two waves of CTAs: registers and shared memory leave four an SM).
// Copied rows wait for memory: 32 trees of up to 21 nodes under masks, 151936 tokens from bf16 to
// fp32, 106 us, 4.7 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "entry.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

constexpr int kPenWarps = 8, kPenThreads = 32 * kPenWarps;
constexpr int kPenRange = 8192;      // tokens of a CTA at most
constexpr int kPenCopied = 4096;     // where rows are copied
constexpr int kPenLeast = 1024;      // and at least
constexpr int kPenMostShared = kPenRange * (4 + 4 + 2);  // bytes of a table, of places of biases, of a list
constexpr int kPenLong = 8192;       // histories from here on have their list in order
constexpr int kSingle = 8;           // logits of a lane on their way at once where they are not loaded in runs
constexpr int kTokens = 16;          // of the history on a thread's way at once
constexpr int kChanges = 4;          // listed tokens of a lane at once
constexpr uint32_t kAsked = 1u << 31, kBiased = 1u << 30, kCount = kBiased - 1;

struct PenaltyParams {
  const void* x;
  void* y;
  int64_t x_stride, y_stride;
  int V, range, ranges;
  const int32_t* history;
  int64_t history_stride;
  int history_cap;
  const int32_t *history_len, *prompt_len, *tokens, *parent, *node_start;
  int total, max_nodes;
  const float *repetition, *frequency, *presence;
  const int32_t *bias_start, *bias_tokens;
  const float* bias_values;
  int total_biases;
  const int32_t* mask;
  int64_t mask_stride;
  int mask_rows;
  const int32_t* mask_row;
  int in_place;
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }

// A lane's run of neighbouring logits, as many as 16 bytes hold of the wider of the two types: lanes side by side then read
// and write whole sectors.
template <typename X, typename Y>
constexpr int kRun = sizeof(X) == 4 || sizeof(Y) == 4 ? 4 : 8;

template <typename X, int kCount>
struct Raw;
template <>
struct Raw<float, 4> {
  float4 a;
  __device__ __forceinline__ void load(const float* p) { a = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void values(float (&v)[4]) const { v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w; }
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void values(float (&v)[4]) const {
    v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xffff0000u);
  }
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
};
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void store_run(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_run(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void store_run(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

struct PenaltyShared {
  int listed[kPenWarps];  // of a warp's part of the table
  int32_t token[SV_MAX_NODES], parent[SV_MAX_NODES];
  uint16_t path[kPenWarps][SV_MAX_NODES];  // a row's path tokens in the range, counted from its start
};

// The list of the tokens that occur, in order: a warp counts those of its part of the table, then writes them.  Neighbouring lanes
// then come to neighbouring logits: 64 histories of 24000 tokens 67 us, 111 us listed as they come; of 3000 tokens 19.1 and
// 15.6 us.
__device__ __forceinline__ int list_in_order(const uint32_t* table, uint16_t* list, int range, int* counts) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = range / kPenWarps;
  const uint4* const words = reinterpret_cast<const uint4*>(table + warp * share);
  auto there = [](uint4 w) { return (w.x != 0) + (w.y != 0) + (w.z != 0) + (w.w != 0); };
  int mine = 0;
  for (int i = lane; i < share / 4; i += 32) mine += there(words[i]);
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
  if (lane == 0) counts[warp] = mine;
  __syncthreads();
  int listed = 0, put_at = 0;
  for (int w = 0; w < kPenWarps; ++w) {
    if (w == warp) put_at = listed;
    listed += counts[w];
  }
  if (mine > 0)
    for (int i = lane; i < share / 4; i += 32) {
      const uint4 w = words[i];
      int sum = there(w);
      const int here = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += u;
      }
      int to = put_at + sum - here;
      const int first = warp * share + 4 * i;
      if (w.x) list[to++] = static_cast<uint16_t>(first);
      if (w.y) list[to++] = static_cast<uint16_t>(first + 1);
      if (w.z) list[to++] = static_cast<uint16_t>(first + 2);
      if (w.w) list[to] = static_cast<uint16_t>(first + 3);
      put_at += __shfl_sync(~0u, sum, 31);
    }
  __syncthreads();
  return listed;
}

template <typename X, typename Y, bool kInOrder>
__global__ void __launch_bounds__(kPenThreads) penalties_kernel(const __grid_constant__ PenaltyParams P) {
  extern __shared__ __align__(16) uint32_t table[];  // [range] counts and marks, then places of biases, then the list
  __shared__ PenaltyShared s;
  wait_for_stream();
  const int b = blockIdx.x / P.ranges, lo = blockIdx.x % P.ranges * P.range, n = min(P.range, P.V - lo);
  const int start = P.node_start[b], end = P.node_start[b + 1], len = P.history_len[b];
  if (len < 0 || start < 0 || end < start || end > P.total || end - start > P.max_nodes) return;
  const int nodes = end - start;
  const int64_t row0 = static_cast<int64_t>(start) + b;
  int32_t* place = reinterpret_cast<int32_t*>(table + P.range);
  uint16_t* list = reinterpret_cast<uint16_t*>(table + (P.bias_start ? 2 : 1) * P.range);
  const float rep = P.repetition ? P.repetition[b] : 1.f, freq = P.frequency ? P.frequency[b] : 0.f,
              pres = P.presence ? P.presence[b] : 0.f;
  const int bias_lo = P.bias_start ? P.bias_start[b] : 0, bias_hi = P.bias_start ? P.bias_start[b + 1] : 0;
  const bool fine = len <= P.history_cap && rep > 0.f && rep < INFINITY && fabsf(freq) < INFINITY && fabsf(pres) < INFINITY &&
                    bias_lo >= 0 && bias_hi >= bias_lo && bias_hi <= P.total_biases;
  if (threadIdx.x == 0) s.listed[0] = 0;
  for (int i = threadIdx.x; i < P.range; i += kPenThreads) {
    table[i] = 0;
    if (P.bias_start) place[i] = -1;
  }
  for (int i = threadIdx.x; i < nodes; i += kPenThreads) {
    s.token[i] = P.tokens[start + i];
    s.parent[i] = P.parent ? P.parent[start + i] : i - 1;
  }
  __syncthreads();
  if (fine) {
    const int asked = P.prompt_len ? min(max(P.prompt_len[b], 0), len) : 0;
    const int32_t* h = P.history + b * P.history_stride;
    // the first one to come to a token puts it on the list, where the list is not made afterwards
    auto mark = [&](int i, uint32_t was) {
      if (was == 0) list[atomicAdd(&s.listed[0], 1)] = static_cast<uint16_t>(i);
    };
    // (where nothing asks for the prompt's tokens they are left out)
    for (int i0 = (P.repetition ? 0 : asked) + threadIdx.x; i0 < len; i0 += kPenThreads * kTokens) {
      int32_t token[kTokens];
#pragma unroll
      for (int k = 0; k < kTokens; ++k) token[k] = i0 + k * kPenThreads < len ? h[i0 + k * kPenThreads] : -1;
#pragma unroll
      for (int k = 0; k < kTokens; ++k) {
        const unsigned at = static_cast<unsigned>(token[k]) - static_cast<unsigned>(lo);
        if (token[k] < 0 || at >= static_cast<unsigned>(n)) continue;
        const bool said = i0 + k * kPenThreads >= asked;
        if constexpr (kInOrder) {
          if (said)
            atomicAdd(&table[at], 1u);
          else
            atomicOr(&table[at], kAsked);
        } else {
          mark(at, said ? atomicAdd(&table[at], 1u) : atomicOr(&table[at], kAsked));
        }
      }
    }
    for (int i = bias_lo + threadIdx.x; i < bias_hi; i += kPenThreads) {
      const unsigned at = static_cast<unsigned>(P.bias_tokens[i]) - static_cast<unsigned>(lo);
      if (at < static_cast<unsigned>(n)) {
        atomicMax(&place[at], i);
        const uint32_t was = atomicOr(&table[at], kBiased);
        if constexpr (!kInOrder) mark(at, was);
        (void)was;
      }
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int listed;
  if constexpr (kInOrder)
    listed = list_in_order(table, list, P.range, s.listed);
  else
    listed = s.listed[0];
  // a warp takes a row, or part of one where there are fewer rows than warps
  const int rows = nodes + 1, parts = max(1, kPenWarps / rows);
  const int step = ((n + parts - 1) / parts + 255) / 256 * 256;
  for (int u = warp; u < rows * parts; u += kPenWarps) {
    const int i = u / parts, from = min(n, u % parts * step), to = min(n, from + step);
    const int64_t row = row0 + i;
    const X* x = static_cast<const X*>(P.x) + row * P.x_stride + lo;
    Y* y = static_cast<Y*>(P.y) + row * P.y_stride + lo;
    // the path, node by node upwards: its tokens of this range
    int on_path = 0;
    bool good = fine;
    uint16_t* path = s.path[warp];
    __syncwarp();
    for (int cur = i - 1; cur >= 0;) {
      const unsigned at = static_cast<unsigned>(s.token[cur]) - static_cast<unsigned>(lo);
      if (at < static_cast<unsigned>(n)) {
        if (lane == 0) path[on_path] = static_cast<uint16_t>(at);
        ++on_path;
      }
      const int up = s.parent[cur];
      if (up < -1 || up >= cur) {
        good = false;
        break;
      }
      cur = up;
    }
    __syncwarp();
    int m = -1;
    if (P.mask) {
      m = P.mask_row ? P.mask_row[row] : static_cast<int>(row);
      if (m < -1 || m >= P.mask_rows) good = false;
    }
    if (!good) {
      for (int v = from + lane; v < to; v += 32) store_logit(y + v, NAN);
      continue;
    }
    const uint32_t* mask = m >= 0 ? reinterpret_cast<const uint32_t*>(P.mask) + m * P.mask_stride + lo / 32 : nullptr;
    auto allowed = [&](int v) { return !mask || (mask[v / 32] >> (v % 32) & 1u); };
    if (mask || !P.in_place) {
      // runs at multiples of their size, where x and y come to them together; what is in front of them and behind them (or
      // all) entry by entry
      constexpr int kLen = kRun<X, Y>, kStep = 32 * kLen, kAhead = 32 / kLen;
      constexpr uint32_t kAll = (1u << kLen) - 1u;
      const int front = static_cast<int>((0 - reinterpret_cast<uintptr_t>(x + from)) % (kLen * sizeof(X)) / sizeof(X));
      const bool together = reinterpret_cast<uintptr_t>(y + from + front) % (kLen * sizeof(Y)) == 0;
      const int begin = min(to, from + front), whole = together ? begin + (to - begin) / kLen * kLen : begin;
      const bool apart = begin % kLen != 0;  // a run's bits may be in two words
      uint32_t bits[kAhead], next[kAhead];  // of the runs, and of the next ones
      auto look = [&](int v0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int v = v0 + kStep * j;
          next[j] = v < whole ? kAll : 0u;
          if (mask && v < whole) {
            next[j] &= mask[v / 32] >> v % 32;
            if (apart && v % 32 > 32 - kLen) next[j] |= mask[v / 32 + 1] << (32 - v % 32) & kAll;
          }
        }
      };
      look(begin + kLen * lane);
#pragma unroll 1
      for (int v0 = begin + kLen * lane; v0 < whole; v0 += kStep * kAhead) {
        Raw<X, kLen> raw[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) bits[j] = next[j];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (bits[j] != 0 && !(P.in_place && bits[j] == kAll)) raw[j].load(x + v0 + kStep * j);
        look(v0 + kStep * kAhead);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int v = v0 + kStep * j;
          if (v >= whole || (P.in_place && bits[j] == kAll)) continue;
          float e[kLen];
          raw[j].values(e);
#pragma unroll
          for (int k = 0; k < kLen; ++k) e[k] = bits[j] >> k & 1u ? e[k] : -INFINITY;
          store_run(y + v, e);
        }
      }
      auto single = [&](int lo_, int hi_) {
#pragma unroll 1
        for (int v0 = lo_ + lane; v0 < hi_; v0 += 32 * kSingle) {
          float e[kSingle];
          bool ok[kSingle];
#pragma unroll
          for (int j = 0; j < kSingle; ++j) {
            const int v = v0 + 32 * j;
            ok[j] = v < hi_ && allowed(v);
            e[j] = ok[j] && !P.in_place ? load_logit(x + v) : -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < kSingle; ++j)
            if (v0 + 32 * j < hi_ && !(ok[j] && P.in_place)) store_logit(y + v0 + 32 * j, e[j]);
        }
      };
      single(from, begin);
      single(whole, to);
      __syncwarp();
    }
    auto put = [&](int v, float z, uint32_t word, int count) {
      if (count > 0 || (word & kAsked)) z = z > 0.f ? z / rep : z * rep;
      z -= freq * static_cast<float>(count);
      if (count > 0) z -= pres;
      if (word & kBiased) z += P.bias_values[place[v]];
      store_logit(y + v, z);
    };
#pragma unroll 1
    for (int e0 = lane; e0 < listed; e0 += 32 * kChanges) {
      int v[kChanges];
      uint32_t word[kChanges];
      float z[kChanges];
#pragma unroll
      for (int j = 0; j < kChanges; ++j) {
        const int e = e0 + 32 * j;
        v[j] = e < listed ? list[e] : -1;
        if (v[j] < from || v[j] >= to || !allowed(v[j])) v[j] = -1;
        word[j] = v[j] >= 0 ? table[v[j]] : 0u;
        z[j] = v[j] >= 0 ? load_logit(x + v[j]) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kChanges; ++j) {
        int count = static_cast<int>(word[j] & kCount);
        for (int k = 0; k < on_path; ++k) count += path[k] == v[j];
        if (v[j] >= 0) put(v[j], z[j], word[j], count);
      }
    }
    for (int k = lane; k < on_path; k += 32) {
      const int v = path[k];
      if (v < from || v >= to || table[v] != 0 || !allowed(v)) continue;
      int count = 0;
      bool first = true;
      for (int j = 0; j < on_path; ++j)
        if (path[j] == v) {
          ++count;
          if (j < k) first = false;
        }
      if (first) put(v, load_logit(x + v), 0u, count);
    }
  }
}

template <bool kInOrder>
auto penalties_variant(sv_dtype in, sv_dtype out) {
  if (in == SV_BF16)
    return out == SV_BF16 ? penalties_kernel<__nv_bfloat16, __nv_bfloat16, kInOrder> : penalties_kernel<__nv_bfloat16, float, kInOrder>;
  return out == SV_BF16 ? penalties_kernel<float, __nv_bfloat16, kInOrder> : penalties_kernel<float, float, kInOrder>;
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_verify_penalties(const void* logits, sv_dtype dt, int64_t logits_stride, void* out, sv_dtype out_dt,
                                           int64_t out_stride, int V, const int32_t* history, int64_t history_stride,
                                           int history_cap, const int32_t* history_len, const int32_t* prompt_len,
                                           const int32_t* node_tokens, const int32_t* parent, const int32_t* node_start,
                                           int B, int total_nodes, int max_nodes, const float* repetition,
                                           const float* frequency, const float* presence, const int32_t* bias_start,
                                           const int32_t* bias_tokens, const float* bias_values, int total_biases,
                                           const int32_t* mask, int64_t mask_stride, int mask_rows, const int32_t* mask_row,
                                           int device, void* cuda_stream) {
  if ((dt != SV_F32 && dt != SV_BF16) || (out_dt != SV_F32 && out_dt != SV_BF16)) return SV_EINVAL;
  if (V < 1 || B < 0 || total_nodes < 0 || max_nodes < 0 || history_cap < 0 || total_biases < 0 || mask_rows < 0)
    return SV_EINVAL;
  if (V > SV_MAX_V || max_nodes > SV_MAX_NODES || history_cap >= (1 << 30)) return SV_EUNSUPPORTED;
  if (B == 0) return SV_OK;
  if (static_cast<int64_t>(total_nodes) + B > INT32_MAX) return SV_EUNSUPPORTED;
  const int rows = total_nodes + B, words = (V + 31) / 32;
  if (!logits || !out || !history_len || !node_start || (history_cap > 0 && !history) || (total_nodes > 0 && !node_tokens))
    return SV_EINVAL;
  if (bias_start && total_biases > 0 && (!bias_tokens || !bias_values)) return SV_EINVAL;
  const size_t es = dt == SV_BF16 ? 2 : 4, eo = out_dt == SV_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) % es || reinterpret_cast<uintptr_t>(out) % eo) return SV_EINVAL;
  for (const void* p : {static_cast<const void*>(history), static_cast<const void*>(history_len),
                        static_cast<const void*>(prompt_len), static_cast<const void*>(node_tokens),
                        static_cast<const void*>(parent), static_cast<const void*>(node_start),
                        static_cast<const void*>(repetition), static_cast<const void*>(frequency),
                        static_cast<const void*>(presence), static_cast<const void*>(bias_start),
                        static_cast<const void*>(bias_tokens), static_cast<const void*>(bias_values),
                        static_cast<const void*>(mask), static_cast<const void*>(mask_row)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SV_EINVAL;
  if (rows > 1 && (logits_stride < 0 || out_stride < V)) return SV_EINVAL;
  if (B > 1 && history_stride < 0) return SV_EINVAL;
  if (mask && ((mask_rows > 1 && mask_stride < words) || (!mask_row && mask_rows < rows))) return SV_EINVAL;
  const bool in_place = logits == out && dt == out_dt && (rows == 1 || logits_stride == out_stride);
  if (!in_place && sv::sure_to_overlap({logits, static_cast<int64_t>(es), V, logits_stride, rows, 0, 1},
                                       {out, static_cast<int64_t>(eo), V, out_stride, rows, 0, 1}))
    return SV_EINVAL;
  // (narrower ranges than these are for fewer CTAs than this)
  if (static_cast<int64_t>((V + sv::kPenCopied - 1) / sv::kPenCopied) * B > INT32_MAX) return SV_EUNSUPPORTED;
  sv::DeviceGuard g(device);
  if (!g.ok) return SV_ECUDA;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return SV_ECUDA;
  // As wide a range as still gives every SM two CTAs.  Rows that are copied have narrower ones, whose tables leave room for
  // more warps (trees of 32 sequences under masks 148 us with 8192, 105 with 4096; 64 chains in place 15.6, 20.9).
  int range = mask || !in_place ? sv::kPenCopied : sv::kPenRange;
  while (range > sv::kPenLeast && static_cast<int64_t>((V + range - 1) / range) * B < 2 * sms) range /= 2;
  sv::PenaltyParams P = {};
  P.x = logits, P.y = out;
  P.x_stride = logits_stride, P.y_stride = out_stride;
  P.V = V, P.range = range, P.ranges = (V + range - 1) / range;
  P.history = history, P.history_stride = history_stride, P.history_cap = history_cap;
  P.history_len = history_len, P.prompt_len = prompt_len, P.tokens = node_tokens, P.parent = parent, P.node_start = node_start;
  P.total = total_nodes, P.max_nodes = max_nodes;
  P.repetition = repetition, P.frequency = frequency, P.presence = presence;
  P.bias_start = bias_start, P.bias_tokens = bias_tokens, P.bias_values = bias_values, P.total_biases = total_biases;
  P.mask = mask, P.mask_stride = mask_stride, P.mask_rows = mask_rows, P.mask_row = mask_row;
  P.in_place = in_place;
  const auto kernel = history_cap >= sv::kPenLong ? sv::penalties_variant<true>(dt, out_dt) : sv::penalties_variant<false>(dt, out_dt);
  const size_t smem = static_cast<size_t>(range) * ((bias_start ? 8 : 4) + 2);
  // (always the same limit: one for this call alone could be lowered by another host thread in front of the launch)
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sv::kPenMostShared) != cudaSuccess)
    return SV_ECUDA;
  return sv::launch_waiting(kernel, static_cast<unsigned>(P.ranges) * static_cast<unsigned>(B), sv::kPenThreads, smem, 1, static_cast<cudaStream_t>(cuda_stream), P) == cudaSuccess
             ? SV_OK
             : SV_ECUDA;
}
