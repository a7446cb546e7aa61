// Penalties, biases and masks on logits rows: spec_verify_penalties.
//
//   z = seen ? (l > 0 ? l / rep : l rep) : l;  z -= freq n + (n > 0 ? pres : 0);  z += bias;  masked: -inf
//
// n counts a token in the sequence's history and among the row's own drafted path.
//
// A CTA takes a range of the vocabulary for one sequence.  It counts the history's
// tokens of its range in shared memory once for all of the sequence's rows, and keeps
// a list of the tokens that occur: only they (and the path's) change, so that in place
// and without a mask nothing else of a row is touched.  Into another tensor, or under
// a mask, a row is first copied in straight 16-byte vectors and its listed tokens are
// put right after that.  Counts are integers: the result does not depend on the order
// of the atomics.
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
constexpr int kPenLeast = 1024;      // and at least
constexpr int kAhead = 4;
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
  int in_place, x_vec, y_vec;
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }

// eight neighbouring logits at a multiple of 16 bytes, as they lie in memory
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p + 4));
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
};
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

struct PenaltyShared {
  int listed, bad;
  int32_t token[SV_MAX_NODES], parent[SV_MAX_NODES];
  uint16_t path[kPenWarps][SV_MAX_NODES];  // a row's path tokens in the range, counted from its start
};

template <typename X, typename Y>
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
  if (threadIdx.x == 0) s.listed = 0;
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
    auto mark = [&](int i, uint32_t was) {
      if (was == 0) list[atomicAdd(&s.listed, 1)] = static_cast<uint16_t>(i);
    };
    const int asked = P.prompt_len ? min(max(P.prompt_len[b], 0), len) : 0;
    const int32_t* h = P.history + b * P.history_stride;
    for (int i = threadIdx.x; i < len; i += kPenThreads) {
      const unsigned at = static_cast<unsigned>(h[i]) - static_cast<unsigned>(lo);
      if (at < static_cast<unsigned>(n)) {
        if (i >= asked)
          mark(at, atomicAdd(&table[at], 1u));
        else if (P.repetition)
          mark(at, atomicOr(&table[at], kAsked));
      }
    }
    for (int i = bias_lo + threadIdx.x; i < bias_hi; i += kPenThreads) {
      const unsigned at = static_cast<unsigned>(P.bias_tokens[i]) - static_cast<unsigned>(lo);
      if (at < static_cast<unsigned>(n)) {
        atomicMax(&place[at], i);
        mark(at, atomicOr(&table[at], kBiased));
      }
    }
  }
  __syncthreads();
  const int listed = s.listed, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
      const bool vec = P.x_vec && P.y_vec;
      const int whole = vec ? from + (to - from) / 8 * 8 : from;
      // runs of eight, kAhead of a lane's on their way at once
#pragma unroll 1
      for (int v0 = from + 8 * lane; v0 < whole; v0 += 256 * kAhead) {
        uint32_t bits[kAhead];
        Raw8<X> raw[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int v = v0 + 256 * j;
          bits[j] = v < whole ? mask ? mask[v / 32] >> (v % 32) & 0xffu : 0xffu : 0u;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (bits[j] != 0 && !(P.in_place && bits[j] == 0xffu)) raw[j].load(x + v0 + 256 * j);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int v = v0 + 256 * j;
          if (v >= whole || (P.in_place && bits[j] == 0xffu)) continue;
          float e[8];
          raw[j].values(e);
#pragma unroll
          for (int k = 0; k < 8; ++k) e[k] = bits[j] >> k & 1u ? e[k] : -INFINITY;
          store8(y + v, e);
        }
      }
      for (int v = whole + lane; v < to; v += 32) {
        const bool ok = allowed(v);
        if (!ok || !P.in_place) store_logit(y + v, ok ? load_logit(x + v) : -INFINITY);
      }
      __syncwarp();
    }
    auto put = [&](int v, uint32_t word, int count) {
      float z = load_logit(x + v);
      if (count > 0 || (word & kAsked)) z = z > 0.f ? z / rep : z * rep;
      z -= freq * static_cast<float>(count);
      if (count > 0) z -= pres;
      if (word & kBiased) z += P.bias_values[place[v]];
      store_logit(y + v, z);
    };
    for (int e = lane; e < listed; e += 32) {
      const int v = list[e];
      if (v < from || v >= to || !allowed(v)) continue;
      const uint32_t word = table[v];
      int count = static_cast<int>(word & kCount);
      for (int k = 0; k < on_path; ++k) count += path[k] == v;
      put(v, word, count);
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
      if (first) put(v, 0u, count);
    }
  }
}

template <typename X>
auto penalties_variant(sv_dtype out) {
  return out == SV_BF16 ? penalties_kernel<X, __nv_bfloat16> : penalties_kernel<X, float>;
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
  // (ranges below the widest are for fewer CTAs than this)
  if (static_cast<int64_t>((V + sv::kPenRange - 1) / sv::kPenRange) * B > INT32_MAX) return SV_EUNSUPPORTED;
  sv::DeviceGuard g(device);
  if (!g.ok) return SV_ECUDA;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return SV_ECUDA;
  // as wide a range as still gives every SM two CTAs
  int range = sv::kPenRange;
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
  P.x_vec = reinterpret_cast<uintptr_t>(logits) % 16 == 0 && (rows == 1 || logits_stride % (16 / static_cast<int64_t>(es)) == 0);
  P.y_vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && (rows == 1 || out_stride % (16 / static_cast<int64_t>(eo)) == 0);
  const auto kernel = dt == SV_BF16 ? sv::penalties_variant<__nv_bfloat16>(out_dt) : sv::penalties_variant<float>(out_dt);
  const size_t smem = static_cast<size_t>(range) * ((bias_start ? 8 : 4) + 2);
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return SV_ECUDA;
  return sv::launch_waiting(kernel, static_cast<unsigned>(P.ranges) * static_cast<unsigned>(B), sv::kPenThreads, smem, 1, static_cast<cudaStream_t>(cuda_stream), P) == cudaSuccess
             ? SV_OK
             : SV_ECUDA;
}
