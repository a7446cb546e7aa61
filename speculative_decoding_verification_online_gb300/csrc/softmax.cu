// Probabilities of logits rows: spec_verify_softmax.
//
//   probs[r, v] = exp((l[r, v] - m_r) / T_r) / sum_w exp((l[r, w] - m_r) / T_r),  m_r = max_w l[r, w]
//
// T_r = 0 is the limit: 1 at the row's first largest logit, 0 elsewhere.
//
// Bound by memory: every logit read once and every probability written once.  A
// row is a cluster of up to sixteen CTAs, each holding its part of the row in
// registers (32 entries a thread) from the one read to the write.  A thread takes
// the exponentials of its own entries against its own largest, so that one
// exchange of (largest, sum) through the cluster is all that the row needs; the
// last factor exp((largest of the thread - largest of the row) / T) / sum is one
// multiplication an entry.  Parts longer than the registers hold are read twice,
// the second time from L2.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "device_guard.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kSoftThreads = 512;  // of a CTA; rows of up to kSoftShort entries take CTAs of kSoftFew
constexpr int kSoftFew = 128;
constexpr int kSoftHeld = 32;  // entries of a row that a thread keeps
constexpr int kSoftPart = kSoftThreads * kSoftHeld, kSoftShort = kSoftFew * kSoftHeld;
constexpr int kSoftCluster = 16;

struct SoftParams {
  const void* x;
  int64_t x_stride;
  float* y;
  int64_t y_stride;
  const float* t_row;
  float t;
  int V, part;  // part: entries of a row for each CTA, a multiple of 4
};

struct SoftShared {
  float warp_m[kSoftThreads / 32], warp_s[kSoftThreads / 32];
  int warp_at[kSoftThreads / 32];
  float m[kSoftCluster], s[kSoftCluster];
  int at[kSoftCluster];
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ float4 load_logits4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load_logits4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

// Entries lo + 4 (j threads + thread) .. + 3 of a row, or with kVec false lo + (4 j + i) threads + thread; -inf
// beyond the part's end
template <typename T, bool kVec, int kThreads>
__device__ __forceinline__ void load_part(const T* x, int lo, int hi, float (&v)[kSoftHeld]) {
#pragma unroll
  for (int j = 0; j < kSoftHeld / 4; ++j) {
    if constexpr (kVec) {
      const int at = lo + 4 * (j * kThreads + threadIdx.x);
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (at + 4 <= hi) {
        f = load_logits4(x + at);
      } else {
        if (at < hi) f.x = load_logit(x + at);
        if (at + 1 < hi) f.y = load_logit(x + at + 1);
        if (at + 2 < hi) f.z = load_logit(x + at + 2);
      }
      v[4 * j] = f.x, v[4 * j + 1] = f.y, v[4 * j + 2] = f.z, v[4 * j + 3] = f.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = lo + (4 * j + i) * kThreads + threadIdx.x;
        v[4 * j + i] = at < hi ? load_logit(x + at) : -INFINITY;
      }
    }
  }
}

template <bool kVec, int kThreads>
__device__ __forceinline__ void store_part(float* y, int lo, int hi, const float (&v)[kSoftHeld], float scale) {
#pragma unroll
  for (int j = 0; j < kSoftHeld / 4; ++j) {
    if constexpr (kVec) {
      const int at = lo + 4 * (j * kThreads + threadIdx.x);
      if (at + 4 <= hi) {
        *reinterpret_cast<float4*>(y + at) =
            make_float4(v[4 * j] * scale, v[4 * j + 1] * scale, v[4 * j + 2] * scale, v[4 * j + 3] * scale);
      } else {
        if (at < hi) y[at] = v[4 * j] * scale;
        if (at + 1 < hi) y[at + 1] = v[4 * j + 1] * scale;
        if (at + 2 < hi) y[at + 2] = v[4 * j + 2] * scale;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = lo + (4 * j + i) * kThreads + threadIdx.x;
        if (at < hi) y[at] = v[4 * j + i] * scale;
      }
    }
  }
}

__device__ __forceinline__ float largest(const float (&v)[kSoftHeld]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < kSoftHeld; ++i) m = fmaxf(m, v[i]);
  return m;
}

// how much a sum against `from` counts in one against `to` >= from
__device__ __forceinline__ float rescale(float from, float to, float c) {
  return from == to ? 1.f : exp2f((from - to) * c);
}

// v becomes exp((v - m) / T), summed.  With m = -inf (nothing but -inf, or NaN) the terms are 0, or NaN.
__device__ __forceinline__ float exponentials(float (&v)[kSoftHeld], float m, float c) {
  const float ref = m == -INFINITY ? 0.f : m;
  float s[4] = {};
#pragma unroll
  for (int i = 0; i < kSoftHeld; ++i) {
    v[i] = exp2f((v[i] - ref) * c);
    s[i % 4] += v[i];
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// the larger logit, the smaller index among equal ones; a NaN wins over everything
__device__ __forceinline__ void take_larger(float& m, int& at, float om, int oat) {
  const bool nan = om != om;
  if (nan || (m == m && (om > m || (om == m && oat < at)))) {
    m = om;
    at = oat;
  }
}

// T = 0
template <typename T, int kThreads>
__device__ __noinline__ void one_hot(SoftShared& s, const T* x, float* y, int lo, int hi) {
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = -INFINITY;
  int at = 0x7fffffff;
  for (int v = lo + threadIdx.x; v < hi; v += kThreads) take_larger(m, at, load_logit(x + v), v);
  for (int o = 16; o; o >>= 1) take_larger(m, at, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, at, o));
  if (lane == 0) s.warp_m[warp] = m, s.warp_at[warp] = at;
  __syncthreads();
  if (warp == 0) {
    m = lane < kThreads / 32 ? s.warp_m[lane] : -INFINITY;
    at = lane < kThreads / 32 ? s.warp_at[lane] : 0x7fffffff;
    for (int o = 16; o; o >>= 1) take_larger(m, at, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, at, o));
    if (lane < ctas) {
      SoftShared* to = cluster.map_shared_rank(&s, lane);
      to->m[rank] = m, to->at[rank] = at;
    }
  }
  cluster.sync();
  m = s.m[0], at = s.at[0];
  for (int r = 1; r < ctas; ++r) take_larger(m, at, s.m[r], s.at[r]);
  const bool valid = fabsf(m) < INFINITY;
  for (int v = lo + threadIdx.x; v < hi; v += kThreads) y[v] = valid ? (v == at ? 1.f : 0.f) : NAN;
}

template <typename T, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) softmax_kernel(const __grid_constant__ SoftParams P) {
  __shared__ SoftShared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  cluster.barrier_arrive();  // every CTA of the cluster runs before any writes into another
  const int64_t r = blockIdx.x / ctas;
  const T* x = static_cast<const T*>(P.x) + r * P.x_stride;
  float* y = P.y + r * P.y_stride;
  const int lo = min(rank * P.part, P.V), hi = min(lo + P.part, P.V);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float t = P.t_row ? P.t_row[r] : P.t;
  if (t == 0.f) {
    cluster.barrier_wait();
    one_hot<T, kThreads>(s, x, y, lo, hi);
    return;
  }
  // 1.44.. / t overflows below 1e-38, where every logit but the largest has no probability
  const float c = fminf(1.4426950408889634f / t, 3.0e38f);
  const bool held = P.part <= kThreads * kSoftHeld;
  float v[kSoftHeld];
  float m, sum;
  if (held) {
    load_part<T, kVec, kThreads>(x, lo, hi, v);
    m = largest(v);
    sum = exponentials(v, m, c);
  } else {
    m = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int at = lo; at < hi; at += kThreads * kSoftHeld) {
      load_part<T, kVec, kThreads>(x, at, hi, v);
      const float mv = largest(v), to = fmaxf(m, mv), sv = exponentials(v, mv, c);
      sum = sum * rescale(m, to, c) + sv * rescale(mv, to, c);
      m = to;
    }
  }
  const float mine = m;
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  sum *= rescale(mine, m, c);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (lane == 0) s.warp_m[warp] = m, s.warp_s[warp] = sum;
  __syncthreads();
  cluster.barrier_wait();
  if (warp == 0) {
    const float wm = lane < kThreads / 32 ? s.warp_m[lane] : -INFINITY;
    float bm = wm, bs = lane < kThreads / 32 ? s.warp_s[lane] : 0.f;
    for (int o = 16; o; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, o));
    bs *= rescale(wm, bm, c);
    for (int o = 16; o; o >>= 1) bs += __shfl_xor_sync(~0u, bs, o);
    if (lane < ctas) {
      SoftShared* to = cluster.map_shared_rank(&s, lane);
      to->m[rank] = bm, to->s[rank] = bs;
    }
  }
  cluster.sync();
  m = s.m[0];
  for (int i = 1; i < ctas; ++i) m = fmaxf(m, s.m[i]);
  sum = 0.f;
  for (int i = 0; i < ctas; ++i) sum += s.s[i] * rescale(s.m[i], m, c);
  // a NaN, a +inf and a row of nothing but -inf have made the sum NaN or 0, and the row NaN
  const float inv = t > 0.f && t < INFINITY ? 1.f / sum : NAN;
  if (held) {
    store_part<kVec, kThreads>(y, lo, hi, v, rescale(mine, m, c) * inv);
  } else {
#pragma unroll 1
    for (int at = lo; at < hi; at += kThreads * kSoftHeld) {
      load_part<T, kVec, kThreads>(x, at, hi, v);
      exponentials(v, m, c);
      store_part<kVec, kThreads>(y, at, hi, v, inv);
    }
  }
}

template <int kThreads>
auto softmax_variant(sv_dtype dt, bool vec) {
  if (dt == SV_BF16)
    return vec ? softmax_kernel<__nv_bfloat16, true, kThreads> : softmax_kernel<__nv_bfloat16, false, kThreads>;
  return vec ? softmax_kernel<float, true, kThreads> : softmax_kernel<float, false, kThreads>;
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_verify_softmax(const void* logits, sv_dtype dt, int64_t logits_stride, int rows, int V,
                                         float temperature, const float* temperature_per_row, float* probs,
                                         int64_t probs_stride, int device, void* cuda_stream) {
  if (dt != SV_F32 && dt != SV_BF16) return SV_EINVAL;
  if (rows < 0 || V < 1) return SV_EINVAL;
  if (V > SV_MAX_V) return SV_EUNSUPPORTED;
  if (!temperature_per_row && !(temperature >= 0.f && std::isfinite(temperature))) return SV_EINVAL;
  if (rows == 0) return SV_OK;
  if (!logits || !probs) return SV_EINVAL;
  const size_t es = dt == SV_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) % es || reinterpret_cast<uintptr_t>(probs) % 4 ||
      reinterpret_cast<uintptr_t>(temperature_per_row) % 4)
    return SV_EINVAL;
  if (rows > 1 && (logits_stride < 0 || probs_stride < V)) return SV_EINVAL;
  sv::DeviceGuard g(device);
  if (!g.ok) return SV_ECUDA;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return SV_ECUDA;
  // enough CTAs a row to hold it, and more while the rows leave room beside two CTAs an SM
  int ctas = 1;
  while (ctas < sv::kSoftCluster && (V > ctas * sv::kSoftPart || (static_cast<int64_t>(rows) * ctas * 2 <= 2ll * sms &&
                                                                  V > ctas * sv::kSoftThreads * 4)))
    ctas *= 2;
  if (static_cast<int64_t>(rows) * ctas > 0x7fffffff) return SV_EUNSUPPORTED;
  const int part = ((V + ctas - 1) / ctas + 3) / 4 * 4;
  const sv::SoftParams P = {logits, logits_stride, probs, probs_stride, temperature_per_row, temperature, V, part};
  const bool vec = reinterpret_cast<uintptr_t>(logits) % (4 * es) == 0 && reinterpret_cast<uintptr_t>(probs) % 16 == 0 &&
                   (rows == 1 || (logits_stride % 4 == 0 && probs_stride % 4 == 0));
  const auto kernel = ctas == 1 && V <= sv::kSoftShort ? sv::softmax_variant<sv::kSoftFew>(dt, vec)
                                                       : sv::softmax_variant<sv::kSoftThreads>(dt, vec);
  // sixteen CTAs are more than the portable eight
  if (ctas > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return SV_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * ctas));
  cfg.blockDim = dim3(ctas == 1 && V <= sv::kSoftShort ? sv::kSoftFew : sv::kSoftThreads);
  cfg.stream = static_cast<cudaStream_t>(cuda_stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? SV_OK : SV_ECUDA;
}
