// Probabilities of logits rows: spec_verify_softmax.
//
//   probs[r, v] = exp((l[r, v] - m_r) / T_r) / sum_w exp((l[r, w] - m_r) / T_r),  m_r = max_w l[r, w]
//
// T_r = 0 is the limit: 1 at the row's first largest logit, 0 elsewhere.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "device_guard.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

constexpr int kSoftThreads = 512;

struct SoftParams {
  const void* x;
  int64_t x_stride;
  float* y;
  int64_t y_stride;
  const float* t_row;
  float t;
  int V;
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// the larger logit, the smaller index among equal ones; a NaN wins over everything
__device__ __forceinline__ void take_larger(float& m, int& at, float om, int oat) {
  const bool nan = om != om;
  if (nan || (m == m && (om > m || (om == m && oat < at)))) {
    m = om;
    at = oat;
  }
}

template <typename T>
__global__ void __launch_bounds__(kSoftThreads) softmax_kernel(SoftParams P) {
  __shared__ float s_m[kSoftThreads / 32];
  __shared__ int s_at[kSoftThreads / 32];
  __shared__ float s_sum[kSoftThreads / 32];
  const int64_t r = blockIdx.x;
  const T* x = static_cast<const T*>(P.x) + r * P.x_stride;
  float* y = P.y + r * P.y_stride;
  const float t = P.t_row ? P.t_row[r] : P.t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = -INFINITY;
  int at = 0x7fffffff;
  for (int v = threadIdx.x; v < P.V; v += kSoftThreads) take_larger(m, at, load_logit(x + v), v);
  for (int o = 16; o; o >>= 1)
    take_larger(m, at, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, at, o));
  if (lane == 0) s_m[warp] = m, s_at[warp] = at;
  __syncthreads();
  m = s_m[0], at = s_at[0];
  for (int w = 1; w < kSoftThreads / 32; ++w) take_larger(m, at, s_m[w], s_at[w]);
  // a NaN, a +inf, every logit -inf, or a temperature that is none: no distribution
  const bool valid = fabsf(m) < INFINITY && t >= 0.f && t < INFINITY;
  const float c = 1.4426950408889634f / t;
  float sum = 0.f;
  if (valid && t > 0.f)
    for (int v = threadIdx.x; v < P.V; v += kSoftThreads) sum += exp2f((load_logit(x + v) - m) * c);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < kSoftThreads / 32; ++w) sum += s_sum[w];
  const float inv = 1.f / sum;
  for (int v = threadIdx.x; v < P.V; v += kSoftThreads) {
    float o = __int_as_float(0x7fffffff);
    if (valid) o = t > 0.f ? exp2f((load_logit(x + v) - m) * c) * inv : (v == at ? 1.f : 0.f);
    y[v] = o;
  }
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
  const sv::SoftParams P = {logits, logits_stride, probs, probs_stride, temperature_per_row, temperature, V};
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (dt == SV_BF16)
    sv::softmax_kernel<__nv_bfloat16><<<rows, sv::kSoftThreads, 0, st>>>(P);
  else
    sv::softmax_kernel<float><<<rows, sv::kSoftThreads, 0, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ECUDA;
}
