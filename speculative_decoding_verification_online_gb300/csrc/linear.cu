// Grouped matrix products with an epilogue: spec_verify_linear.
//
//   y[g, m, n] = act(sum_k x[g, m, k] w[g, n, k] + bias[g, n]) + residual[g, m, n]
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "device_guard.cuh"
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
  float cap;
};

__device__ __forceinline__ float load_either(const void* p, int64_t i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ float activate(float z, int act, float cap) {
  switch (act) {
    case SV_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case SV_ACT_SILU: return z / (1.f + expf(-z));
    case SV_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678f));
    case SV_ACT_GELU_TANH: return 0.5f * z * (1.f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
    case SV_ACT_SOFTCAP: return cap * tanhf(z / cap);
    default: return z;
  }
}

// The sum's way out: the one rounding to bf16, where y is bf16, is the last step.
__device__ __forceinline__ void finish_value(const LinearParams& P, int g, int64_t m, int64_t n, float z) {
  if (P.bias) z += load_either(P.bias, g * P.b_group + n, P.bias_bf16);
  z = activate(z, P.act, P.cap);
  if (P.res) z += load_either(P.res, g * P.r_group + m * P.r_row + n, P.res_bf16);
  const int64_t at = g * P.y_group + m * P.y_row + n;
  if (P.y_bf16)
    static_cast<__nv_bfloat16*>(P.y)[at] = __float2bfloat16(z);
  else
    static_cast<float*>(P.y)[at] = z;
}

constexpr int kPlainTile = 64, kPlainK = 32;

// Any sizes, strides and alignment: 64 x 64 tiles of y by 256 threads, each
// 4 x 4 sums in fp32, elements loaded one by one.
__global__ void __launch_bounds__(256) plain_kernel(LinearParams P) {
  __shared__ float sx[kPlainK][kPlainTile + 1], sw[kPlainK][kPlainTile + 1];
  const int64_t tn = (P.N + kPlainTile - 1) / kPlainTile, tm = (P.M + kPlainTile - 1) / kPlainTile;
  for (int64_t tile = blockIdx.x; tile < tn * tm * P.groups; tile += gridDim.x) {
    const int g = static_cast<int>(tile / (tn * tm));
    const int64_t m0 = tile / tn % tm * kPlainTile, n0 = tile % tn * kPlainTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < P.K; k0 += kPlainK) {
      for (int i = threadIdx.x; i < kPlainK * kPlainTile; i += 256) {
        const int kk = i % kPlainK, r = i / kPlainK;
        const bool in = k0 + kk < P.K;
        sx[kk][r] = in && m0 + r < P.M ? __bfloat162float(P.x[g * P.x_group + (m0 + r) * P.x_row + k0 + kk]) : 0.f;
        sw[kk][r] = in && n0 + r < P.N ? __bfloat162float(P.w[g * P.w_group + (n0 + r) * P.w_row + k0 + kk]) : 0.f;
      }
      __syncthreads();
#pragma unroll 8
      for (int kk = 0; kk < kPlainK; ++kk)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) acc[i][j] += sx[kk][ty + 16 * i] * sw[kk][tx + 16 * j];
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j)
        if (m0 + ty + 16 * i < P.M && n0 + tx + 16 * j < P.N)
          finish_value(P, g, m0 + ty + 16 * i, n0 + tx + 16 * j, acc[i][j]);
  }
}

bool valid_dtype(int d) { return d == SV_F32 || d == SV_BF16; }
bool aligned_to(const void* p, int d) { return reinterpret_cast<uintptr_t>(p) % (d == SV_BF16 ? 2 : 4) == 0; }

// rows of N values at g * group + m * row that never share a place
bool rows_apart(int64_t row, int64_t group, int64_t M, int64_t groups, int64_t N) {
  if (M == 1) return groups == 1 || group >= N;
  if (groups == 1) return row >= N;
  if (row <= group) return row >= N && group >= row * (M - 1) + N;
  return group >= N && row >= group * (groups - 1) + N;
}

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
  if (act == SV_ACT_SOFTCAP && !(cap > 0.f && std::isfinite(cap))) return SV_EINVAL;
  if (x_row < 0 || x_group < 0 || w_row < 0 || w_group < 0 || bias_group < 0 || residual_row < 0 ||
      residual_group < 0 || y_row < 0 || y_group < 0)
    return SV_EINVAL;
  for (const int64_t stride : {x_row, x_group, w_row, w_group, bias_group, residual_row, residual_group, y_row, y_group})
    if (stride >= (int64_t{1} << 40)) return SV_EUNSUPPORTED;
  if (groups == 0 || M == 0 || N == 0) return SV_OK;
  if (!y || (K > 0 && (!x || !w))) return SV_EINVAL;
  if (!sv::aligned_to(x, SV_BF16) || !sv::aligned_to(w, SV_BF16) || !sv::aligned_to(y, y_dt) ||
      (bias && !sv::aligned_to(bias, bias_dt)) || (residual && !sv::aligned_to(residual, residual_dt)))
    return SV_EINVAL;
  if (!sv::rows_apart(y_row, y_group, M, groups, N)) return SV_EINVAL;
  sv::DeviceGuard guard(device);
  if (!guard.ok) return SV_ECUDA;
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
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int64_t tiles = (static_cast<int64_t>(N) + sv::kPlainTile - 1) / sv::kPlainTile *
                        ((static_cast<int64_t>(M) + sv::kPlainTile - 1) / sv::kPlainTile) * groups;
  const unsigned grid = static_cast<unsigned>(tiles < (1 << 20) ? tiles : (1 << 20));
  sv::plain_kernel<<<grid, 256, 0, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ECUDA;
}
