// Attention of drafted rows over a cache of 8-bit entries: spec_verify_attend.
//
//   out[r, h] = sum_p softmax_p(scale q[r, h] . K[p]) V[p],  p over the committed positions and the row's path
//
// The softmax runs over tiles of positions with the largest logit so far and the sum
// of the weights against it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "cache.cuh"
#include "entry.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

struct AttendParams {
  CacheView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t q_row, q_head, out_row, out_head;
  int q_heads, group;
  float scale;
  const int32_t *context, *node_start, *parent;
  int B, total, max_nodes;
};

constexpr int kTile = 128;

__device__ __forceinline__ float block_reduce(float v, bool sum, float* warps) {
  for (int o = 16; o; o >>= 1) {
    const float u = __shfl_xor_sync(~0u, v, o);
    v = sum ? v + u : fmaxf(v, u);
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = v;
  __syncthreads();
  v = warps[0];
  for (int w = 1; w < kTile / 32; ++w) v = sum ? v + warps[w] : fmaxf(v, warps[w]);
  return v;
}

// a CTA for each row and query head, a thread for each position of a tile, then for each d
__global__ void __launch_bounds__(kTile) attend_kernel(const __grid_constant__ AttendParams P) {
  __shared__ float q[128], weight[kTile], warps[kTile / 32];
  __shared__ uint32_t path[(SV_MAX_NODES + 31) / 32];
  __shared__ int bad;
  wait_for_stream();
  const CacheView& c = P.c;
  int at = blockIdx.x;
  const int head = at % P.q_heads;
  at /= P.q_heads;
  const int place = at % (P.max_nodes + 1), b = at / (P.max_nodes + 1);
  const int64_t context = P.context[b];
  const int start = P.node_start[b], stop = P.node_start[b + 1];
  if (context < 0 || start < 0 || stop < start || stop > P.total || stop - start > P.max_nodes || place > stop - start) return;
  const int64_t row = static_cast<int64_t>(start) + b + place;
  const int h = head / P.group, nodes = stop - start;
  if (threadIdx.x < (SV_MAX_NODES + 31) / 32) path[threadIdx.x] = 0;
  if (threadIdx.x == 0) bad = 0;
  if (static_cast<int>(threadIdx.x) < c.dim)
    q[threadIdx.x] = __bfloat162float(P.q[row * P.q_row + head * P.q_head + threadIdx.x]) * P.scale * 1.4426950408889634f;
  __syncthreads();
  const int64_t end = context + 1 + nodes;
  for (int64_t p = threadIdx.x * (int64_t{1} << c.page_log); p < end; p += static_cast<int64_t>(kTile) << c.page_log)
    if (c.page_of(b, p) < 0) bad = 1;
  for (int i = threadIdx.x; i < nodes; i += kTile) {
    const int up = P.parent ? P.parent[start + i] : i - 1;
    if (up < -1 || up >= i) bad = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0 && !bad)
    for (int i = place - 1; i >= 0; i = P.parent ? P.parent[start + i] : i - 1) path[i / 32] |= 1u << i % 32;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int64_t t0 = 0; t0 < end && !bad; t0 += kTile) {
    const int64_t pos = t0 + threadIdx.x;
    float x = -INFINITY;
    const int64_t node = pos - context - 1;
    if (pos < end && (node < 0 || (path[node / 32] >> (node % 32) & 1u))) {
      const int page = c.page_of(b, pos);
      const uint8_t* k = c.entries[0] + c.entry_at(page, h, pos);
      x = 0.f;
      for (int d = 0; d < c.dim; d += 2) {
        const float2 f = from_e4m3x2(*reinterpret_cast<const uint16_t*>(k + d));
        x += f.x * q[d] + f.y * q[d + 1];
      }
      x *= c.scales[0][c.scale_at(page, h, pos)];
    }
    const float to = fmaxf(m, block_reduce(x, false, warps));
    const float w = x == -INFINITY ? 0.f : exp2f(x - to), keep = m == to ? 1.f : exp2f(m - to);
    weight[threadIdx.x] = w;
    l = l * keep + block_reduce(w, true, warps);
    o *= keep;
    m = to;
    if (static_cast<int>(threadIdx.x) < c.dim)
      for (int i = 0; i < kTile && t0 + i < end; ++i) {
        const int64_t v_node = t0 + i - context - 1;
        if (v_node >= 0 && !(path[v_node / 32] >> (v_node % 32) & 1u)) continue;
        const int page = c.page_of(b, t0 + i);
        const uint8_t e = c.entries[1][c.entry_at(page, h, t0 + i) + threadIdx.x];
        o += weight[i] * c.scales[1][c.scale_at(page, h, t0 + i)] * from_e4m3x2(e).x;
      }
    __syncthreads();
  }
  if (static_cast<int>(threadIdx.x) < c.dim)
    P.out[row * P.out_row + head * P.out_head + threadIdx.x] = __float2bfloat16(bad ? NAN : o / l);
}

}  // namespace
}  // namespace sv

extern "C" size_t spec_verify_attend_workspace(int heads, int q_heads, int dim, int max_nodes, int device) {
  (void)heads, (void)q_heads, (void)dim, (void)max_nodes, (void)device;
  return 0;
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
  if (static_cast<int64_t>(total_nodes) + B > INT32_MAX) return SV_EUNSUPPORTED;
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
  if (reinterpret_cast<uintptr_t>(workspace) % 16 ||
      workspace_bytes < spec_verify_attend_workspace(cache->heads, q_heads, cache->dim, max_nodes, device))
    return SV_EINVAL;
  const __int128 grid = static_cast<__int128>(B) * (std::min(max_nodes, total_nodes) + 1) * q_heads;
  if (grid > INT32_MAX) return SV_EUNSUPPORTED;
  sv::DeviceGuard g(device);
  if (!g.ok) return SV_ECUDA;
  sv::AttendParams P = {};
  P.c = sv::view_of(*cache, page_table, table_stride, table_cols);
  P.q = static_cast<const __nv_bfloat16*>(q), P.out = static_cast<__nv_bfloat16*>(out);
  P.q_row = q_row, P.q_head = q_head, P.out_row = out_row, P.out_head = out_head;
  P.q_heads = q_heads, P.group = q_heads / cache->heads;
  P.scale = scale;
  P.context = context, P.node_start = node_start, P.parent = parent;
  P.B = B, P.total = total_nodes, P.max_nodes = max_nodes;
  P.max_nodes = std::min(max_nodes, total_nodes);
  return sv::launch_waiting(sv::attend_kernel, static_cast<unsigned>(grid), sv::kTile, 0, 1,
                            static_cast<cudaStream_t>(cuda_stream), P) == cudaSuccess
             ? SV_OK
             : SV_ECUDA;
}
