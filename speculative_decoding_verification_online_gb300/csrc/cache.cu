// Rows into a cache of 8-bit entries, and the rows of an accepted path together:
// spec_verify_cache_write, spec_verify_cache_keep.
//
// Writing: a CTA has the new rows of one block of entries, of keys or of values, and keeps
// them in registers between the search for the largest magnitude and the rounding: rows
// are read once.  Rows of 64 trees of up to 21 nodes, 8 heads of 128, bf16: 5.9 us; 32
// prompts of up to 2048 tokens: 54.3 us, 5.6 TB/s (in fp32 77.5 us).  What bounds that one is instructions as much as memory:
// the largest magnitude is therefore looked for among the bits, two bf16 at once, and
// finiteness is one question for the whole block (80.8 us with a test and a float
// maximum for every entry).  128 threads with 8 runs each were the best: 256 with 4 take
// 67.5 us, several blocks a CTA with the next one's rows on their way 133 us.
//
// Keeping: a CTA has some of a sequence's rows, and a warp moves one row of one head with
// its scale; where the rows lie is looked up once for all.  64 accepted paths in 16 layers
// of 8 heads of 128: 8.0 us, which is latency: the path, the pages, the scales, the rows,
// each known from the one before.
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

constexpr int kWriteThreads = 128;
constexpr int kWriteHeld = 8;  // runs of eight entries that a thread keeps between its two passes

struct WriteParams {
  CacheView c;
  const void* x[2];
  int64_t row[2], head[2];
  int vec[2];
  const int32_t *context, *node_start;
  int total, max_nodes, blocks;  // blocks: of a sequence at most
};

template <typename T>
struct Run;  // eight neighbouring entries as they lie in memory
template <>
struct Run<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, bool vec) {
    if (vec) {
      a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    } else {
      a = make_float4(p[0], p[1], p[2], p[3]), b = make_float4(p[4], p[5], p[6], p[7]);
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  // the largest bits of a magnitude (as whole numbers: those of infinities and NaN are above all others), and them as fp32's
  __device__ __forceinline__ uint32_t most(uint32_t m) const {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
  }
  static __device__ __forceinline__ uint32_t top(uint32_t m) { return m; }
};
template <>
struct Run<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool vec) {
    if (vec) {
      a = *reinterpret_cast<const uint4*>(p);
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
      a = make_uint4(q[0] | static_cast<uint32_t>(q[1]) << 16, q[2] | static_cast<uint32_t>(q[3]) << 16,
                     q[4] | static_cast<uint32_t>(q[5]) << 16, q[6] | static_cast<uint32_t>(q[7]) << 16);
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  __device__ __forceinline__ uint32_t most(uint32_t m) const {  // of both halves
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[i] & 0x7fff7fffu));
    return m;
  }
  static __device__ __forceinline__ uint32_t top(uint32_t m) { return max(m & 0xffffu, m >> 16) << 16; }
};

// the largest finite magnitude
__device__ __forceinline__ float largest(const float (&v)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(v[i]);
    m = a < INFINITY ? fmaxf(m, a) : m;
  }
  return m;
}

__device__ __forceinline__ uint2 pack8(const float (&v)[8]) {
  return make_uint2(e4m3x2(v[0], v[1]) | e4m3x2(v[2], v[3]) << 16, e4m3x2(v[4], v[5]) | e4m3x2(v[6], v[7]) << 16);
}

// A CTA writes one block of tokens of one head, of k or of v.
template <typename T>
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const __grid_constant__ WriteParams P) {
  __shared__ uint32_t warp_most[kWriteThreads / 32];
  wait_for_stream();
  const CacheView& c = P.c;
  int at = blockIdx.x;
  const int which = at & 1;
  at >>= 1;
  const int h = at % c.heads;
  at /= c.heads;
  const int j = at % P.blocks, b = at / P.blocks;
  const int64_t context = P.context[b];
  const int start = P.node_start[b], stop = P.node_start[b + 1];
  if (context < 0 || start < 0 || stop < start || stop > P.total || stop - start > P.max_nodes) return;
  const int size = 1 << c.block_log;
  const int64_t end = context + (stop - start) + 1;  // behind the new rows
  const int64_t p0 = ((context >> c.block_log) + j) << c.block_log;
  if (p0 >= end) return;
  const int64_t from = max(p0, context), to = min(p0 + size, end);
  const int runs_log = c.dim == 128 ? 4 : 3, runs = 1 << runs_log, count = static_cast<int>(to - from) << runs_log;
  const T* x = static_cast<const T*>(P.x[which]) + (start + b + (from - context)) * P.row[which] + h * P.head[which];
  auto source = [&](int i) { return x + (i >> runs_log) * P.row[which] + (i & (runs - 1)) * 8; };
  Run<T> held[kWriteHeld];
#pragma unroll
  for (int k = 0; k < kWriteHeld; ++k) {
    const int i = threadIdx.x + k * kWriteThreads;
    if (i < count) held[k].load(source(i), P.vec[which]);
  }
  // (the page is looked up while the rows are on their way)
  const int page = c.page_of(b, p0);
  if (page < 0) return;
  float* scale = c.scales[which] + c.scale_at(page, h, p0);
  const float old = from > p0 ? *scale : 0.f;
  // f of every run, held or not
  auto each = [&](auto f) {
#pragma unroll
    for (int k = 0; k < kWriteHeld; ++k)
      if (static_cast<int>(threadIdx.x) + k * kWriteThreads < count) f(threadIdx.x + k * kWriteThreads, held[k]);
    for (int i = threadIdx.x + kWriteHeld * kWriteThreads; i < count; i += kWriteThreads) {
      Run<T> r;
      r.load(source(i), P.vec[which]);
      f(i, r);
    }
  };
  auto over_all = [&](uint32_t bits) {
    bits = __reduce_max_sync(~0u, bits);
    if (threadIdx.x % 32 == 0) warp_most[threadIdx.x / 32] = bits;
    __syncthreads();
    for (int w = 0; w < kWriteThreads / 32; ++w) bits = max(bits, warp_most[w]);
    return bits;
  };
  uint32_t bits = 0;
  each([&](int, const Run<T>& r) { bits = r.most(bits); });
  bits = over_all(Run<T>::top(bits));
  float v[8];
  const bool finite = bits < 0x7f800000u;
  if (!finite) {  // once more, without what is not
    float most = 0.f;
    each([&](int, const Run<T>& r) {
      r.values(v);
      most = largest(v, most);
    });
    __syncthreads();
    bits = over_all(__float_as_uint(most));
  }
  const float most = __uint_as_float(bits);
  const float need = scale_for(most);
  const float now = from > p0 ? (need > old ? need : old) : need;
  uint8_t* entries = c.entries[which] + c.entry_at(page, h, p0);
  const float inverse = 1.f / now;
  if (from > p0 && now != old) {
    const int older = static_cast<int>(from - p0) << runs_log;
    for (int i = threadIdx.x; i < older; i += kWriteThreads) {
      uint2* p = reinterpret_cast<uint2*>(entries + (i >> runs_log) * c.token + (i & (runs - 1)) * 8);
      const uint2 e = *p;
      const uint32_t two[4] = {e.x & 0xffffu, e.x >> 16, e.y & 0xffffu, e.y >> 16};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = from_e4m3x2(two[k]);
        v[2 * k] = f.x * old * inverse, v[2 * k + 1] = f.y * old * inverse;
      }
      *p = pack8(v);
    }
  }
  each([&](int i, const Run<T>& r) {
    r.values(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = finite || fabsf(v[k]) < INFINITY ? v[k] * inverse : NAN;
    *reinterpret_cast<uint2*>(entries + (from - p0 + (i >> runs_log)) * c.token + (i & (runs - 1)) * 8) = pack8(v);
  });
  if (threadIdx.x == 0) *scale = now;
}

// ------------------------------------------------------------ accepted rows

struct KeepParams {
  CacheView c;
  const int32_t *path, *accepted, *context;
  int32_t* new_context;
  int max_depth, layers, parts, tasks;  // tasks: of a CTA at most
};

constexpr int kKeepThreads = 256;

struct KeepShared {
  // of a moved row: its entries before and after, and its scale before (of head 0)
  int64_t from[SV_MAX_NODES], to[SV_MAX_NODES], scale[SV_MAX_NODES];
  int bad;
};

// A CTA looks up where the rows of one sequence lie, and its warps move them, each in every n-th of its tasks: a head of a
// layer, of k or of v.  path[t] >= t rises, so that rows in rising order never lie where an earlier one was put: a block's
// sources are in blocks from its own on, whose scales and entries are still the old ones when its turn comes.
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepParams P) {
  __shared__ KeepShared s;
  wait_for_stream();
  const CacheView& c = P.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / P.parts, part = blockIdx.x % P.parts;
  const int64_t context = P.context[b], first = context + 1;
  const int len = P.accepted[b];
  const int32_t* path = P.path + static_cast<int64_t>(b) * P.max_depth;
  const int size = 1 << c.block_log;
  const int64_t p0 = first >> c.block_log << c.block_log;  // the first block that may receive rows
  bool good = context >= 0 && len >= 0 && len <= P.max_depth;
  if (threadIdx.x == 0) s.bad = 0;
  __syncthreads();
  if (good)
    for (int t = threadIdx.x; t < len; t += kKeepThreads) {
      const int node = path[t];
      const int page_to = c.page_of(b, first + t);
      int page_from = -1;
      if (node > (t ? path[t - 1] : -1)) page_from = c.page_of(b, first + node);
      if (page_from < 0 || page_to < 0) {
        s.bad = 1;
      } else {
        s.from[t] = c.entry_at(page_from, 0, first + node), s.to[t] = c.entry_at(page_to, 0, first + t);
        s.scale[t] = c.scale_at(page_from, 0, first + node);
      }
    }
  __syncthreads();
  good = good && !s.bad;
  if (part == 0 && threadIdx.x == 0 && P.new_context)
    P.new_context[b] = static_cast<int32_t>(good ? first + len : context);
  if (!good || len == 0) return;
  const int per_page = c.page_log - c.block_log, per_row = c.dim / 16, rows_at_once = 32 / per_row;
  const int mine = lane / per_row, byte = lane % per_row * 16;
  const int tasks = min(P.tasks, P.layers * c.heads * 2 - part * P.tasks);
#pragma unroll 1
  for (int i = warp; i < tasks; i += kKeepThreads / 32) {
    const int task = part * P.tasks + i, which = task & 1, h = (task >> 1) % c.heads, layer = (task >> 1) / c.heads;
    uint8_t* const entries = c.entries[which] + layer * c.layer + h * c.head;
    float* const scales = c.scales[which] + layer * c.scale_layer + (static_cast<int64_t>(h) << per_page);
#pragma unroll 1
    for (int64_t block = p0; block < first + len; block += size) {
      // rows of the block: `stay` from its beginning on, then the moved ones t0 .. t1 - 1
      const int stay = static_cast<int>(max(first - block, int64_t{0})), t0 = static_cast<int>(max(block - first, int64_t{0}));
      const int t1 = static_cast<int>(min(block + size - first, static_cast<int64_t>(len)));
      const int64_t at = s.to[t0] - stay * c.token;  // the block's first row
      // the block's own scale lies with that of its first moved row's destination
      const int64_t own_at = c.scale_at(c.page_of(b, block), 0, block);
      // the first rows' entries are on their way with the scales
      auto load = [&](int t) {
        return t < t1 ? *reinterpret_cast<const uint4*>(entries + s.from[t] + byte) : make_uint4(0, 0, 0, 0);
      };
      uint4 e = load(t0 + mine);
      const float own = scales[own_at];
      float most = stay > 0 ? own : 0.f;
      for (int t = t0 + lane; t < t1; t += 32) most = fmaxf(most, scales[s.scale[t]]);
      for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
      auto rescaled = [&](uint4 v, float f) {
        if (f == 1.f) return v;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = from_e4m3x2(w[k] & 0xffffu), hi = from_e4m3x2(w[k] >> 16);
          w[k] = e4m3x2(lo.x * f, lo.y * f) | e4m3x2(hi.x * f, hi.y * f) << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
      };
      // rows that stay follow a scale that grows
      if (stay > 0 && most != own)
        for (int d = mine; d < stay; d += rows_at_once) {
          uint4* const p = reinterpret_cast<uint4*>(entries + at + d * c.token + byte);
          *p = rescaled(*p, most > 0.f ? own / most : 1.f);
        }
#pragma unroll 1
      for (int t = t0 + mine; t - mine < t1; t += rows_at_once) {
        const float f = t < t1 && most > 0.f ? scales[s.scale[t]] / most : 1.f;
        const uint4 v = rescaled(e, f);
        const bool moves = t < t1 && (f != 1.f || s.from[t] != s.to[t]);
        e = load(t + rows_at_once);
        __syncwarp();
        if (moves) *reinterpret_cast<uint4*>(entries + s.to[t] + byte) = v;
        __syncwarp();
      }
      if (lane == 0 && most != own) scales[own_at] = most;
      __syncwarp();
    }
  }
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_verify_cache_write(const sv_cache* cache, const void* k, const void* v, sv_dtype dt, int64_t k_row,
                                             int64_t k_head, int64_t v_row, int64_t v_head, const int32_t* page_table,
                                             int64_t table_stride, int table_cols, const int32_t* context,
                                             const int32_t* node_start, int B, int total_nodes, int max_nodes, int device,
                                             void* cuda_stream) {
  if (sv_status s = sv::check_cache(cache, 1); s != SV_OK) return s;
  if (sv_status s = sv::check_table(page_table, table_stride, table_cols, B); s != SV_OK) return s;
  if (dt != SV_F32 && dt != SV_BF16) return SV_EINVAL;
  if (B < 0 || total_nodes < 0 || max_nodes < 0) return SV_EINVAL;
  if (k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0) return SV_EINVAL;
  for (const int64_t s : {k_row, k_head, v_row, v_head})
    if (s >= (int64_t{1} << 40)) return SV_EUNSUPPORTED;
  if (B == 0) return SV_OK;
  if (static_cast<int64_t>(total_nodes) + B > INT32_MAX) return SV_EUNSUPPORTED;
  if (!k || !v || !context || !node_start) return SV_EINVAL;
  const size_t es = dt == SV_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(k) % es || reinterpret_cast<uintptr_t>(v) % es || reinterpret_cast<uintptr_t>(context) % 4 ||
      reinterpret_cast<uintptr_t>(node_start) % 4)
    return SV_EINVAL;
  if (cache->pages == 0) return SV_OK;
  // max_nodes + 1 rows from any place in a block on
  const int blocks =
      static_cast<int>((std::min(max_nodes, total_nodes) + static_cast<int64_t>(cache->block) - 1) / cache->block) + 1;
  const __int128 grid = static_cast<__int128>(blocks) * B * cache->heads * 2;
  if (grid > INT32_MAX) return SV_EUNSUPPORTED;
  if (!sv::lies_apart(cache)) return SV_EINVAL;
  sv::DeviceGuard g(device);
  if (!g.ok) return SV_ECUDA;
  sv::WriteParams P = {};
  P.c = sv::view_of(*cache, page_table, table_stride, table_cols);
  P.x[0] = k, P.x[1] = v;
  P.row[0] = k_row, P.row[1] = v_row, P.head[0] = k_head, P.head[1] = v_head;
  for (int i = 0; i < 2; ++i)
    P.vec[i] = reinterpret_cast<uintptr_t>(P.x[i]) % 16 == 0 && P.row[i] * es % 16 == 0 && P.head[i] * es % 16 == 0;
  P.context = context, P.node_start = node_start;
  P.total = total_nodes, P.max_nodes = max_nodes;
  P.blocks = blocks;
  const auto kernel = dt == SV_BF16 ? sv::write_kernel<__nv_bfloat16> : sv::write_kernel<float>;
  return sv::launch_waiting(kernel, static_cast<unsigned>(grid), sv::kWriteThreads, 0, 1, static_cast<cudaStream_t>(cuda_stream),
                            P) == cudaSuccess
             ? SV_OK
             : SV_ECUDA;
}

extern "C" sv_status spec_verify_cache_keep(const sv_cache* cache, const int32_t* path, int max_depth,
                                            const int32_t* accepted_len, const int32_t* page_table, int64_t table_stride,
                                            int table_cols, const int32_t* context, int32_t* new_context, int B, int device,
                                            void* cuda_stream) {
  if (sv_status s = sv::check_cache(cache, 0); s != SV_OK) return s;
  if (sv_status s = sv::check_table(page_table, table_stride, table_cols, B); s != SV_OK) return s;
  if (B < 0 || max_depth < 0) return SV_EINVAL;
  if (max_depth > SV_MAX_NODES) return SV_EUNSUPPORTED;
  if (B == 0) return SV_OK;
  if ((max_depth > 0 && !path) || !accepted_len || !context || context == new_context) return SV_EINVAL;
  for (const void* p : {static_cast<const void*>(path), static_cast<const void*>(accepted_len),
                        static_cast<const void*>(context), static_cast<const void*>(new_context)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SV_EINVAL;
  const int64_t all = static_cast<int64_t>(cache->layers) * cache->heads * 2;
  if (static_cast<__int128>(all) * B > INT32_MAX) return SV_EUNSUPPORTED;
  if (!sv::lies_apart(cache)) return SV_EINVAL;
  // CTAs read while another one writes its sequence's
  if (new_context) {
    const sv::Extent to = {new_context, 4, B, 0, 1, 0, 1};
    if (sv::sure_to_overlap({context, 4, B, 0, 1, 0, 1}, to) || sv::sure_to_overlap({accepted_len, 4, B, 0, 1, 0, 1}, to) ||
        (max_depth > 0 && sv::sure_to_overlap({path, 4, max_depth, max_depth, B, 0, 1}, to)))
      return SV_EINVAL;
  }
  // A CTA has eight tasks at least, one a warp, and more where there are CTAs enough without
  const int64_t tasks = std::max<int64_t>(8, std::min<int64_t>(64, (all * B / 1024 + 7) / 8 * 8));
  const int64_t parts = (all + tasks - 1) / tasks;
  sv::DeviceGuard g(device);
  if (!g.ok) return SV_ECUDA;
  sv::KeepParams P = {};
  P.c = sv::view_of(*cache, page_table, table_stride, table_cols);
  P.path = path, P.accepted = accepted_len, P.context = context, P.new_context = new_context;
  P.max_depth = max_depth, P.layers = cache->layers;
  P.parts = static_cast<int>(parts), P.tasks = static_cast<int>(tasks);
  return sv::launch_waiting(sv::keep_kernel, static_cast<unsigned>(parts * B), sv::kKeepThreads, 0, 1,
                            static_cast<cudaStream_t>(cuda_stream), P) == cudaSuccess
             ? SV_OK
             : SV_ECUDA;
}
