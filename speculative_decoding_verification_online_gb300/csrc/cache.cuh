// A cache in pages of 8-bit entries, as the kernels see it.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <iterator>

#include "spec_verify.h"

namespace sv {

// the checks of spec_verify.h that the host can make; rows of the table are not among them
inline sv_status check_cache(const sv_cache* c, int layers) {
  if (!c) return SV_EINVAL;
  if (c->layers < 1 || c->pages < 0 || c->heads < 1) return SV_EINVAL;
  if (layers > 0 && c->layers != layers) return SV_EINVAL;
  const auto power = [](int n) { return n > 0 && (n & (n - 1)) == 0; };
  if (!power(c->page_tokens) || !power(c->block) || c->block > c->page_tokens) return SV_EINVAL;
  if (c->page_tokens < 16 || c->page_tokens > 256 || (c->dim != 64 && c->dim != 128)) return SV_EUNSUPPORTED;
  if (c->layer_stride < 0 || c->page_stride < 0 || c->head_stride < 0 || c->token_stride < c->dim || c->scale_layer_stride < 0)
    return SV_EINVAL;
  for (const int64_t s : {c->layer_stride, c->page_stride, c->head_stride, c->token_stride}) {
    if (s % 16) return SV_EINVAL;
    if (s >= (int64_t{1} << 40)) return SV_EUNSUPPORTED;
  }
  // pages and heads that share their place
  if ((c->pages > 1 && c->page_stride < c->dim) || (c->heads > 1 && c->head_stride < c->dim) ||
      (c->layers > 1 && c->layer_stride < c->dim))
    return SV_EINVAL;
  if (c->pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return SV_EINVAL;
  if (reinterpret_cast<uintptr_t>(c->k) % 16 || reinterpret_cast<uintptr_t>(c->v) % 16 ||
      reinterpret_cast<uintptr_t>(c->k_scale) % 4 || reinterpret_cast<uintptr_t>(c->v_scale) % 4)
    return SV_EINVAL;
  return SV_OK;
}

// whether no two entries of a cache that is written, and no two scales, share their place (as far as strides tell)
inline bool lies_apart(const sv_cache* c) {
  struct Dimension {
    int64_t stride, count;
  } d[] = {{c->layer_stride, c->layers}, {c->page_stride, c->pages}, {c->head_stride, c->heads}, {c->token_stride, c->page_tokens}};
  std::sort(std::begin(d), std::end(d), [](const Dimension& a, const Dimension& b) { return a.stride < b.stride; });
  __int128 span = c->dim;
  for (const Dimension& one : d) {
    if (one.count <= 1) continue;
    if (one.stride < span) return false;
    span += static_cast<__int128>(one.stride) * (one.count - 1);
  }
  const __int128 scales = static_cast<__int128>(c->pages) * c->heads * (c->page_tokens / c->block);
  return c->layers == 1 || c->scale_layer_stride >= scales;
}

inline sv_status check_table(const int32_t* page_table, int64_t table_stride, int table_cols, int B) {
  if (table_cols < 0 || (B > 1 && table_stride < 0) || (table_cols > 0 && !page_table)) return SV_EINVAL;
  if (table_stride >= (int64_t{1} << 40)) return SV_EUNSUPPORTED;
  return reinterpret_cast<uintptr_t>(page_table) % 4 ? SV_EINVAL : SV_OK;
}

inline int log2_of(int power) {
  int l = 0;
  while (1 << l < power) ++l;
  return l;
}

struct CacheView {
  uint8_t* entries[2];  // k, v
  float* scales[2];
  int64_t layer, page, head, token, scale_layer;  // bytes, and scales
  int pages, heads, dim;
  int page_log, block_log;
  const int32_t* table;
  int64_t table_stride;
  int table_cols;

  // the page of a sequence's position, -1 where it has none
  __device__ __forceinline__ int page_of(int b, int64_t pos) const {
    const int64_t col = pos >> page_log;
    if (col >= table_cols) return -1;
    const int p = table[b * table_stride + col];
    return p >= 0 && p < pages ? p : -1;
  }
  __device__ __forceinline__ int64_t entry_at(int page_id, int h, int64_t pos) const {
    return page_id * page + h * head + (pos & ((1 << page_log) - 1)) * token;
  }
  __device__ __forceinline__ int64_t scale_at(int page_id, int h, int64_t pos) const {
    return ((static_cast<int64_t>(page_id) * heads + h) << (page_log - block_log)) +
           ((pos & ((1 << page_log) - 1)) >> block_log);
  }
};

inline CacheView view_of(const sv_cache& c, const int32_t* table, int64_t table_stride, int table_cols) {
  CacheView v = {};
  v.entries[0] = static_cast<uint8_t*>(c.k), v.entries[1] = static_cast<uint8_t*>(c.v);
  v.scales[0] = c.k_scale, v.scales[1] = c.v_scale;
  v.layer = c.layer_stride, v.page = c.page_stride, v.head = c.head_stride, v.token = c.token_stride;
  v.scale_layer = c.scale_layer_stride;
  v.pages = c.pages, v.heads = c.heads, v.dim = c.dim;
  v.page_log = log2_of(c.page_tokens), v.block_log = log2_of(c.block);
  v.table = table, v.table_stride = table_stride, v.table_cols = table_cols;
  return v;
}

// 2^ceil(log2(a / 448)), 2^-100 at least.  448 is 0.875 * 2^9, and a = f * 2^e with f in [1/2, 1).
__device__ __forceinline__ float scale_for(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 126;
  const int k = max(-100, (u & 0x7fffffu) <= 0x600000u ? e - 9 : e - 8);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// two values to e4m3, to nearest, ties to even, 448 at most; the first one in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// two entries as floats (exact)
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  float2 f;
  asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

}  // namespace sv
