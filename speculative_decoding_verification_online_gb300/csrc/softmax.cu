// Probabilities of logits rows: spec_verify_softmax.
//
//   probs[r, v] = exp((l[r, v] - m_r) / T_r) / sum_w exp((l[r, w] - m_r) / T_r),  m_r = max_w l[r, w]
//
// T_r = 0 is the limit: 1 at the row's first largest logit, 0 elsewhere.
//
// Bound by memory: every logit read once and every probability written once.  A
// row is a cluster of up to sixteen CTAs, each holding its part of the row in
// registers (32 entries a thread) from the one read to the write.  A cluster takes
// every n-th row, and its next rows are on their way into shared memory (every
// thread copies and reads back its own entries) while it works on one.  A thread takes
// the exponentials of its own entries against its own largest, so that one
// exchange of (largest, sum) through the cluster is all that the row needs; the
// last factor exp((largest of the thread - largest of the row) / T) / sum is one
// multiplication an entry.  Parts longer than the registers hold are read twice,
// the second time from L2.
//
// Measured on a GB300: 384 rows of 128256 bf16 logits 55 to 62 us repeated on the same
// ones, 63 us on others each time, 4.7 to 5.4 TB/s of 6.78 (36 clusters of eight CTAs
// fit; a row's turn is its arithmetic, 17 warp instructions for 32 entries, then an
// exchange that the other CTA of the SM has to cover); 746 x 62236 49 us, 5.7 TB/s;
// seven rows of 262143 fp32 logits 5.1 us; 64 rows of 400000 bf16 logits, read twice,
// 48 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "entry.cuh"
#include "spec_verify.h"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kSoftThreads = 512;  // of a CTA; rows of up to kSoftShort entries take CTAs of kSoftFew
constexpr int kSoftFew = 128;
constexpr int kSoftHeld = 32;  // entries of a row that a thread keeps
constexpr int kSoftPart = kSoftThreads * kSoftHeld, kSoftShort = kSoftFew * kSoftHeld;
constexpr int kSoftCluster = 16;
constexpr int kSoftSpare = 32;  // bytes of a stage for what lies around a part in its first and last block

struct SoftParams {
  const void* x;
  int64_t x_stride;
  float* y;
  int64_t y_stride;
  const float* t_row;
  float t;
  int64_t rows;
  int V, part;  // part: entries of a row for each CTA, a multiple of 8
};

struct SoftShared {
  float warp_m[kSoftThreads / 32], warp_s[kSoftThreads / 32];
  int warp_at[kSoftThreads / 32];
  // the CTAs' parts of a row, by turns: a CTA writes a place again only after every other one has passed the
  // exchange between
  float2 part[2][kSoftCluster];  // (largest, sum)
  float m[2][kSoftCluster];      // (largest, its place) where T = 0
  int at[2][kSoftCluster];
  uint64_t arrived[2], copied[3];
  volatile int dead, copy_dead;  // two marks: a row whose exchange failed still waits for its copy
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Two floats in a 64-bit register: one instruction for both, each rounded by itself.
using Two = unsigned long long;

__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(Two t) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(t));
  return f;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^x; results below 2^-126 become 0
__device__ __forceinline__ float power(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// four neighbouring logits, as they lie in memory
template <typename T>
struct Four;
template <>
struct Four<float> {
  float4 f;
  __device__ __forceinline__ void set(float a, float b, float c, float d) { f = make_float4(a, b, c, d); }
  __device__ __forceinline__ void load(const void* p) { f = *static_cast<const float4*>(p); }
  __device__ __forceinline__ float max() const { return fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)); }
  __device__ __forceinline__ Two first() const { return two(f.x, f.y); }
  __device__ __forceinline__ Two second() const { return two(f.z, f.w); }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void set(float a, float b, float c, float d) {
    u.x = __float_as_uint(a) >> 16 | __float_as_uint(b);  // bf16 values: the low halves are 0
    u.y = __float_as_uint(c) >> 16 | __float_as_uint(d);
  }
  __device__ __forceinline__ void load(const void* p) { u = *static_cast<const uint2*>(p); }
  __device__ __forceinline__ float max() const {
    uint32_t m;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(u.x), "r"(u.y));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  __device__ __forceinline__ Two first() const {
    return two(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
  }
  __device__ __forceinline__ Two second() const {
    return two(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  }
};

constexpr int kSoftFours = kSoftHeld / 4;

// The j-th four of a thread are the entries 4 (j threads + thread) .. + 3 of a part of n, or with kVec false the entries
// (4 j + i) threads + thread; -inf behind the part.
template <typename T, bool kVec, int kThreads>
__device__ __forceinline__ void load_four(Four<T>& f, const T* part, int n, int j) {
  if constexpr (kVec) {
    const int at = 4 * (j * kThreads + static_cast<int>(threadIdx.x));
    if (4 * (j + 1) * kThreads <= n || at + 4 <= n)
      f.load(part + at);
    else
      f.set(at < n ? load_logit(part + at) : -INFINITY, at + 1 < n ? load_logit(part + at + 1) : -INFINITY,
            at + 2 < n ? load_logit(part + at + 2) : -INFINITY, -INFINITY);
  } else {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = (4 * j + i) * kThreads + static_cast<int>(threadIdx.x);
      v[i] = (4 * j + i + 1) * kThreads <= n || at < n ? load_logit(part + at) : -INFINITY;
    }
    f.set(v[0], v[1], v[2], v[3]);
  }
}

// The exponentials exp((l - m) / T) of a part's entries against the thread's largest m, and their sum.  With nothing
// but -inf (or NaN) m is -inf and the terms are 0 (or NaN).
template <typename T, bool kVec, int kThreads>
__device__ __forceinline__ void load_part(const T* part, int n, float c, Two (&e)[2 * kSoftFours], float& m, float& sum) {
  Four<T> f[kSoftFours];
#pragma unroll
  for (int j = 0; j < kSoftFours; ++j) load_four<T, kVec, kThreads>(f[j], part, n, j);
  m = f[0].max();
#pragma unroll
  for (int j = 1; j < kSoftFours; ++j) m = fmaxf(m, f[j].max());
  const float ref = m == -INFINITY ? 0.f : -m;
  const Two ref2 = two(ref, ref), c2 = two(c, c);
  Two s[2] = {};
#pragma unroll
  for (int j = 0; j < kSoftFours; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = both(mul2(add2(i ? f[j].second() : f[j].first(), ref2), c2));
      e[2 * j + i] = two(power(a.x), power(a.y));
      s[i] = add2(s[i], e[2 * j + i]);
    }
  const float2 t = both(add2(s[0], s[1]));
  sum = t.x + t.y;
}

template <bool kVec, int kThreads>
__device__ __forceinline__ void store_part(float* y, int lo, int hi, const Two (&e)[2 * kSoftFours], float scale) {
  const Two scale2 = two(scale, scale);
#pragma unroll
  for (int j = 0; j < kSoftFours; ++j) {
    const float2 a = both(mul2(e[2 * j], scale2)), b = both(mul2(e[2 * j + 1], scale2));
    if constexpr (kVec) {
      const int at = lo + 4 * (j * kThreads + static_cast<int>(threadIdx.x));
      if (4 * (j + 1) * kThreads <= hi - lo || at + 4 <= hi) {
        *reinterpret_cast<float4*>(y + at) = make_float4(a.x, a.y, b.x, b.y);
      } else {
        if (at < hi) y[at] = a.x;
        if (at + 1 < hi) y[at + 1] = a.y;
        if (at + 2 < hi) y[at + 2] = b.x;
      }
    } else {
      const float v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = lo + (4 * j + i) * kThreads + static_cast<int>(threadIdx.x);
        if (at < hi) y[at] = v[i];
      }
    }
  }
}

// how much a sum against `from` counts in one against `to` >= from
__device__ __forceinline__ float rescale(float from, float to, float c) {
  return from == to ? 1.f : power((from - to) * c);
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
__device__ __noinline__ void one_hot(SoftShared& s, const T* x, float* y, int lo, int hi, int turn) {
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
      to->m[turn][rank] = m, to->at[turn][rank] = at;
    }
  }
  cluster.sync();
  m = s.m[turn][0], at = s.at[turn][0];
  for (int r = 1; r < ctas; ++r) take_larger(m, at, s.m[turn][r], s.at[turn][r]);
  const bool valid = fabsf(m) < INFINITY;
  for (int v = lo + threadIdx.x; v < hi; v += kThreads) y[v] = valid ? (v == at ? 1.f : 0.f) : NAN;
}

// A part's entries on their way into a stage: one thread.  The copy takes the aligned blocks of 16 bytes that hold an
// entry of the part (an allocation has all of such a block); the first entry lies `shift_of` bytes into the stage.
__device__ __forceinline__ unsigned shift_of(const void* first) {
  return static_cast<unsigned>(reinterpret_cast<uintptr_t>(first) & 15);
}

template <typename T>
__device__ __forceinline__ void copy_part(const T* x, int lo, int hi, uint8_t* stage, uint64_t* bar) {
  const unsigned shift = shift_of(x + lo);
  const unsigned bytes = hi > lo ? (shift + static_cast<unsigned>(hi - lo) * static_cast<unsigned>(sizeof(T)) + 15) / 16 * 16 : 0;
  mbar_expect(bar, bytes);
  if (bytes > 0)
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(stage)),
                 "l"(reinterpret_cast<const uint8_t*>(x + lo) - shift), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

template <typename T>
constexpr int kSoftStages = sizeof(T) == 2 ? 3 : 1;  // two CTAs of 512 threads fill an SM's shared memory

template <typename T, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) softmax_kernel(const __grid_constant__ SoftParams P) {
  extern __shared__ __align__(16) uint8_t stages[];
  __shared__ SoftShared s;
  constexpr int kStages = kSoftStages<T>, kStageBytes = kThreads * kSoftHeld * sizeof(T) + kSoftSpare;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int clusters = gridDim.x / ctas;
  if (threadIdx.x == 0) {
    mbar_init(&s.arrived[0], 1);
    mbar_init(&s.arrived[1], 1);
    for (int i = 0; i < 3; ++i) mbar_init(&s.copied[i], 1);
    s.dead = s.copy_dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster.sync();  // every CTA of the cluster runs before any writes into another
  wait_for_stream();
  unsigned phases = 0;  // of the two barriers
  const T* x0 = static_cast<const T*>(P.x);
  const int lo = min(rank * P.part, P.V), hi = min(lo + P.part, P.V);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool held = P.part <= kThreads * kSoftHeld;
  int64_t r = blockIdx.x / ctas;
  uint32_t stage = 0, stage_phase = 0;  // of row r
  if (held && threadIdx.x == 0)
    for (int i = 0; i < kStages; ++i)
      if (r + i * clusters < P.rows)
        copy_part<T>(x0 + (r + i * clusters) * P.x_stride, lo, hi, stages + i * kStageBytes, &s.copied[i]);
  for (int turn = 0; r < P.rows; r += clusters, turn ^= 1) {
    const T* x = x0 + r * P.x_stride;
    float* y = P.y + r * P.y_stride;
    const float t = P.t_row ? P.t_row[r] : P.t;
    // 1.44.. / t overflows below 1e-38, where every logit but the largest has no probability
    float c = t > 0.f ? fminf(1.4426950408889634f / t, 3.0e38f) : 1.f;
    Two e[2 * kSoftFours];
    float m, sum;
    if (held) {
      if (!mbar_wait(&s.copied[stage], stage_phase, &s.copy_dead)) c = NAN;  // what lies in the stage is not the row
      load_part<T, kVec, kThreads>(reinterpret_cast<const T*>(stages + stage * kStageBytes + shift_of(x + lo)), hi - lo, c, e,
                                   m, sum);
    } else {
      m = -INFINITY, sum = 0.f;
#pragma unroll 1
      for (int at = lo; at < hi; at += kThreads * kSoftHeld) {
        float mv, sv;
        load_part<T, kVec, kThreads>(x + at, hi - at, c, e, mv, sv);
        const float to = fmaxf(m, mv);
        sum = sum * rescale(m, to, c) + sv * rescale(mv, to, c);
        m = to;
      }
    }
    // once every thread has read its stage, the row that is to follow there
    auto ahead = [&]() {
      if (!held) return;
      const int64_t next = r + static_cast<int64_t>(kStages) * clusters;
      if (threadIdx.x == 0 && next < P.rows && !s.copy_dead)
        copy_part<T>(x0 + next * P.x_stride, lo, hi, stages + stage * kStageBytes, &s.copied[stage]);
      if (++stage == kStages) stage = 0, stage_phase ^= 1;
    };
    if (t == 0.f) {
      one_hot<T, kThreads>(s, x, y, lo, hi, turn);
      ahead();
      continue;
    }
    const float mine = m;
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    sum *= rescale(mine, m, c);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) s.warp_m[warp] = m, s.warp_s[warp] = sum;
    __syncthreads();
    ahead();
    if (warp == 0) {
      const float wm = lane < kThreads / 32 ? s.warp_m[lane] : -INFINITY;
      float bm = wm, bs = lane < kThreads / 32 ? s.warp_s[lane] : 0.f;
      for (int o = 16; o; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, o));
      bs *= rescale(wm, bm, c);
      for (int o = 16; o; o >>= 1) bs += __shfl_xor_sync(~0u, bs, o);
      // Every CTA writes its part into every other's memory, and the write itself counts there.  A cluster barrier
      // would first wait for the stores of the row before.
      const bool heard = !s.dead;  // a phase that did not come is not begun again
      if (lane == 0 && heard) mbar_expect(&s.arrived[turn], ctas * sizeof(float2));
      if (lane < ctas && heard)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                         in_cta(&s.part[turn][rank], lane)),
                     "l"(two(bm, bs)), "r"(in_cta(&s.arrived[turn], lane))
                     : "memory");
    }
    const bool ok = mbar_wait(&s.arrived[turn], phases >> turn & 1, &s.dead);
    phases ^= 1u << turn;
    const float2 part = lane < ctas ? s.part[turn][lane] : make_float2(-INFINITY, 0.f);
    m = part.x;
    for (int o = kSoftCluster / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o, kSoftCluster));
    sum = lane < ctas ? part.y * rescale(part.x, m, c) : 0.f;
    for (int o = kSoftCluster / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o, kSoftCluster);
    m = __shfl_sync(~0u, m, 0), sum = __shfl_sync(~0u, sum, 0);
    // a NaN, a +inf and a row of nothing but -inf have made the sum NaN or 0, and the row NaN
    const float inv = ok && t > 0.f && t < INFINITY ? 1.f / sum : NAN;
    if (held) {
      store_part<kVec, kThreads>(y, lo, hi, e, rescale(mine, m, c) * inv);
    } else {
#pragma unroll 1
      for (int at = lo; at < hi; at += kThreads * kSoftHeld) {
        float mv, sv;
        load_part<T, kVec, kThreads>(x + at, hi - at, c, e, mv, sv);
        store_part<kVec, kThreads>(y, at, hi, e, rescale(mv, m, c) * inv);
      }
    }
  }
  if (s.dead || s.copy_dead) stay_behind();
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
  const bool in_place = logits == probs && dt == SV_F32 && (rows == 1 || logits_stride == probs_stride);
  if (!in_place && sv::sure_to_overlap({logits, static_cast<int64_t>(es), V, logits_stride, rows, 0, 1},
                                       {probs, 4, V, probs_stride, rows, 0, 1}))
    return SV_EINVAL;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return SV_ECUDA;
  // Enough CTAs a row to hold it, and more while the rows leave room beside two CTAs an SM.  Half as many, as chosen and twice
  // as many: 7 x 262143 fp32 8.8, 5.1 us (no more than 16); 20 x 128256 bf16 7.4, 6.2, 8.8 us; 80 x 32000 7.4, 5.9, 7.4 us;
  // 384 x 32000 18.1, 14.0, 24.2 us; 384 x 128256 67.8, 55.3, 108 us; 200 x 128256 fp32 43.0, 40.1, 56.7 us.  Above 131072
  // entries holding a row takes 16, of which 14 clusters fit: 300 x 151936 bf16 86 us; read twice by 8 110 us, by 4 75 us.
  int ctas = 1;
  while (ctas < sv::kSoftCluster && (V > ctas * sv::kSoftPart || (static_cast<int64_t>(rows) * ctas * 2 <= 2ll * sms &&
                                                                  V > ctas * sv::kSoftThreads * 4)))
    ctas *= 2;
  const int part = ((V + ctas - 1) / ctas + 7) / 8 * 8;
  const bool vec = reinterpret_cast<uintptr_t>(logits) % (4 * es) == 0 && reinterpret_cast<uintptr_t>(probs) % 16 == 0 &&
                   (rows == 1 || (logits_stride % 4 == 0 && probs_stride % 4 == 0));
  const bool few = ctas == 1 && V <= sv::kSoftShort;
  const int threads = few ? sv::kSoftFew : sv::kSoftThreads;
  const auto kernel = few ? sv::softmax_variant<sv::kSoftFew>(dt, vec) : sv::softmax_variant<sv::kSoftThreads>(dt, vec);
  const bool held = part <= threads * sv::kSoftHeld;
  const sv::SoftParams P = {logits, logits_stride, probs, probs_stride, temperature_per_row, temperature, rows, V, part};
  const int stages = dt == SV_BF16 ? sv::kSoftStages<__nv_bfloat16> : sv::kSoftStages<float>;
  const size_t smem = held ? stages * (threads * sv::kSoftHeld * es + sv::kSoftSpare) : 0;
  // how many clusters of this variant run at once: asked once a device
  static std::atomic<int> known[64][2][2][2][2][5];
  int log = 0;
  while (1 << log < ctas) ++log;
  std::atomic<int>* at = device < 64 ? &known[device][dt == SV_BF16][vec][few][held][log] : nullptr;
  int resident = at ? at->load() : 0;
  if (resident == 0) {
    if (sv::prepare_waiting(kernel, threads, smem, ctas, &resident) != cudaSuccess || resident < 1) return SV_ECUDA;
    if (at) at->store(resident);
  }
  const int64_t clusters = std::min<int64_t>(rows, resident);
  return sv::launch_waiting(kernel, static_cast<unsigned>(clusters * ctas), threads, smem, ctas,
                            static_cast<cudaStream_t>(cuda_stream), P) == cudaSuccess
             ? SV_OK
             : SV_ECUDA;
}
