// Shared by the entry points that take no handle: a device made current for a
// scope, programmatic dependent launches, and waits that give up.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace sv {

struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) {
      ok = false;
      return;
    }
    if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

// Where an operand's entries lie: `groups` times `rows` rows of n entries of `size` bytes, strides counting entries.
struct Extent {
  const void* p;
  int64_t size, n, row, rows, group, groups;
  // bytes from the first entry to behind the last (strides below 2^40 times counts up to 2^30)
  __int128 span() const {
    return (static_cast<__int128>(row) * (rows - 1) + static_cast<__int128>(group) * (groups - 1) + n) * size;
  }
  // whether every byte between them is one of its own
  bool dense() const { return span() == static_cast<__int128>(n) * rows * groups * size; }
};

// Whether two operands (neither of them empty) share memory for certain: they start at one place, or lie in parts of memory
// that meet and have no gaps.  Rows that lie between another operand's rows are not told apart.
inline bool sure_to_overlap(const Extent& a, const Extent& b) {
  if (a.p == b.p) return true;
  const __int128 pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return pa < pb + b.span() && pb < pa + a.span() && a.dense() && b.dense();
}

// rows of N values at g * group + m * row that never share a place
inline bool rows_apart(int64_t row, int64_t group, int64_t M, int64_t groups, int64_t N) {
  if (M == 1) return groups == 1 || group >= N;
  if (groups == 1) return row >= N;
  // strides below 2^40 times counts up to 2^30
  const __int128 rows = static_cast<__int128>(row) * (M - 1) + N, all = static_cast<__int128>(group) * (groups - 1) + N;
  return row <= group ? row >= N && group >= rows : group >= N && row >= all;
}

// A kernel's first step: everything before it in the stream is done and visible.
// Then the next kernel may come in as CTAs leave (it waits here in its turn).
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---- mbarriers in shared memory

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint64_t* bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar, int times) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(times) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint64_t* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Waits for a phase; gives up after two seconds, or when another wait of the CTA
// has, and marks that in *dead.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, unsigned parity, volatile int* dead) {
  if (mbar_try(bar, parity)) return true;
  unsigned long long since = 0;
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (mbar_try(bar, parity)) return true;
    const unsigned long long t = now_ns();
    if (since == 0) since = t;
    if (*dead || t - since > 2000000000ull) {
      *dead = 1;
      return false;
    }
  }
}

// The end of a CTA of which a wait gave up.  Its copies, and what the other CTAs of
// its cluster write into its memory, may still be on their way.  It stays for more
// than three waits, the most that another CTA can pass before it misses this one's
// part and gives up too.
__device__ __forceinline__ void stay_behind() {
  const unsigned long long since = now_ns();
  while (now_ns() - since < 8000000000ull) __nanosleep(1000000);
}

// the address of the same place in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ uint32_t in_cta(const void* p, unsigned rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}

// What a kernel needs once a device before launch_waiting: its dynamic shared memory,
// clusters of more than the portable eight CTAs, and how many clusters run at once.
template <typename K>
cudaError_t prepare_waiting(K kernel, unsigned threads, size_t smem, unsigned ctas, int* resident) {
  cudaError_t e = cudaSuccess;
  if (smem > 0)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(resident, kernel, &cfg);
}

// The launch of a kernel that calls wait_for_stream, in clusters of `ctas`: it may
// become resident while its predecessor drains.
template <typename K, typename... A>
cudaError_t launch_waiting(K kernel, dim3 grid, unsigned threads, size_t smem, unsigned ctas, cudaStream_t st,
                           const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sv
