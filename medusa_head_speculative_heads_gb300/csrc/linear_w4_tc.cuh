// What the two tensor-memory kernels of medusa_linear_w4 share: rings, waits, tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "host_util.h"
#include "linear_w4.h"
#include "sm100.cuh"

namespace medusa {
namespace w4 {
using namespace sm100;

constexpr int kCols = 128;                 // columns of a block
constexpr uint32_t kRing = 229376;         // 224 KB for a CTA's rings
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainNs = 100000000ull;

// A place in a ring and the parity of its present round.
struct Ring {
  int i = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      ++round;
    }
  }
  // The phase that ends when this place is full; the one that ended when it was last emptied.
  __device__ __forceinline__ uint32_t full() const { return round & 1u; }
  __device__ __forceinline__ uint32_t empty() const { return (round - 1u) & 1u; }
  __device__ __forceinline__ bool used() const { return round > 0; }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
  return ok != 0;
}
// Barriers by their shared-memory addresses: what a wait costs in instructions, the unpacking warps have less for
// their work.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
// What follows a try that came back empty, out of line: the roles' loops have to stay in the instruction caches next
// to one another.
static __device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = global_timer_ns();
  while (!try_wait(bar, parity)) {
    if (*abort) return false;
    if ((int64_t)(global_timer_ns() - t0) > (int64_t)kWaitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// All lanes wait for a phase; true when all saw it end.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
  const bool ok = wait_longer(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) { return warp_wait(smem_u32(bar), parity, abort); }
// A value that is the same in all lanes, known to be so by the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
// Descriptors of K-major operands with 128-byte swizzle are a constant half and an address in units of 16 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The scales and zeros of a row in a block of columns: GROUPS of them.  Where their rows lie on 16 bytes they come with
// the weights by TMA (TILED); else a thread loads its own, a block ahead.
template <int GROUPS>
struct Raw {
  uint32_t s[GROUPS], z[GROUPS];
};
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ host side

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    cudaGetLastError();
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// [rows][cols] with `pitch` bytes between rows, boxes of bc columns by br rows.
inline bool make_map(CUtensorMap* m, CUtensorMapDataType ty, const void* base, long long cols, long long rows, long long pitch, int bc, int br,
                     CUtensorMapSwizzle sw) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {(cuuint32_t)bc, (cuuint32_t)br}, es[2] = {1, 1};
  return encode_fn()(m, ty, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch in clusters of `share` CTAs, which may begin before the kernel in front of it has ended.
template <typename... K, typename... A>
inline cudaError_t launch_clusters(void (*kern)(K...), int grid, int threads, size_t smem, int share, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = share;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<A&&>(args)...);
}

}  // namespace w4
}  // namespace medusa
