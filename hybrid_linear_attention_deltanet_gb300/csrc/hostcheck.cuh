// Host-side argument checks and launches shared by the entry points of the
// operators around the mixer.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gdn {
namespace hostcheck {

// The longest axis that 32-bit coordinates of tiles up to 256 wide hold.
constexpr int32_t kLongestAxis = 0x7fffff00;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct Span {
  uintptr_t lo, hi;   // [lo, hi)
};
inline Span span_of(const void* p, size_t bytes) {
  return {(uintptr_t)p, (uintptr_t)p + (p ? bytes : 0)};
}
inline bool intersect(Span a, Span b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// Any output overlapping an input or another output?
template <size_t NI, size_t NO>
bool any_overlap(const Span (&ins)[NI], const Span (&outs)[NO]) {
  for (size_t o = 0; o < NO; ++o) {
    for (size_t i = 0; i < NI; ++i)
      if (intersect(ins[i], outs[o])) return true;
    for (size_t p = 0; p < o; ++p)
      if (intersect(outs[p], outs[o])) return true;
  }
  return false;
}

// SMs of the current device (0 when it cannot be read).
inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// Allows a kernel its dynamic shared memory, once a device (a bit each in `on`).
inline cudaError_t allow_smem(const void* kern, size_t bytes, std::atomic<uint64_t>& on) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (on.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) on.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace hostcheck

// The matrix products and the sums of parts are launched as programmatic
// dependents: a grid may start while the one before it in the stream still
// runs, does what needs no data (barriers, tensor memory), and waits in
// grid_wait() for that grid's end and memory before its first access to global
// memory; every kernel launched so calls it.  (About 1 us of a product's 5 to
// 15 with few tokens; the attribute costs the host 1.5 us a launch, more than
// the norms themselves would gain.)
__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Loads of what the grid before may have written, for after grid_wait().  (This
// grid is resident while that one writes, so the memory is not read-only for its
// lifetime: a non-coherent load may return what an SM's L1 still holds of it, and
// the compiler may move one across the wait.)
__device__ __forceinline__ float ld_waited(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 ld_waited(const float4* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_waited(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ int32_t ld_waited(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
// The next grid may start once every CTA of this one has come here.
__device__ __forceinline__ void grid_release_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// dependent: as a programmatic dependent.  cluster: CTAs of a cluster along x,
// 0 where the kernel itself says so.
template <typename... P, typename... A>
cudaError_t launch(bool dependent, void (*kern)(P...), dim3 grid, unsigned threads, size_t smem,
                   unsigned cluster, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  unsigned n = 0;
  if (dependent) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) (void)cudaGetLastError();   // reported here, not to the caller's next call
  return e;
}

}  // namespace gdn
