// Host-side argument checks shared by the entry points of the operators
// around the mixer.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace hostcheck {

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

}  // namespace hostcheck
}  // namespace gdn
