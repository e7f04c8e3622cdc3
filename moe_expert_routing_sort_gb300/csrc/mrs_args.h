// mrs_args.h -- argument checks shared by the C entry points: address spans, alignment and
// the status of a launch.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "moe_route_sort.h"

namespace mrs {

struct Span {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Span span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + bytes};
}

inline bool overlap(const Span& a, const Span& b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

// Outputs must not overlap each other or any input.
inline bool any_alias(const Span* outs, int nout, const Span* ins, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = i + 1; j < nout; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (int j = 0; j < nin; ++j)
      if (overlap(outs[i], ins[j])) return true;
  }
  return false;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int launch_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_RS_OK;
  cudaGetLastError();  // clear a non-sticky launch error
  return MOE_RS_ERR_LAUNCH;
}

}  // namespace mrs
