// What the gate, the norm and the fp8 products share besides mdc_common.h.
#pragma once

#include "mdc_common.h"

namespace {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// A grid of n workgroups in two dimensions: a launch takes fewer than 2^32
// threads along one.  The kernel's number is grid_block(), which may be >= n.
constexpr unsigned kGridRow = 1u << 20;
inline dim3 grid_of(int64_t n) {
  return n <= kGridRow ? dim3((unsigned)n) : dim3(kGridRow, (unsigned)((n + kGridRow - 1) / kGridRow));
}
__device__ __forceinline__ int64_t grid_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

}  // namespace
