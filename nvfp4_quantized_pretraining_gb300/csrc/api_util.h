// Host-side helpers shared by the units that hold C-ABI entry points (defined in api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "nvfp4_gb300.h"

namespace nvfp4 {

// Records the thread-local message that fp4_last_error() returns, and returns st.
fp4_status fail(fp4_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

#define CUDA_TRY(expr)                                                                      \
  do {                                                                                      \
    cudaError_t e_ = (expr);                                                                \
    if (e_ != cudaSuccess)                                                                  \
      return fail(FP4_ERR_CUDA, "%s failed: %s", #expr, cudaGetErrorString(e_));            \
  } while (0)

// SMs of the current device.
int sm_count();

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }
inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace nvfp4
