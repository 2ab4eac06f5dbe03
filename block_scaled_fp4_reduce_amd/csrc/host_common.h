// host_common.h -- host-side helpers shared by the entry points: pointer
// alignment, launch status and the device's size.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp4q.h"

namespace fp4q {

constexpr int64_t kMaxElems = (int64_t)1 << 40;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Status of the launches an entry point queued (each launch reports its own
// result, see launch(); the thread's last-error state is never read).
inline int launched(hipError_t e) { return e == hipSuccess ? FP4_OK : FP4_E_HIP; }

// First failure of a sequence of launches.
inline hipError_t first(hipError_t a, hipError_t b) { return a != hipSuccess ? a : b; }

// Compute units of the current device (queried once per device; 256 on MI355X).
inline int num_cus() {
  static int cached[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (cached[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cached[dev] = n;
  }
  return cached[dev];
}

}  // namespace fp4q
