// Host helpers shared by the C ABI entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tdi8.h"

namespace tdi8 {

// Records the error for tdi8_last_hip_error and returns TDI8_ERR_HIP.
int hip_fail(hipError_t e);

// Initialises the current device; its compute units, or a status.
int device_units(int *num_cu);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool overlaps(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) { return a0 < b1 && b0 < a1; }

}  // namespace tdi8
