// host.hpp -- host helpers shared by the files of the C ABI (implemented in api.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace effort {

// Records a failed HIP status for effort_last_hip_error(); true if it is one.
bool hip_failed(hipError_t e);
// EFFORT_OK or EFFORT_EHIP, recorded.
int status_of(hipError_t e);
// Compute units of the current device (cached per device).
int cu_count();
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace effort
