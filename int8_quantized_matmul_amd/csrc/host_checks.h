// Host-side checks shared by the C-ABI layers (api.cpp, adapt_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/i8mm.h"

namespace i8mm {

// I8MM_OK if the current HIP device is a gfx950, else I8MM_EDEVICE.
i8mm_status check_device();

inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline bool aligned16(const void* p) { return aligned_to(p, 16); }

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

inline i8mm_status launched(hipError_t e) { return e == hipSuccess ? I8MM_OK : I8MM_ELAUNCH; }

}  // namespace i8mm
