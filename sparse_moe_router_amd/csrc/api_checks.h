// Argument checks and error records shared by the C-ABI sources.
#pragma once

#include "moe_internal.h"
#include "moe_layer.h"
#include "regions.h"

namespace moe {

// MOE_ERR_HIP, with e kept for moe_last_hip_error() of this thread.
moe_status_t hip_fail(hipError_t e);

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace moe
