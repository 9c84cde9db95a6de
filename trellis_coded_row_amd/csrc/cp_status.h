// The C-ABI layer's view of a HIP result, shared by its source files.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/cp.h"

namespace cpk {

// CP_OK, or the status of a failed HIP call, whose code is kept for
// cp_last_hip_error and taken off the runtime's per-thread "last error".
cp_status status_of(hipError_t e);

}  // namespace cpk
