// Host-side helpers of the C entry points (defined in api.hip): the calling
// thread's error message and the checks the entry points share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

// Set the calling thread's message and return the status.
nvfp4_status fail(nvfp4_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clear it: NVFP4_OK.
nvfp4_status ok();
const char* last_error();
nvfp4_status hip_status(hipError_t e, const char* what);
bool aligned(const void* p, uintptr_t a);
// The GEMMs' rules on K.
nvfp4_status check_k(int64_t K);

}  // namespace nvfp4
