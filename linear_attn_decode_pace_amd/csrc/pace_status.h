// Status and argument helpers shared by the files that define C entry points.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/pace.h"

#define PACE_API extern "C" __attribute__((visibility("default")))

namespace pace {

// set the calling thread's message and return `code`
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// clear the message; PACE_OK
int ok();
// a HIP error as a status; clears the runtime's sticky last error
int hip_fail(hipError_t e, const char *what);

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// batch, heads and state sizes the recurrent-state kernels are built for
int check_shape(int32_t batch, int32_t heads, int32_t d_k, int32_t d_v);
int check_dtype(int32_t dt);

}  // namespace pace
