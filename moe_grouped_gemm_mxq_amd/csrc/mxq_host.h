// Host-side helpers shared by the units that define entry points: the
// thread-local error message, the gfx950 device gate and the launch check
// (defined in mxq_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxq.h"

namespace mxq {

// sets the thread's error message and returns st
mxq_status fail(mxq_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// clears the message
mxq_status ok();
// MXQ_OK iff the current HIP device is gfx950
mxq_status check_current_device();
// status of a launch that returned e
mxq_status launched(hipError_t e, const char* what);

inline bool aligned_to(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace mxq

#define MXQ_REQUIRE(cond, ...) \
  do {                         \
    if (!(cond)) return fail(MXQ_ERR_INVALID_ARGUMENT, __VA_ARGS__); \
  } while (0)

#define MXQ_REQUIRE_DEVICE()                     \
  do {                                           \
    mxq_status _s = check_current_device();      \
    if (_s != MXQ_OK) return _s;                 \
  } while (0)
