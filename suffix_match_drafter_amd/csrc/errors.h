// errors.h -- the thread-local error text behind sfx_last_error (internal to libsfx).
#pragma once

#include <hip/hip_runtime.h>

namespace sfx {

// Stores the formatted text and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// SFX_EHIP with the runtime's text for `e`.
int hip_fail(hipError_t e, const char* what);

}  // namespace sfx

#define HIP_OR_RETURN(expr, what)                         \
  do {                                                    \
    hipError_t e_ = (expr);                               \
    if (e_ != hipSuccess) return sfx::hip_fail(e_, what); \
  } while (0)
