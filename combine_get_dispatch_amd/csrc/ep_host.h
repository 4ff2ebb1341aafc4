// Host-side helpers shared by the files that hold entry points beside
// ep_api.hip.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "ep.h"

namespace ep {

// Defined with the other entry points (ep_api.hip): records the message
// ep_last_error() returns on this thread and returns st.
ep_status_t set_error(ep_status_t st, const char *message);

inline ep_status_t failf(ep_status_t st, const char *fmt, ...) {
  char text[320];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  return set_error(st, text);
}

// The status of the launches just made on this thread.
inline ep_status_t launched(const char *what) {
  const hipError_t err = hipGetLastError();
  if (err == hipSuccess) return EP_OK;
  return failf(EP_ERR_HIP, "%s: %s", what, hipGetErrorString(err));
}

inline bool aligned_to(const void *p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// Whether two arrays share bytes; NULL shares none.
inline bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && p < q + (uintptr_t)b_bytes && q < p + (uintptr_t)a_bytes;
}

}  // namespace ep

#define EP_TRY(expr)                \
  do {                              \
    const ep_status_t st_ = (expr); \
    if (st_ != EP_OK) return st_;   \
  } while (0)
