// What the host entry points share: the calling thread's error text and small checks
// (defined in api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sdm_dense.h"

namespace sdm {

extern thread_local char g_err[512];   // sdm_last_error()'s text

// Stores the text and returns code.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char *what);

// CUs of the current device, after its one-time setup (kernel attributes).
int device_cus(int *cus);

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace sdm
