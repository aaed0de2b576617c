// What the host entry points share: the calling thread's error text and small checks
// (defined in api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sdm_dense.h"
#include "sdm_linear.h"

namespace sdm {

extern thread_local char g_err[512];   // sdm_last_error()'s text

// Stores the text and returns code.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char *what);

// CUs of the current device, after its one-time setup (kernel attributes).
int device_cus(int *cus);

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// An array of dense rows of `width` elements of `es` bytes, up to three axes of strides >= 0 (in elements) over them.
struct Extent {
    struct Axis {
        int64_t n, stride;
    };
    const void *data;
    Axis axis[3];
    int64_t width;
    int es;
    // Whether its rows are one dense run in the axes' order.
    bool dense() const;
    // Whether one of its rows meets the n bytes at p. (Exact, but for axes that interleave, which count as solid.)
    bool meets(const void *p, size_t n) const;
};
// ... and of two dense runs.
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

}  // namespace sdm
