// errors.h -- the calling thread's error message (gr_last_error), set by the
// entry points of every source file of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include "gr.h"

namespace gr {

// Record a printf-style message for gr_last_error and return `s`.
gr_status fail(gr_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gr_status hip_fail(hipError_t e, const char* what);

}  // namespace gr

#define HIP_TRY(expr, what)                       \
    do {                                          \
        hipError_t e_ = (expr);                   \
        if (e_ != hipSuccess) return gr::hip_fail(e_, what); \
    } while (0)
