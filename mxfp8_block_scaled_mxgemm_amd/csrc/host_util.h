// Error reporting and pointer checks shared by the C entry points.
#pragma once

#include <hip/hip_runtime.h>

namespace mxg {

// Sets the calling thread's error message and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// MXGEMM_OK if p is memory that kernels on `device` can access.
int gpu_accessible(const void* p, const char* name, int device);

}  // namespace mxg

// A failing HIP call is reported through the return code and the message;
// the thread's last HIP error is cleared so that a later, unrelated launch
// check does not report it again.
#define HIP_TRY(expr)                                                                   \
    do {                                                                                \
        hipError_t e_ = (expr);                                                         \
        if (e_ != hipSuccess) {                                                         \
            (void)hipGetLastError();                                                    \
            return mxg::fail(MXGEMM_EHIP, "%s failed: %s", #expr, hipGetErrorString(e_)); \
        }                                                                               \
    } while (0)
