// Error reporting and argument checks shared by the C entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "mxgemm_seg.h"

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

#define TRY(expr)                 \
    do {                          \
        const int rc_ = (expr);   \
        if (rc_ != MXGEMM_OK)     \
            return rc_;           \
    } while (0)

namespace mxg {

// Compute units of the current device, which must be a gfx950; looked up
// once per device.
inline int current_device(int* dev, int* cus)
{
    constexpr int kMaxDevices = 64;
    static std::atomic<int> known[kMaxDevices];     // 0: not looked up, else compute units
    HIP_TRY(hipGetDevice(dev));
    if (*dev < 0 || *dev >= kMaxDevices)
        return fail(MXGEMM_EUNSUPPORTED, "device index %d out of range", *dev);
    *cus = known[*dev].load(std::memory_order_relaxed);
    if (*cus == 0) {
        hipDeviceProp_t prop;
        HIP_TRY(hipGetDeviceProperties(&prop, *dev));
        if (strncmp(prop.gcnArchName, "gfx950", 6) != 0)
            return fail(MXGEMM_EUNSUPPORTED, "device %d is %s; this library is built for gfx950", *dev,
                        prop.gcnArchName);
        *cus = prop.multiProcessorCount;
        known[*dev].store(*cus, std::memory_order_relaxed);
    }
    return MXGEMM_OK;
}

struct Buffer {
    const void* p;
    const char* name;
    int align;
    bool optional;
};

template <size_t N>
int check_buffers(const Buffer (&b)[N], int dev)
{
    for (const Buffer& x : b) {
        if (!x.p) {
            if (x.optional)
                continue;
            return fail(MXGEMM_EINVAL, "%s is NULL", x.name);
        }
        if ((uintptr_t)x.p % x.align != 0)
            return fail(MXGEMM_EINVAL, "%s must be %d-byte aligned", x.name, x.align);
        const int rc = gpu_accessible(x.p, x.name, dev);
        if (rc != MXGEMM_OK)
            return rc;
    }
    return MXGEMM_OK;
}

inline int check_stride(const char* name, int64_t ld, int64_t cols)
{
    if (ld < cols)
        return fail(MXGEMM_EINVAL, "row stride %lld of %s is less than its %lld columns", (long long)ld, name,
                    (long long)cols);
    return MXGEMM_OK;
}

}  // namespace mxg
