// Activations and their derivatives in FP32.  The smooth ones are written
// with exponentials of the sign that cannot cancel: gelu_tanh as
// z / (1 + exp(-2 u)), which equals 0.5 z (1 + tanh u).
#pragma once

#include "device_util.h"
#include "linear.h"

namespace mxg {

// 1 / (1 + exp(-x)): 0 and 1 at the infinities
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }

constexpr float kGeluC = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float relu(float z) { return z != z ? z : fmaxf(z, 0.f); }
// The normal distribution function 0.5 (1 + erf(z / sqrt 2)).  Its tail is
// exp(-z^2 / 2) times a smooth function of |z|, which is fitted as a polynomial
// in t = 1 / (1 + 0.35 |z|): least largest relative error over |z| <= 15
// (3.2e-8; beyond, the tail is below FP32's range), by iteratively reweighted
// least squares.  No branches, as a full-precision erf has: the epilogue is
// bound by instructions.  The tail is formed on the side where it is small, so
// nothing cancels there.  Evaluated in FP32: 1.8e-8 off in rms over gelu of
// N(0, 1), and by 7e-7 of the value at z = -3, 7e-6 at -12 (the rounding of
// z^2 / 2).  Four steps fewer, good to 1.5e-7 absolute, save 0.6% of 8192 x
// 8192 x 8192 native with gelu and 3% of x 2048.
__device__ __forceinline__ float normal_cdf(float z)
{
    const float t = __builtin_amdgcn_rcpf(1.f + 0.35f * fabsf(z));
    float p = 0.144060203f - 0.0291637983f * t;
    p = -0.255900672f + t * p;
    p = 0.159391613f + t * p;
    p = -0.0232629887f + t * p;
    p = 0.105574466f + t * p;
    p = 0.119815577f + t * p;
    p = 0.139864326f + t * p;
    p = 0.139621259f + t * p;
    const float tail = t * p * __expf(-0.5f * z * z);
    return z < 0.f ? tail : 1.f - tail;
}
__device__ __forceinline__ float gelu(float z) { return z * normal_cdf(z); }
__device__ __forceinline__ float gelu_tanh(float z) { return z * sigmoid(kGeluC * z * (1.f + kGeluA * z * z)); }
__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }

// act(z) of N values: one branch for all of them, eight at a time (the fence
// keeps the scheduler from holding the temporaries of all of them at once).
template <int N, class F>
__device__ __forceinline__ void by_eights(float (&z)[N], const F& f)
{
#pragma unroll
    for (int k = 0; k < N; k += 8) {
#pragma unroll
        for (int u = k; u < k + 8 && u < N; ++u)
            z[u] = f(z[u]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int N>
__device__ __forceinline__ void activate(int act, float (&z)[N])
{
    if (act == kActNone)
        return;
    if (act == kActSilu)
        by_eights(z, silu);
    else if (act == kActGeluTanh)
        by_eights(z, gelu_tanh);
    else if (act == kActRelu)
        by_eights(z, relu);
    else
        by_eights(z, gelu);
}

// act(z) in y; returns act'(z) (relu: 0 at 0).
__device__ __forceinline__ float activate_grad(int act, float z, float& y)
{
    switch (act) {
    case kActRelu:
        y = relu(z);
        return z > 0.f ? 1.f : 0.f;
    case kActGelu: {
        const float cdf = normal_cdf(z);
        y = z * cdf;
        return cdf + z * 0.3989422804014327f * __expf(-0.5f * z * z);
    }
    case kActGeluTanh: {
        // s is 0 or 1 long before |z| = 100; past it z * z may overflow, and
        // 0 times infinity must not come of it
        const float zz = fminf(z * z, 1e4f);
        const float s = sigmoid(kGeluC * z * (1.f + kGeluA * zz));
        y = z * s;
        return s + z * s * (1.f - s) * kGeluC * (1.f + 3.f * kGeluA * zz);
    }
    case kActSilu: {
        const float s = sigmoid(z);
        y = z * s;
        return s * (1.f + z * (1.f - s));
    }
    default:
        y = z;
        return 1.f;
    }
}

// z becomes act'(z), y gets act(z): one branch for all values.
template <int N>
__device__ __forceinline__ void activate_grads(int act, float (&z)[N], float (&y)[N])
{
    auto each = [&](int which) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < N; ++u)
            z[u] = activate_grad(which, z[u], y[u]);
    };
    if (act == kActSilu)
        each(kActSilu);
    else if (act == kActGeluTanh)
        each(kActGeluTanh);
    else if (act == kActGelu)
        each(kActGelu);
    else if (act == kActRelu)
        each(kActRelu);
    else
        each(kActNone);
}

}  // namespace mxg
