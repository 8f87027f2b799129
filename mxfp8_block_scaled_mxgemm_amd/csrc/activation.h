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

__device__ __forceinline__ float activate(int act, float z)
{
    switch (act) {
    case kActRelu: return z != z ? z : fmaxf(z, 0.f);
    case kActGelu: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case kActGeluTanh: return z * sigmoid(kGeluC * (z + kGeluA * z * z * z));
    case kActSilu: return z * sigmoid(z);
    default: return z;
    }
}

__device__ __forceinline__ void activate8(int act, float (&z)[8])
{
    if (act == kActNone)
        return;
#pragma unroll
    for (int u = 0; u < 8; ++u)
        z[u] = activate(act, z[u]);
}

// act(z) in y; returns act'(z) (relu: 0 at 0).
__device__ __forceinline__ float activate_grad(int act, float z, float& y)
{
    switch (act) {
    case kActRelu:
        y = z != z ? z : fmaxf(z, 0.f);
        return z > 0.f ? 1.f : 0.f;
    case kActGelu: {
        const float cdf = 0.5f * (1.f + erff(z * 0.70710678118654752f));
        y = z * cdf;
        return cdf + z * 0.3989422804014327f * __expf(-0.5f * z * z);
    }
    case kActGeluTanh: {
        const float s = sigmoid(kGeluC * (z + kGeluA * z * z * z));
        y = z * s;
        return s + z * s * (1.f - s) * kGeluC * (1.f + 3.f * kGeluA * z * z);
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

}  // namespace mxg
