// FP32 -> MXFP8 conversion rules (codes and block exponents) shared by the
// kernels that quantise.
#pragma once

#include "device_util.h"

namespace mxg {

// E4M3 (OCP "FN") code of a non-NaN float, round-to-nearest-even, sign of
// zero kept; magnitudes above 448 after rounding (infinities included)
// saturate to 448 (code 0x7E).  Normal range: keep 3 mantissa bits and
// round on the 20 dropped bits; below 2^-6 the grid step is 2^-9, so
// y * 512 rounded to an integer is the code (8 is the smallest normal,
// code 0x08).
__device__ __forceinline__ uint32_t e4m3_rne(float y)
{
    const uint32_t u = __float_as_uint(y);
    const uint32_t sign = (u >> 24) & 0x80u;
    const uint32_t a = u & 0x7FFFFFFFu;
    uint32_t code;
    if (a < 0x3C800000u) {                       // |y| < 2^-6
        code = (uint32_t)rintf(__uint_as_float(a) * 512.0f);
    } else {
        const uint32_t keep = (a >> 20) & 7u;
        const uint32_t rest = a & 0xFFFFFu;
        code = (((a >> 23) - 120u) << 3) | keep;  // biased exponent 127 -> 7
        if (rest > 0x80000u || (rest == 0x80000u && (keep & 1u)))
            code += 1u;
        if (code > 0x7Eu)
            code = 0x7Eu;
    }
    return code | sign;
}

// E5M2 (OCP, bias 15) code of a float, round-to-nearest-even, saturating at
// the largest finite value 57344 (code 0x7B) instead of producing infinity.
// Normal range: keep 2 mantissa bits and round on the 21 dropped bits;
// below 2^-14 the grid step is 2^-16, so y * 65536 rounded to an integer is
// the code (4 is the smallest normal, code 0x04).
__device__ __forceinline__ uint32_t e5m2_rne(float y)
{
    const uint32_t u = __float_as_uint(y);
    const uint32_t sign = (u >> 24) & 0x80u;
    const uint32_t a = u & 0x7FFFFFFFu;
    uint32_t code;
    if (a < 0x38800000u) {                       // |y| < 2^-14
        code = (uint32_t)rintf(__uint_as_float(a) * 65536.0f);
    } else {
        const uint32_t keep = (a >> 21) & 3u;
        const uint32_t rest = a & 0x1FFFFFu;
        code = (((a >> 23) - 112u) << 2) | keep;  // biased exponent 127 -> 15
        if (rest > 0x100000u || (rest == 0x100000u && (keep & 1u)))
            code += 1u;
        if (code > 0x7Bu)
            code = 0x7Bu;
    }
    return code | sign;
}

// Smallest e with fmax * 2^e >= amax, clamped to [-127, 127], for the
// format's largest finite value fmax = 1.75 * 2^EMAX (448: EMAX = 8 for
// E4M3; 57344: EMAX = 15 for E5M2).  With amax = 1.m * 2^x, e = x - EMAX
// when 1.m <= 1.75, else x - EMAX + 1.  Zero and float32 subnormals give
// -127 (the clamp), +inf gives 127 (the clamp of an unbounded e); amax is
// never NaN here (NaN blocks are handled by the caller).
template <int EMAX>
__device__ __forceinline__ int e8m0_exponent(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int ex = (int)(u >> 23);
    if (ex == 0)
        return -127;
    if (ex == 255)
        return 127;
    int e = ex - 127 - EMAX + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = e < -127 ? -127 : e;
    return e > 127 ? 127 : e;
}

template <int F>
__device__ __forceinline__ uint32_t fp8_rne(float y)
{
    return F == kE5M2 ? e5m2_rne(y) : e4m3_rne(y);
}

// A block of 32 from its amax, given as the largest |x| bit pattern: for
// non-negative floats the integer order is the numeric order, and every NaN
// pattern lies above +inf (0x7F800000), so a NaN anywhere in the block is
// seen (a float max would drop it).
struct MxScale {
    int e;              // elements are divided by 2^e
    uint8_t byte;       // E8M0
    bool nan;
};

template <int F>
__device__ __forceinline__ MxScale mx_scale(uint32_t amax_bits)
{
    MxScale s;
    s.nan = amax_bits > 0x7F800000u;
    s.e = s.nan ? 0 : e8m0_exponent<F == kE5M2 ? 15 : 8>(__uint_as_float(amax_bits));
    s.byte = s.nan ? 0xFF : (uint8_t)(s.e + 127);
    return s;
}

// Codes of four elements of the block, first in the low byte, by the
// conversion instructions (round to nearest even, subnormal codes kept;
// elements within the format's range after scaling, as they are, but for
// infinities, which the clamp saturates).  Same codes as fp8_rne.
template <int F>
__device__ __forceinline__ uint32_t mx_codes(const MxScale& s, float a, float b, float c, float d)
{
    constexpr float kMax = F == kE5M2 ? 57344.f : 448.f;
    a = __builtin_amdgcn_fmed3f(ldexpf(a, -s.e), -kMax, kMax);
    b = __builtin_amdgcn_fmed3f(ldexpf(b, -s.e), -kMax, kMax);
    c = __builtin_amdgcn_fmed3f(ldexpf(c, -s.e), -kMax, kMax);
    d = __builtin_amdgcn_fmed3f(ldexpf(d, -s.e), -kMax, kMax);
    int w;
    if constexpr (F == kE5M2) {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    }
    return s.nan ? 0x7F7F7F7Fu : (uint32_t)w;
}

// max of x over four consecutive lanes (all of them active).
__device__ __forceinline__ uint32_t quad_max(uint32_t x)
{
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));    // lanes 1, 0, 3, 2
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true)); // lanes 2, 3, 0, 1
}

}  // namespace mxg
