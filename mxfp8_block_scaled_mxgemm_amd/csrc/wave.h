// Sums and maxima over the 64 lanes of a wave, on the vector unit's own lane
// permutations (no LDS); every lane of the wave takes part.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxg {

// DPP controls: lanes 1 0 3 2, lanes 2 3 0 1, halves of sixteen mirrored,
// sixteen mirrored, the row before's last lane, the half before's last lane
enum { kDppSwap1 = 0xB1, kDppSwap2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140, kDppBcast15 = 0x142,
       kDppBcast31 = 0x143 };

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, ROWS == 0xF);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float x)
{
    return __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(x)));
}

// over sixteen consecutive lanes, in each of them
__device__ __forceinline__ float row16_sum(float x)
{
    x += dpp<kDppSwap1>(x);
    x += dpp<kDppSwap2>(x);
    x += dpp<kDppHalfMirror>(x);
    return x + dpp<kDppMirror>(x);
}
__device__ __forceinline__ uint32_t row16_max(uint32_t x)
{
    x = max(x, dpp<kDppSwap1>(x));
    x = max(x, dpp<kDppSwap2>(x));
    x = max(x, dpp<kDppHalfMirror>(x));
    return max(x, dpp<kDppMirror>(x));
}

// over the wave, the same in all lanes
__device__ __forceinline__ float wave_sum(float x)
{
    x = row16_sum(x);
    x += dpp<kDppBcast15, 0xA>(x);
    x += dpp<kDppBcast31, 0xC>(x);
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 63));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    x = row16_max(x);
    x = max(x, dpp<kDppBcast15, 0xA>(x));
    x = max(x, dpp<kDppBcast31, 0xC>(x));
    return __builtin_amdgcn_readlane(x, 63);
}

}  // namespace mxg
