// Loads and stores of eight consecutive elements as FP32 values.
#pragma once

#include <hip/hip_fp16.h>

#include "device_util.h"
#include "moe.h"

namespace mxg {

// Storage of one element type and its FP32 value.  Stores round to nearest
// even, once.
template <int TYPE>
struct Element;

template <>
struct Element<kBF16> {
    typedef uint16_t T;
    __device__ static __forceinline__ float get(T v) { return __uint_as_float((uint32_t)v << 16); }
    __device__ static __forceinline__ T put(float f) { return f32_to_bf16_rne(f); }
};
template <>
struct Element<kFP16> {
    typedef uint16_t T;
    __device__ static __forceinline__ float get(T v) { return (float)__builtin_bit_cast(_Float16, v); }
    __device__ static __forceinline__ T put(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
};
template <>
struct Element<kFP32> {
    typedef float T;
    __device__ static __forceinline__ float get(T v) { return v; }
    __device__ static __forceinline__ T put(float f) { return f; }
};

// N consecutive elements.  Loaded and stored through a copy of their bytes,
// so any element-aligned address is allowed (the memory unit takes 16-byte
// accesses at any address).
template <int TYPE, int N>
struct Pack {
    typedef typename Element<TYPE>::T T;
    T v[N];
    __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(v, p, sizeof(v)); }
    __device__ __forceinline__ void store(T* p) const { __builtin_memcpy(p, v, sizeof(v)); }
    __device__ __forceinline__ float get(int i) const { return Element<TYPE>::get(v[i]); }
    __device__ __forceinline__ void put(int i, float f) { v[i] = Element<TYPE>::put(f); }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = 0;
    }
};

// A row of `cols` elements as pieces of V: the last one is moved back to
// end with the row (it then repeats elements of the piece before it).
template <int V>
__device__ __forceinline__ int piece_start(int piece, int cols)
{
    const int c = piece * V;
    return c + V <= cols ? c : cols - V;
}

}  // namespace mxg
