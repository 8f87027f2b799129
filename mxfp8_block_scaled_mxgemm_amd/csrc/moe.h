// Internal interface between the host side and the kernels of the expert
// layer: tokens sorted by expert and back.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxg {

// Element types of tokens (the values of MXGEMM_TYPE_*)
constexpr int kBF16 = 0, kFP16 = 1, kFP32 = 2;

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortMaxExperts = 1024;
constexpr int kSortMaxBlocks = 128;
constexpr int kGroupK = 128;      // granule of a k_offsets segment (one MFMA K-step)

struct SortArgs {
    const void* ids;              // [pairs] int32 or int64
    int64_t pairs;
    int experts, ids64;
    int iters, blocks;            // 64-pair pieces per wave; work-groups
    int32_t* offsets;             // [experts + 1]
    int32_t* k_offsets;           // [experts + 1]
    int32_t* row_of;              // [pairs]
    int32_t* pair_of;             // [pairs]
    uint32_t* ws;                 // blocks > 1: [blocks][experts + 1]
};

// Rows of `cols` elements; strides in elements.  live: the number of kept
// rows (offsets[experts]); row_of[t * k + j] >= *live is a dropped pair.
struct TokenArgs {
    const int32_t* live;
    const int32_t* row_of;        // [tokens][k]
    int64_t tokens;
    int64_t all_rows;             // tokens k of the call; a launch may hold fewer tokens
    int k, cols;
    const void* x;                // dispatch: tokens; combine: residual (may be null); backward: d_out
    int64_t ld_x;
    const void* rows;             // combine, combine backward: read
    int64_t ld_rows;
    const float* weights;         // [tokens][k] or null (all one)
    void* out;                    // dispatch, combine backward: rows; combine: tokens
    int64_t ld_out;
    float* d_weights;             // combine backward: [tokens][k]
    uint8_t* q;                   // dispatch to MXFP8: codes [tokens k][cols]
    uint8_t* s;                   // and scale bytes [tokens k][cols / 32]
    int fmt;
};

hipError_t launch_sort(const SortArgs& a, hipStream_t stream);
hipError_t launch_dispatch(const TokenArgs& a, int type, hipStream_t stream);
hipError_t launch_dispatch_mx(const TokenArgs& a, int type, hipStream_t stream);
hipError_t launch_combine(const TokenArgs& a, int type, hipStream_t stream);
hipError_t launch_combine_backward(const TokenArgs& a, int type, hipStream_t stream);

}  // namespace mxg
