// Tokens of one expert in chunks of 128, as k_offsets lays them out.
#pragma once

#include <hip/hip_runtime.h>

namespace mxg {

constexpr int kSegmentRows = 128;

// First token of chunk `chunk` and the end of its expert; false past the
// last segment (and past the last chunk, whatever k_offsets holds).  Without
// offsets: of the rows as one segment.
template <class Args>
__device__ __forceinline__ bool segment_rows(const Args& p, int chunk, int& row0, int& end)
{
    row0 = chunk * kSegmentRows;
    end = p.rows;
    if (!p.offsets)
        return true;
    // the expert whose padded segment holds this chunk
    const int at = row0;
    if (chunk >= p.chunks || at >= p.k_offsets[p.groups])
        return false;
    int lo = 0, hi = p.groups;              // k_offsets[lo] <= at < k_offsets[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.k_offsets[mid] <= at)
            lo = mid;
        else
            hi = mid;
    }
    row0 = p.offsets[lo] + at - p.k_offsets[lo];
    end = p.offsets[lo + 1];
    end = end < p.rows ? end : p.rows;
    row0 = row0 < 0 ? 0 : row0;
    return true;
}

}  // namespace mxg
