// The epilogue of a product whose K was split over work-groups.
#include "linear_impl.h"

namespace mxg {

// Eight outputs of a row per thread: the splits' sums added in order, then
// the epilogue.  With MXFP8 output four lanes share a block; work-groups are
// whole blocks wide, and every lane takes part.  A launch of its own, since
// the last of a tile's splits could only be found with counters that are
// cleared before each call.  Bound by latency: 4.2 us for eight splits of 64 x
// 2048.
template <bool GATED>
__global__ void __launch_bounds__(256) linear_finish_kernel(LinArgs p)
{
    const int cols = GATED ? p.N / 2 : p.N;
    const int per = (cols + 31) / 32 * 4;               // eights per row, whole blocks
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t total = (int64_t)p.rows * per;
    const int row = (int)((i < total ? i : total - 1) / per);
    const int c = 8 * (int)((i < total ? i : total - 1) % per);
    const bool ok = i < total && c < cols;
    Bias8<GATED> bias;
    bias.load(p, 0, c, cols);
    const Raw8 res[1] = {residual8(p, row, p.rows, c, cols)};
    float z[8], z1[GATED ? 8 : 1];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        z[u] = 0.f;
        if constexpr (GATED)
            z1[u] = 0.f;
    }
    const float* src = p.part + (int64_t)row * p.N;
    const int64_t plane = (int64_t)p.rows * p.N;
    for (int k0 = 0; k0 < p.split; k0 += 8) {
        // eight splits' loads at a time; those past the last read it again
        Raw8 x[8][GATED ? 2 : 1];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int h = 0; h < (GATED ? 2 : 1); ++h)
                x[k][h] = raw8(kFP32, src + (k0 + k < p.split ? k0 + k : p.split - 1) * plane, h * cols, c, cols);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < p.split) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    z[u] += __uint_as_float(x[k][0].v[u >> 2][u & 3]);
                    if constexpr (GATED)
                        z1[u] += __uint_as_float(x[k][1].v[u >> 2][u & 3]);
                }
            }
    }
    finish<GATED, 1, 1>(p, 0, row, c, cols, ok ? 1 : 0, z, z1, bias, res, threadIdx.x & 63);
}

hipError_t launch_linear_finish(const LinArgs& a, hipStream_t stream)
{
    const int cols = a.gated ? a.N / 2 : a.N;
    const int64_t threads = (int64_t)a.rows * ((cols + 31) / 32 * 4);
    const dim3 grid((unsigned)((threads + 255) / 256));
    if (a.gated)
        hipLaunchKernelGGL(linear_finish_kernel<true>, grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(linear_finish_kernel<false>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxg
