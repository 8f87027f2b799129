// Byte matrices transposed: operands that come with their other axis
// contiguous, laid out for the product.
#include "device_util.h"
#include "linear.h"

namespace mxg {

// dst[b][c][r] = src[b][r][c].  A work-group takes 128 x 128 bytes; a thread
// takes 4 rows x 16 columns, turned in registers into one word of four row
// bytes per column, so LDS and the stores move words and 16-byte pieces.
// Rows of LDS are 36 words apart: 16-byte aligned, spread over the banks.
// Bound by memory: every byte read and written once.
constexpr int kTurn = 128, kTurnLd = 36;

__global__ void __launch_bounds__(256) transpose_kernel(TransposeArgs p)
{
    __shared__ __attribute__((aligned(16))) uint32_t t[kTurn * kTurnLd];
    const int tid = threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.y * kTurn, c0 = (int64_t)blockIdx.x * kTurn;
    const uint8_t* src = p.src + blockIdx.z * p.src_batch;
    uint8_t* dst = p.dst + blockIdx.z * p.rows * p.cols;
    {
        const int cl = (tid & 7) * 16, rl = (tid >> 3) * 4;
        const int64_t c = c0 + cl;
        uint32_t in[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + rl + i;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                in[i][w] = 0;
            if (r >= p.rows)
                continue;
            const uint8_t* row = src + r * p.ld_src + c;
            if (c + 16 <= p.cols) {
                __builtin_memcpy(in[i], row, 16);
            } else {
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    if (c + u < p.cols)
                        in[i][u >> 2] |= (uint32_t)row[u] << (8 * (u & 3));
            }
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            // bytes of rows 0, 1 and 2, 3 interleaved, then the halves
            const uint32_t lo01 = __builtin_amdgcn_perm(in[1][w], in[0][w], 0x05010400u);
            const uint32_t hi01 = __builtin_amdgcn_perm(in[1][w], in[0][w], 0x07030602u);
            const uint32_t lo23 = __builtin_amdgcn_perm(in[3][w], in[2][w], 0x05010400u);
            const uint32_t hi23 = __builtin_amdgcn_perm(in[3][w], in[2][w], 0x07030602u);
            uint32_t* o = t + (cl + 4 * w) * kTurnLd + (rl >> 2);
            o[0 * kTurnLd] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
            o[1 * kTurnLd] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
            o[2 * kTurnLd] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
            o[3 * kTurnLd] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
        }
    }
    __syncthreads();
    const int rl = (tid & 7) * 16;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int cl = (tid >> 3) + 32 * k;
        const int64_t c = c0 + cl, r = r0 + rl;
        if (c >= p.cols || r >= p.rows)
            continue;
        const u32x4 v = *reinterpret_cast<const u32x4*>(t + cl * kTurnLd + (rl >> 2));
        uint8_t* out = dst + c * p.rows + r;
        if (r + 16 <= p.rows) {
            __builtin_memcpy(out, &v, 16);
        } else {
#pragma unroll
            for (int u = 0; u < 16; ++u)
                if (r + u < p.rows)
                    out[u] = (uint8_t)(v[u >> 2] >> (8 * (u & 3)));
        }
    }
}

hipError_t launch_transpose(const TransposeArgs& a, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.cols + kTurn - 1) / kTurn), (unsigned)((a.rows + kTurn - 1) / kTurn),
                    (unsigned)a.batch);
    hipLaunchKernelGGL(transpose_kernel, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxg
