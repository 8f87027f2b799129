// Byte matrices transposed: operands that come with their other axis
// contiguous, laid out for the product.
#include "device_util.h"
#include "linear.h"

namespace mxg {

// dst[b][c][r] = src[b][r][c].  A work-group takes 128 x 128 bytes; a thread
// takes 4 rows x 16 columns, turned in registers into one word of four row
// bytes per column, so LDS and the stores move words and 16-byte pieces.  In
// LDS a column's eight 16-byte pieces are XOR-swizzled by bits 4-6 of the
// column: the eight threads that write columns 16 apart meet different banks.
// Bound by memory, every byte read and written once: 24 x 2048 x 2048, 35 us
// (201 MB, 5.7 TB/s); 7168 x 4096, 15 us.
constexpr int kTurn = 128;

// Word w of column c.
__device__ __forceinline__ int turn_at(int c, int w) { return c * (kTurn / 4) + (w ^ (4 * (c >> 4))); }

__global__ void __launch_bounds__(256) transpose_kernel(TransposeArgs p)
{
    __shared__ __attribute__((aligned(16))) uint32_t t[kTurn * kTurn / 4];
    const int tid = threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.y * kTurn, c0 = (int64_t)blockIdx.x * kTurn;
    const uint8_t* src = p.src + blockIdx.z * p.src_batch;
    uint8_t* dst = p.dst + blockIdx.z * p.rows * p.cols;
    {
        const int cl = (tid & 7) * 16, rl = (tid >> 3) * 4;
        const int64_t c = c0 + cl;
        uint32_t in[4][4];
        const uint8_t* row = src + (r0 + rl) * p.ld_src + c;
        if (r0 + kTurn <= p.rows && c0 + kTurn <= p.cols) {     // no lane branches: the loads go out together
#pragma unroll
            for (int i = 0; i < 4; ++i)
                __builtin_memcpy(in[i], row + i * p.ld_src, 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const uint32_t x = r0 + rl + i < p.rows && c + u < p.cols ? row[i * p.ld_src + u] : 0;
                    in[i][u >> 2] = (u & 3 ? in[i][u >> 2] : 0) | x << (8 * (u & 3));
                }
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            // bytes of rows 0, 1 and 2, 3 interleaved, then the halves
            const uint32_t lo01 = __builtin_amdgcn_perm(in[1][w], in[0][w], 0x05010400u);
            const uint32_t hi01 = __builtin_amdgcn_perm(in[1][w], in[0][w], 0x07030602u);
            const uint32_t lo23 = __builtin_amdgcn_perm(in[3][w], in[2][w], 0x05010400u);
            const uint32_t hi23 = __builtin_amdgcn_perm(in[3][w], in[2][w], 0x07030602u);
            const int o = turn_at(cl, rl >> 2) + 4 * w * (kTurn / 4);       // cl: multiples of 16
            t[o] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
            t[o + kTurn / 4] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
            t[o + 2 * (kTurn / 4)] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
            t[o + 3 * (kTurn / 4)] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
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
        const u32x4 v = *reinterpret_cast<const u32x4*>(t + turn_at(cl, rl >> 2));
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
