// Gradient of the product's epilogue, held in MXFP8 both ways.
#include "activation.h"
#include "element.h"
#include "linear.h"
#include "quant.h"

namespace mxg {

// Eight consecutive columns [c, c + 8) of row `at` of an [.., n] array as
// FP32; zero past n.
template <int TYPE>
__device__ __forceinline__ void load8(const void* base, int64_t at, int c, int n, float (&v)[8])
{
    const typename Element<TYPE>::T* p = static_cast<const typename Element<TYPE>::T*>(base) + at + c;
    if (c + 8 <= n) {
        Pack<TYPE, 8> x;
        x.load(p);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = x.get(u);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = c + u < n ? Element<TYPE>::get(p[u]) : 0.f;
    }
}

__device__ __forceinline__ void load8(int type, const void* base, int64_t at, int c, int n, float (&v)[8])
{
    if (type == kBF16)
        load8<kBF16>(base, at, c, n, v);
    else if (type == kFP16)
        load8<kFP16>(base, at, c, n, v);
    else
        load8<kFP32>(base, at, c, n, v);
}

// A work-group takes 128 tokens x 64 columns of dz.  Thread (rl, cl) computes
// eight columns of rows rl, rl + 32, ...: dz = d_out act'(z), or, gated, the
// column's half of [d_out u act'(g), d_out act(g)].  Along the columns, four
// threads share a block of 32 and quantise it at once.  The FP32 values also
// go to LDS, transposed to [column][token] and padded so that neither side
// piles onto a few banks; there a thread takes one column's block of 32
// tokens: its sum, its scale, its codes (32 bytes; four threads write one
// column's 128 bytes).  Tokens past the expert's last one count as zeros, so
// blocks never cross experts.  Bound by memory: d_out and z are read once
// and the two bytes per element written.
constexpr int kGradRows = 128, kGradCols = 64, kGradLd = kGradRows + 1;

template <int F>
__global__ void __launch_bounds__(256) grad_kernel(GradArgs p)
{
    __shared__ float t[kGradCols * kGradLd];
    const int tid = threadIdx.x, lane = tid & 63;
    const int chunk = blockIdx.y;
    const int n0 = blockIdx.x * kGradCols;
    int row0 = chunk * kGradRows, end = p.rows;
    if (p.offsets) {
        // the expert whose padded segment holds this chunk
        const int at = chunk * kGradRows;
        if (at >= p.k_offsets[p.groups])
            return;
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
    }
    const int half = p.N / 2;
    const int cl = tid & 7, rl = tid >> 3;
    const int c = n0 + 8 * cl;                  // first of the thread's columns
#pragma unroll 1
    for (int r = rl; r < kGradRows; r += 32) {
        const int row = row0 + r;
        float dz[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            dz[u] = 0.f;
        if (row < end) {
            // the thread's columns as [first, first + 8) of d_out: a gated
            // piece that reaches over the middle is taken a column at a time
            const bool up = p.gated && c >= half;
            if (!p.gated || up || c + 8 <= half) {
                float y;
                const int width = p.gated ? half : p.N;
                const int first = up ? c - half : c;
                load8(p.d_type, p.d, row * p.ld_d, first, width, dz);
                if (p.z && (p.gated || p.act != kActNone)) {
                    float z[8], z1[8];
                    load8<kBF16>(p.z, row * p.ld_z, first, width, z);
                    if (p.gated)
                        load8<kBF16>(p.z, row * p.ld_z + half, first, width, z1);
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const float slope = activate_grad(p.act, z[u], y);
                        dz[u] *= p.gated ? (up ? y : slope * z1[u]) : slope;
                    }
                }
            } else {
#pragma unroll 1
                for (int u = 0; u < 8 && c + u < p.N; ++u) {
                    const bool hi = c + u >= half;
                    const int col = hi ? c + u - half : c + u;
                    float d1[8], z[8], z1[8], y;
                    load8(p.d_type, p.d, row * p.ld_d, col, col + 1, d1);
                    load8<kBF16>(p.z, row * p.ld_z, col, col + 1, z);
                    load8<kBF16>(p.z, row * p.ld_z + half, col, col + 1, z1);
                    const float slope = activate_grad(p.act, z[0], y);
                    const float x = d1[0] * (hi ? y : slope * z1[0]);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        dz[v] = v == u ? x : dz[v];
                }
            }
        }
        if (p.q) {
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                m = max(m, __float_as_uint(dz[u]) & 0x7FFFFFFFu);
            m = max(m, (uint32_t)__shfl_xor((int)m, 1));
            m = max(m, (uint32_t)__shfl_xor((int)m, 2));
            const MxScale s = mx_scale<F>(m);
            if (row < end && c < p.ld_q) {
                *reinterpret_cast<u32x2*>(p.q + row * p.ld_q + c) =
                    u32x2{mx_codes<F>(s, dz[0], dz[1], dz[2], dz[3]), mx_codes<F>(s, dz[4], dz[5], dz[6], dz[7])};
                if ((lane & 3) == 0)
                    p.s[row * (p.ld_q >> 5) + (c >> 5)] = s.byte;
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            t[(8 * cl + u) * kGradLd + r] = dz[u];
    }
    if (!p.qt && !p.part)
        return;
    __syncthreads();
    const int col = tid >> 2, b = tid & 3;      // column, block of 32 tokens
    const float* v = t + col * kGradLd + 32 * b;
    float x[32], sum = 0.f;
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 32; ++u) {
        x[u] = v[u];
        sum += x[u];
        m = max(m, __float_as_uint(x[u]) & 0x7FFFFFFFu);
    }
    if (p.part) {
        sum += __shfl_xor(sum, 1);
        sum += __shfl_xor(sum, 2);
        if (b == 0 && n0 + col < p.N)
            p.part[(int64_t)chunk * p.N + n0 + col] = sum;
    }
    if (p.qt && n0 + col < p.N) {
        const MxScale s = mx_scale<F>(m);
        u32x4 code[2];
#pragma unroll
        for (int w = 0; w < 8; ++w)
            code[w >> 2][w & 3] = mx_codes<F>(s, x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3]);
        const int64_t at = (n0 + col) * p.ld_qt + (int64_t)chunk * kGradRows + 32 * b;
        *reinterpret_cast<u32x4*>(p.qt + at) = code[0];
        *reinterpret_cast<u32x4*>(p.qt + at + 16) = code[1];
        p.st[at >> 5] = s.byte;
    }
}

// d_bias[e][n]: the column sums of the expert's tiles, in order.
__global__ void __launch_bounds__(256) grad_bias_kernel(GradArgs p)
{
    const int n = blockIdx.x * 256 + threadIdx.x;
    const int e = blockIdx.y;
    if (n >= p.N)
        return;
    int lo = 0, hi = p.chunks;
    if (p.k_offsets) {
        lo = p.k_offsets[e] / kGradRows;
        hi = p.k_offsets[e + 1] / kGradRows;
        lo = lo < 0 ? 0 : lo;
        hi = hi < p.chunks ? hi : p.chunks;
    }
    float sum = 0.f;
#pragma unroll 8
    for (int k = lo; k < hi; ++k)
        sum += p.part[(int64_t)k * p.N + n];
    p.d_bias[(int64_t)e * p.N + n] = sum;
}

hipError_t launch_grad(const GradArgs& a, hipStream_t stream)
{
    // columns up to the row codes' padded width (their padding is written too)
    const int64_t width = a.q ? a.ld_q : a.N;
    const dim3 grid((unsigned)((width + kGradCols - 1) / kGradCols), (unsigned)a.chunks);
    if (a.chunks > 0) {
        if (a.fmt == kE5M2)
            hipLaunchKernelGGL(grad_kernel<kE5M2>, grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL(grad_kernel<kE4M3>, grid, dim3(256), 0, stream, a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.d_bias)
        return e;
    hipLaunchKernelGGL(grad_bias_kernel, dim3((unsigned)((a.N + 255) / 256), (unsigned)(a.groups ? a.groups : 1)),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxg
