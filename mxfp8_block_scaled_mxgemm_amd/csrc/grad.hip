// Gradient of the product's epilogue, held in MXFP8 both ways.
#include "activation.h"
#include "element.h"
#include "linear.h"
#include "quant.h"
#include "schedule.h"
#include "segments.h"

namespace mxg {

// Eight 16-bit elements as loaded.
struct Raw16 {
    u32x4 v;
    __device__ __forceinline__ void load(const void* base, int64_t at)
    {
        v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at);
    }
    __device__ __forceinline__ void get(int type, float (&f)[8]) const
    {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t w = v[u >> 1];
            f[u] = type == kFP16 ? Element<kFP16>::get((uint16_t)(w >> (16 * (u & 1))))
                                 : __uint_as_float(u & 1 ? w & 0xFFFF0000u : w << 16);
        }
    }
};

// A work-group takes 128 tokens x 64 columns of dz; gated with halves of whole
// blocks (FUSED), 32 columns of both halves, [d_out u act'(g), d_out act(g)],
// so that d_out and z are read and the activation is evaluated once.  A
// thread computes eight columns (FUSED: eight of each half) of a few rows;
// the loads of all its rows go out before the first is used.  Along the
// columns, four threads share a block of 32 and quantise it at once.  The
// FP32 values also go to LDS, transposed to [column][token]; there a thread
// takes one column's block of 32 tokens: its sum, its scale, its codes (32
// bytes; four threads write one column's 128 bytes).  Tokens past the expert's
// last one count as zeros, so blocks never cross experts.  d_out and z are read
// once and the two bytes per element written: 4096 x 4096 with gelu_tanh, 31
// us (103 MB, 3.3 TB/s); 8002 rows of 2 x 1024 gated with silu over 24
// experts, 33 us (92 MB, 2.8 TB/s).  Bound by instructions: two quantisations
// and the activation's slope per element.  Without VEC a row's loads wait for
// the row before: 4096 x 4096 FP32 with silu 28 us (bfloat16 24 in the same
// loop), 4096 rows of 2 x 1041 gated 40 us.
constexpr int kGradRows = 128, kGradCols = 64;

// Place of (tile column, row) in LDS: spread so that neither eight columns 8
// apart of neighbouring rows (the writes) nor eight columns by four blocks of
// 32 rows (the reads) meet in one of 32 banks.
constexpr int kGradWords = 132 * kGradCols + 64;
__device__ __forceinline__ int grad_at(int col, int row)
{
    return 132 * col + 8 * (col >> 3) + 4 * (col >> 5) + row + (row >> 5);
}

// By expert, what no segment holds is zero: the rows of dropped pairs, and the
// columns of qt past the last segment.  Chunk `chunk` past the last segment
// clears its own columns of qt (the grid's last chunk, past ld_qt, has none),
// and all such chunks share the dropped rows in turn.  A work-group clears tile
// columns [n0, n0 + 64).  Bound by the bytes cleared: 16384 rows of 2 x 2048,
// silu, over 32 experts, 2% dropped 103 us in all (100 without), half dropped
// 51 (38); 1024 rows of 2 x 1024 over 1024 experts 127 (100).
__device__ __forceinline__ void grad_rest(const GradArgs& p, int chunk, int n0)
{
    const int tid = threadIdx.x;
    if (p.qt && chunk < p.chunks && n0 + (tid >> 2) < p.N) {
        const int64_t at = (n0 + (tid >> 2)) * p.ld_qt + (int64_t)chunk * kGradRows + 32 * (tid & 3);
        *reinterpret_cast<u32x4*>(p.qt + at) = u32x4{0, 0, 0, 0};
        *reinterpret_cast<u32x4*>(p.qt + at + 16) = u32x4{0, 0, 0, 0};
        p.st[at >> 5] = 0;
    }
    if (!p.q)
        return;
    int first = p.k_offsets[p.groups], live = p.offsets[p.groups];
    first = first < 0 ? 0 : (first + kGradRows - 1) / kGradRows;
    first = first < p.chunks ? first : p.chunks;
    live = live < 0 ? 0 : live;
    const int64_t stride = (int64_t)(p.chunks + 1 - first) * 64;
    for (int64_t row = live + (int64_t)(chunk - first) * 64 + (tid >> 2); row < p.rows; row += stride) {
        const int c = n0 + 16 * (tid & 3);          // ld_q is a multiple of 128
        *reinterpret_cast<u32x4*>(p.q + row * p.ld_q + c) = u32x4{0, 0, 0, 0};
        if ((tid & 1) == 0)
            p.s[row * (p.ld_q >> 5) + (c >> 5)] = 0;
    }
}

// dz of columns [c, c + 8) of one row, the general way: any width and gating.
__device__ __forceinline__ void grad_columns(const GradArgs& p, int64_t row, int c, float (&dz)[8])
{
    const int half = p.N / 2;
    // the thread's columns as [first, first + 8) of d_out: a gated piece that
    // reaches over the middle is taken a column at a time
    const bool up = p.gated && c >= half;
    if (!p.gated || up || c + 8 <= half) {
        const int width = p.gated ? half : p.N;
        const int first = up ? c - half : c;
        load8(p.d_type, p.d, row * p.ld_d, first, width, dz);
        if (p.z && (p.gated || p.act != kActNone)) {
            float z[8], z1[8], y[8];
            load8<kBF16>(p.z, row * p.ld_z, first, width, z);
            if (p.gated)
                load8<kBF16>(p.z, row * p.ld_z + half, first, width, z1);
            activate_grads(p.act, z, y);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                dz[u] *= p.gated ? (up ? y[u] : z[u] * z1[u]) : z[u];
        }
        return;
    }
#pragma unroll 1
    for (int u = 0; u < 8 && c + u < p.N; ++u) {
        const bool hi = c + u >= half;
        const int col = hi ? c + u - half : c + u;
        float d1[8], z[8], z1[8], y[8];
        load8(p.d_type, p.d, row * p.ld_d, col, col + 1, d1);
        load8<kBF16>(p.z, row * p.ld_z, col, col + 1, z);
        load8<kBF16>(p.z, row * p.ld_z + half, col, col + 1, z1);
        activate_grads(p.act, z, y);
        const float x = d1[0] * (hi ? y[0] : z[0] * z1[0]);
#pragma unroll
        for (int v = 0; v < 8; ++v)
            dz[v] = v == u ? x : dz[v];
    }
}

// Eight columns of dz along the columns, and to LDS (tile column tc, row r).
template <int F>
__device__ __forceinline__ void grad_put(const GradArgs& p, float* t, int row, int r, int end, int c, int tc,
                                         const float (&dz)[8], int lane)
{
    if (p.q) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            m = max(m, __float_as_uint(dz[u]) & 0x7FFFFFFFu);
        const MxScale s = mx_scale<F>(quad_max(m));
        if (row < end && c < p.ld_q) {
            *reinterpret_cast<u32x2*>(p.q + row * p.ld_q + c) =
                u32x2{mx_codes<F>(s, dz[0], dz[1], dz[2], dz[3]), mx_codes<F>(s, dz[4], dz[5], dz[6], dz[7])};
            if ((lane & 3) == 0)
                p.s[row * (p.ld_q >> 5) + (c >> 5)] = s.byte;
        }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
        t[grad_at(tc, r) + 132 * u] = dz[u];     // tc is a multiple of 8
}

// FUSED tiles take 64 bytes of a row of d_out: two neighbours share a line, so
// both go to one XCD (else every line is fetched into two L2s: 94 MB for 49,
// and 34 us against 31 for the 8002 rows above).
__device__ __forceinline__ int paired_tile()
{
    const int x = blockIdx.x;
    if (gridDim.x % kNumXcd != 0 || (x | (2 * kNumXcd - 1)) >= (int)gridDim.x)
        return x;
    const int i = x % (2 * kNumXcd);
    return x - i + 2 * (i % kNumXcd) + i / kNumXcd;
}

// VEC: whole eights of 16-bit d_out (and z) columns, so a row's loads are
// plain; rows past the end read the last one and count as zeros.
template <int F, bool FUSED, bool VEC>
__global__ void __launch_bounds__(256) grad_kernel(GradArgs p)
{
    __shared__ float t[kGradWords];
    const int tid = threadIdx.x, lane = tid & 63;
    const int chunk = blockIdx.y;
    int row0, end;
    if (!segment_rows(p, chunk, row0, end)) {
        grad_rest(p, chunk, blockIdx.x * kGradCols);
        return;
    }
    const int half = p.N / 2;
    const int n0 = (FUSED ? paired_tile() : blockIdx.x) * kGradCols;    // FUSED: columns n0 / 2 of both halves
    constexpr int kLanes = FUSED ? 4 : 8;       // threads across the columns
    constexpr int kPasses = kGradRows * kLanes / 256;
    const int cl = tid % kLanes, rl = tid / kLanes;
    const int c = (FUSED ? n0 / 2 : n0) + 8 * cl;
    if constexpr (VEC) {
        const int width = FUSED ? half : p.N;
        const int cc = c < width ? c : width - 8;
        const bool act = p.z && p.act != kActNone;
        Raw16 d[kPasses], z[kPasses], z1[FUSED ? kPasses : 1];
        // (rows of an empty tail read row 0 at worst: there is one)
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            int64_t row = row0 + rl + k * (256 / kLanes);
            row = row < end ? row : end > 0 ? end - 1 : 0;
            d[k].load(p.d, row * p.ld_d + cc);
            if (FUSED || act)
                z[k].load(p.z, row * p.ld_z + cc);
            if constexpr (FUSED)
                z1[k].load(p.z, row * p.ld_z + half + cc);
        }
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            const int r = rl + k * (256 / kLanes), row = row0 + r;
            const bool ok = row < end && c < width;
            float x[8], x1[8], slope[8], y[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                x[u] = 0.f;
            if (ok)
                d[k].get(p.d_type, x);
            if (FUSED || act) {
                z[k].get(kBF16, slope);
                activate_grads(p.act, slope, y);
            }
            if constexpr (FUSED) {
                z1[k].get(kBF16, x1);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float dg = x[u] * slope[u] * x1[u];
                    x1[u] = ok ? x[u] * y[u] : 0.f;
                    x[u] = ok ? dg : 0.f;
                }
            } else if (act) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    x[u] = ok ? x[u] * slope[u] : 0.f;
            }
            grad_put<F>(p, t, row, r, end, c, 8 * cl, x, lane);
            if constexpr (FUSED)
                grad_put<F>(p, t, row, r, end, half + c, 32 + 8 * cl, x1, lane);
        }
    } else {
#pragma unroll 1
        for (int r = rl; r < kGradRows; r += 256 / kLanes) {
            const int row = row0 + r;
            float dz[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                dz[u] = 0.f;
            if (row < end)
                grad_columns(p, row, c, dz);
            grad_put<F>(p, t, row, r, end, c, 8 * cl, dz, lane);
        }
    }
    if (!p.qt && !p.part)
        return;
    __syncthreads();
    const int col = tid >> 2, b = tid & 3;      // column, block of 32 tokens
    const int n = FUSED ? n0 / 2 + (col & 31) + (col >= 32 ? half : 0) : n0 + col;
    const bool there = FUSED ? n0 / 2 + (col & 31) < half : n < p.N;
    const float* v = t + grad_at(col, 32 * b);
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
        if (b == 0 && there)
            p.part[(int64_t)chunk * p.N + n] = sum;
    }
    if (p.qt && there) {
        const MxScale s = mx_scale<F>(m);
        u32x4 code[2];
#pragma unroll
        for (int w = 0; w < 8; ++w)
            code[w >> 2][w & 3] = mx_codes<F>(s, x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3]);
        const int64_t at = n * p.ld_qt + (int64_t)chunk * kGradRows + 32 * b;
        *reinterpret_cast<u32x4*>(p.qt + at) = code[0];
        *reinterpret_cast<u32x4*>(p.qt + at + 16) = code[1];
        p.st[at >> 5] = s.byte;
    }
}

// Zero codes of the row codes' padding, columns [N, ld_q) (whole blocks past
// the last column's; FUSED tiles do not reach them).
__global__ void __launch_bounds__(256) grad_pad_kernel(GradArgs p)
{
    const int first = (p.N + 31) / 32 * 32, width = (int)p.ld_q - first;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / width;
    const int c = first + (int)(i % width);
    if (row >= p.rows)
        return;
    p.q[row * p.ld_q + c] = 0;
    if (c % 32 == 0)
        p.s[row * (p.ld_q >> 5) + c / 32] = 0;
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

template <int F>
static void grad_launch(const GradArgs& a, hipStream_t stream)
{
    auto aligned = [](const void* p, int64_t ld) { return (ld & 7) == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    const int width = a.gated ? a.N / 2 : a.N;
    const bool vec = a.rows > 0 && a.d_type != kFP32 && (width & 7) == 0 && aligned(a.d, a.ld_d) &&
                     (!a.z || aligned(a.z, a.ld_z));
    const unsigned chunks = (unsigned)a.chunks + (a.k_offsets ? 1 : 0);     // one past the end: grad_rest
    if (vec && a.gated && (width & 31) == 0) {
        const dim3 grid((unsigned)(width / 32), chunks);
        hipLaunchKernelGGL((grad_kernel<F, true, true>), grid, dim3(256), 0, stream, a);
        if (a.q && a.ld_q > a.N)
            hipLaunchKernelGGL(grad_pad_kernel, dim3((unsigned)((a.rows * (a.ld_q - a.N) + 255) / 256)), dim3(256), 0,
                               stream, a);
        return;
    }
    // columns up to the row codes' padded width (their padding is written too)
    const int64_t all = a.q ? a.ld_q : a.N;
    const dim3 grid((unsigned)((all + kGradCols - 1) / kGradCols), chunks);
    if (vec && !a.gated)
        hipLaunchKernelGGL((grad_kernel<F, false, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((grad_kernel<F, false, false>), grid, dim3(256), 0, stream, a);
}

hipError_t launch_grad(const GradArgs& a, hipStream_t stream)
{
    if (a.chunks > 0 || a.k_offsets) {
        if (a.fmt == kE5M2)
            grad_launch<kE5M2>(a, stream);
        else
            grad_launch<kE4M3>(a, stream);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.d_bias)
        return e;
    hipLaunchKernelGGL(grad_bias_kernel, dim3((unsigned)((a.N + 255) / 256), (unsigned)(a.groups ? a.groups : 1)),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxg
