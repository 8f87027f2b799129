// Norms before and after a block, fused with its gate and residual scale.
#include "block.h"
#include "element.h"
#include "wave.h"

namespace mxg {

// ------------------------------------------------------------------- rows --

// A row's elements as a worker of NT threads holds them: eight per thread,
// thread t from column 8 t on.  Elements past the row are zero, and neither
// read nor written.
template <int TYPE, int NT>
struct RawRow {
    Pack<TYPE, 8> v;
    __device__ __forceinline__ void load(const void* base, int64_t at, int cols, int t)
    {
        const typename Element<TYPE>::T* p = static_cast<const typename Element<TYPE>::T*>(base) + at + 8 * t;
        if (8 * t + 8 <= cols) {
            v.load(p);
        } else {
            v.zero();
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (8 * t + u < cols)
                    v.v[u] = p[u];
        }
    }
    __device__ __forceinline__ void store(void* base, int64_t at, int cols, int t) const
    {
        typename Element<TYPE>::T* p = static_cast<typename Element<TYPE>::T*>(base) + at + 8 * t;
        if (8 * t + 8 <= cols) {
            v.store(p);
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (8 * t + u < cols)
                    p[u] = v.v[u];
        }
    }
    __device__ __forceinline__ void zero() { v.zero(); }
    __device__ __forceinline__ float get(int i) const { return v.get(i); }
    __device__ __forceinline__ void put(int i, float f) { v.put(i, f); }
};

// Weights or a gate row, of any element type, as FP32.
template <int NT>
__device__ __forceinline__ void load_row(int type, const void* base, int64_t at, int cols, int t, float (&f)[8])
{
    load8(type, base, at, 8 * t, cols, f);
}

// Sums over a worker's threads, the same in all of them: over lanes, then
// over waves in order.  `lds`: two sets of N values for each wave, used in
// turns, so that one barrier a sum is enough.
template <int NT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* lds, int& turn, int t)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = wave_sum(v[i]);
    if constexpr (NT > 64) {
        constexpr int W = NT / 64;
        float* mine = lds + turn * (4 * W);
        turn ^= 1;
        if ((t & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                mine[i * W + (t >> 6)] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = mine[i * W];
#pragma unroll
            for (int w = 1; w < W; ++w)
                v[i] += mine[i * W + w];
        }
    }
}

// v's mean taken off (layer; elements past the row stay zero) and 1 / its
// root mean square, all sums in FP32 over the values themselves: the variance
// is a sum of squares about the mean, which does not cancel.
template <int NT>
__device__ __forceinline__ float centre(float (&v)[8], const NormArgs& p, float inv_n, float* lds, int& turn, int t)
{
    if (p.layer) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[0] += v[i];
        row_sums<NT>(s, lds, turn, t);
        const float mean = s[0] * inv_n;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 8 * t + i < p.cols ? v[i] - mean : 0.f;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        s[0] += v[i] * v[i];
    row_sums<NT>(s, lds, turn, t);
    return 1.f / sqrtf(s[0] * inv_n + p.eps);
}

// v *= f w
__device__ __forceinline__ void times(float (&v)[8], float f, const float (&w)[8])
{
#pragma unroll
    for (int u = 0; u < 8; ++u)
        v[u] = v[u] * f * w[u];
}

template <int NT>
struct Worker {
    static constexpr int kPerGroup = NT == 64 ? 4 : 1;      // workers of a work-group
    static constexpr int kThreads = NT * kPerGroup;
    static constexpr int kLds = NT > 64 ? 8 * (NT / 64) : 1;
};

// r = residual + scale gate post(x), rounded to its type; y = pre(r), of the
// rounded r (what the next block and the gradient have).  A worker takes rows
// in turn; the next row's loads go out before this row's sums, which are two
// trips over lanes and LDS.
template <int TYPE, int NT>
__global__ void __launch_bounds__(Worker<NT>::kThreads) norm_kernel(NormArgs p)
{
    __shared__ float lds[Worker<NT>::kLds];
    const int t = threadIdx.x % NT;
    const int64_t workers = (int64_t)gridDim.x * Worker<NT>::kPerGroup;
    int64_t row = (int64_t)blockIdx.x * Worker<NT>::kPerGroup + (NT == 64 ? threadIdx.x / 64 : 0);
    if (row >= p.rows)
        return;
    const float inv_n = 1.f / (float)p.cols;
    int turn = 0;
    float post[8], pre[8], gate[8];
    if (p.post)
        load_row<NT>(p.post_type, p.post, 0, p.cols, t, post);
    if (p.pre)
        load_row<NT>(p.pre_type, p.pre, 0, p.cols, t, pre);
    RawRow<TYPE, NT> nx, nres;
    nx.load(p.x, row * p.ld_x, p.cols, t);
    nres.zero();
    if (p.residual)
        nres.load(p.residual, row * p.ld_res, p.cols, t);
    for (; row < p.rows; row += workers) {
        const RawRow<TYPE, NT> x = nx, res = nres;
        if (p.gate)
            load_row<NT>(p.gate_type, p.gate, row / p.per_gate * p.ld_gate, p.cols, t, gate);
        const int64_t next = row + workers;
        if (next < p.rows) {
            nx.load(p.x, next * p.ld_x, p.cols, t);
            if (p.residual)
                nres.load(p.residual, next * p.ld_res, p.cols, t);
        }
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = x.get(i);
        if (p.post) {
            const float rstd = centre<NT>(v, p, inv_n, lds, turn, t);
            times(v, rstd, post);
        }
        if (p.gate)
            times(v, 1.f, gate);
        RawRow<TYPE, NT> out;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            out.put(i, res.get(i) + p.scale * v[i]);
            v[i] = out.get(i);
        }
        out.store(p.r, row * p.ld_r, p.cols, t);
        if (p.pre) {
            const float rstd = centre<NT>(v, p, inv_n, lds, turn, t);
            times(v, rstd, pre);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                out.put(i, v[i]);
            out.store(p.y, row * p.ld_y, p.cols, t);
        }
    }
}

// Partial or whole sums of one gate row's gradient.
template <int NT>
__device__ __forceinline__ void store_gate(const NormArgs& p, int64_t g, const float (&s)[8], int t)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = 8 * t + i;
        if (c >= p.cols)
            continue;
        const int64_t at = g * p.cols + c;
        if (p.gate_type == kFP32)
            static_cast<float*>(p.d_gate)[at] = s[i];
        else if (p.gate_type == kFP16)
            static_cast<uint16_t*>(p.d_gate)[at] = Element<kFP16>::put(s[i]);
        else
            static_cast<uint16_t*>(p.d_gate)[at] = Element<kBF16>::put(s[i]);
    }
}

template <int NT>
__device__ __forceinline__ void store_part(const NormArgs& p, int which, int64_t worker, const float (&s)[8], int t)
{
    float* out = p.part + ((int64_t)which * p.workers + worker) * p.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = 8 * t + i;
        if (c < p.cols)
            out[c] = s[i];
    }
}

// Gradient.  With h = (r - mean) rstd of the pre norm and n = post(x):
//   d_res = d_r + rstd (e - h <e h> [- <e>]), e = d_y pre, <> the row's mean
//   d_pre += d_y h;  u = scale d_res;  d_gate += u n;  m = u gate
//   d_post += m xhat;  d_x = rstd_x (f - xhat <f xhat> [- <f>]), f = m post
// (bracketed terms: layer).  Everything is read once and both statistics are
// formed again from the rows; a worker takes consecutive units of rows, keeps
// its columns' sums in registers and leaves them as one partial row, which
// norm_sums_kernel adds in order.
template <int TYPE, int NT>
__global__ void __launch_bounds__(Worker<NT>::kThreads) norm_backward_kernel(NormArgs p)
{
    __shared__ float lds[Worker<NT>::kLds];
    const int t = threadIdx.x % NT;
    const int64_t worker = (int64_t)blockIdx.x * Worker<NT>::kPerGroup + (NT == 64 ? threadIdx.x / 64 : 0);
    if (worker >= p.workers)
        return;
    const float inv_n = 1.f / (float)p.cols;
    const int64_t all = p.gates * p.units;
    const int64_t share = all / p.workers, more = all % p.workers;
    const int64_t u0 = worker * share + (worker < more ? worker : more), u1 = u0 + share + (worker < more ? 1 : 0);
    int turn = 0;
    float post[8], pre[8], gate[8];
    float s_post[8], s_pre[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        s_post[i] = s_pre[i] = 0.f;
    if (p.post)
        load_row<NT>(p.post_type, p.post, 0, p.cols, t, post);
    if (p.pre)
        load_row<NT>(p.pre_type, p.pre, 0, p.cols, t, pre);
    for (int64_t u = u0; u < u1; ++u) {
        const int64_t g = u / p.units, first = (u % p.units) * p.per_unit;
        int64_t row = g * p.per_gate + first;
        const int64_t left = p.per_gate - first, end = row + (left < p.per_unit ? left : p.per_unit);
        float s_gate[8];
        if (p.gate) {
            load_row<NT>(p.gate_type, p.gate, g * p.ld_gate, p.cols, t, gate);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s_gate[i] = 0.f;
        }
        for (; row < end; ++row) {
            RawRow<TYPE, NT> dr, raw;
            float d[8], v[8];
            dr.zero();
            if (p.d_r)
                dr.load(p.d_r, row * p.ld_dr, p.cols, t);
            RawRow<TYPE, NT> xraw;
            if (p.post || p.gate)
                xraw.load(p.x, row * p.ld_x, p.cols, t);
            if (p.pre && p.d_y) {
                raw.load(p.d_y, row * p.ld_dy, p.cols, t);
                RawRow<TYPE, NT> r;
                r.load(p.r, row * p.ld_r, p.cols, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = r.get(i);
                    d[i] = raw.get(i);
                }
                const float rstd = centre<NT>(v, p, inv_n, lds, turn, t);
                float s[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] *= rstd;
                    s_pre[i] += d[i] * v[i];
                }
                times(d, 1.f, pre);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[0] += d[i] * v[i];
                    s[1] += d[i];
                }
                row_sums<NT>(s, lds, turn, t);
                const float dot = s[0] * inv_n, mean = p.layer ? s[1] * inv_n : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = dr.get(i) + rstd * (d[i] - v[i] * dot - mean);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = dr.get(i);
            }
            RawRow<TYPE, NT> out;
            if (p.d_residual) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    out.put(i, d[i]);
                out.store(p.d_residual, row * p.ld_dres, p.cols, t);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] *= p.scale;
            float rstd = 1.f;
            if (p.post || p.gate) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = xraw.get(i);
            }
            if (p.post) {
                rstd = centre<NT>(v, p, inv_n, lds, turn, t);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] *= rstd;
            }
            if (p.gate) {
                float n[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    n[i] = d[i] * v[i];
                if (p.post)
                    times(n, 1.f, post);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s_gate[i] += n[i];
                times(d, 1.f, gate);
            }
            if (p.post) {
                float s[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s_post[i] += d[i] * v[i];
                times(d, 1.f, post);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[0] += d[i] * v[i];
                    s[1] += d[i];
                }
                row_sums<NT>(s, lds, turn, t);
                const float dot = s[0] * inv_n, mean = p.layer ? s[1] * inv_n : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = rstd * (d[i] - v[i] * dot - mean);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                out.put(i, d[i]);
            out.store(p.d_x, row * p.ld_dx, p.cols, t);
        }
        if (p.gate) {
            if (p.units == 1)
                store_gate<NT>(p, g, s_gate, t);
            else        // then a worker has one unit
                store_part<NT>(p, 2, worker, s_gate, t);
        }
    }
    if (p.post)
        store_part<NT>(p, 0, worker, s_post, t);
    if (p.pre)
        store_part<NT>(p, 1, worker, s_pre, t);
}

// Column sums of the workers' partial rows: 64 columns a work-group, its
// sixteen waves take every sixteenth row and are added in order.  blockIdx.y:
// post, pre, then (units > 1) the gate rows.
__global__ void __launch_bounds__(1024) norm_sums_kernel(NormArgs p)
{
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane, job = blockIdx.y;
    float* out = job == 0 ? p.d_post : job == 1 ? p.d_pre : nullptr;
    if (job < 2 && !out)
        return;
    const int64_t first = job < 2 ? 0 : (job - 2) * p.units, n = job < 2 ? p.workers : p.units;
    const float* part = p.part + ((int64_t)(job < 2 ? job : 2) * p.workers + first) * p.cols;
    float sum = 0.f;
    if (c < p.cols) {
#pragma unroll 8
        for (int64_t w = wave; w < n; w += 16)
            sum += part[w * p.cols + c];
    }
    lds[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || c >= p.cols)
        return;
    sum = lds[0][lane];
#pragma unroll
    for (int w = 1; w < 16; ++w)
        sum += lds[w][lane];
    if (job < 2) {
        out[c] = sum;
        return;
    }
    const int64_t at = (int64_t)(job - 2) * p.cols + c;
    if (p.gate_type == kFP32)
        static_cast<float*>(p.d_gate)[at] = sum;
    else if (p.gate_type == kFP16)
        static_cast<uint16_t*>(p.d_gate)[at] = Element<kFP16>::put(sum);
    else
        static_cast<uint16_t*>(p.d_gate)[at] = Element<kBF16>::put(sum);
}

// ----------------------------------------------------------------- launch --

NormShape norm_shape(int cols)
{
    if (cols <= 512)
        return {64, 256};
    const int threads = cols <= 1024 ? 128 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : 1024;
    return {threads, threads};
}

template <int TYPE, int NT>
static void norm_launch(const NormArgs& a, bool backward, int cus, hipStream_t stream)
{
    typedef Worker<NT> W;
    if (backward) {
        hipLaunchKernelGGL((norm_backward_kernel<TYPE, NT>),
                           dim3((unsigned)((a.workers + W::kPerGroup - 1) / W::kPerGroup)), dim3(W::kThreads), 0, stream, a);
        return;
    }
    int64_t groups = (a.rows + W::kPerGroup - 1) / W::kPerGroup;
    const int64_t most = (int64_t)cus * (2048 / W::kThreads);       // as many as are resident
    groups = groups < most ? groups : most;
    hipLaunchKernelGGL((norm_kernel<TYPE, NT>), dim3((unsigned)groups), dim3(W::kThreads), 0, stream, a);
}

template <int TYPE>
static void norm_launch(const NormArgs& a, bool backward, int cus, hipStream_t stream)
{
    if (a.cols <= 512)
        norm_launch<TYPE, 64>(a, backward, cus, stream);
    else if (a.cols <= 1024)
        norm_launch<TYPE, 128>(a, backward, cus, stream);
    else if (a.cols <= 2048)
        norm_launch<TYPE, 256>(a, backward, cus, stream);
    else if (a.cols <= 4096)
        norm_launch<TYPE, 512>(a, backward, cus, stream);
    else
        norm_launch<TYPE, 1024>(a, backward, cus, stream);
}

static hipError_t norm_any(const NormArgs& a, int type, bool backward, int cus, hipStream_t stream)
{
    if (type == kBF16)
        norm_launch<kBF16>(a, backward, cus, stream);
    else if (type == kFP16)
        norm_launch<kFP16>(a, backward, cus, stream);
    else
        norm_launch<kFP32>(a, backward, cus, stream);
    return hipGetLastError();
}

hipError_t launch_norm(const NormArgs& a, int type, int cus, hipStream_t stream)
{
    return norm_any(a, type, false, cus, stream);
}

hipError_t launch_norm_backward(const NormArgs& a, int type, hipStream_t stream)
{
    if (a.workers > 0) {
        const hipError_t e = norm_any(a, type, true, 0, stream);
        if (e != hipSuccess)
            return e;
    }
    const unsigned jobs = 2 + (a.gate && a.units != 1 ? (unsigned)a.gates : 0);
    if (!a.post && !a.pre && jobs == 2)
        return hipSuccess;
    hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)((a.cols + 63) / 64), jobs), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxg
