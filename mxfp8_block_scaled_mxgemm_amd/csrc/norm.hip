// Norms before and after a block, fused with its gate and residual scale.
#include "block.h"
#include "element.h"
#include "wave.h"

namespace mxg {

// ------------------------------------------------------------------- rows --

// A row's elements as a worker of NT threads holds them: eight per thread,
// thread t from column 8 t on, as loaded.  Elements past the row are zero.
// WHOLE: rows of whole eights, whose loads go out without a branch (threads
// past the row read its last eight and put them aside).
template <int TYPE, bool WHOLE>
struct RawRow {
    static constexpr int kWords = TYPE == kFP32 ? 8 : 4;
    typedef typename Element<TYPE>::T T;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const void* base, int64_t at, int cols, int t)
    {
        const T* p = static_cast<const T*>(base) + at;
        if constexpr (WHOLE) {
            const bool live = 8 * t < cols;
            __builtin_memcpy(w, p + (live ? 8 * t : cols - 8), sizeof(w));
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = live ? w[i] : 0;
        } else if (8 * t + 8 <= cols) {
            __builtin_memcpy(w, p + 8 * t, sizeof(w));
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (8 * t + u < cols) {
                    if constexpr (TYPE == kFP32)
                        w[u] = __float_as_uint(p[8 * t + u]);
                    else
                        w[u / 2] |= (uint32_t)p[8 * t + u] << (16 * (u & 1));
                }
        }
    }
    __device__ __forceinline__ void store(void* base, int64_t at, int cols, int t) const
    {
        T* p = static_cast<T*>(base) + at + 8 * t;
        if (8 * t + 8 <= cols) {
            __builtin_memcpy(p, w, sizeof(w));
        } else if constexpr (!WHOLE) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (8 * t + u < cols) {
                    if constexpr (TYPE == kFP32)
                        p[u] = __uint_as_float(w[u]);
                    else
                        p[u] = (uint16_t)(w[u / 2] >> (16 * (u & 1)));
                }
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            w[i] = 0;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if constexpr (TYPE == kFP32)
                f[u] = __uint_as_float(w[u]);
            else if constexpr (TYPE == kBF16)
                f[u] = __uint_as_float(u & 1 ? w[u / 2] & 0xFFFF0000u : w[u / 2] << 16);
            else
                f[u] = Element<kFP16>::get((uint16_t)(w[u / 2] >> (16 * (u & 1))));
        }
    }
    // rounds to nearest even
    __device__ __forceinline__ void put(const float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (TYPE == kFP32)
                w[i] = __float_as_uint(f[i]);
            else if constexpr (TYPE == kBF16)
                w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
            else
                w[i] = Element<kFP16>::put(f[2 * i]) | (uint32_t)Element<kFP16>::put(f[2 * i + 1]) << 16;
        }
    }
};

// Weights or a gate row, of any element type, as FP32.
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
// rounded r (what the next block and the gradient have).  A worker takes a run
// of rows; the next row's loads go out before this row's sums, which are two
// trips over lanes and LDS, and a gate row is loaded where it begins.  Bound by
// memory where there are many rows: 8192 x 4096 bfloat16 with everything, 269 MB
// in 55 us (4.9 TB/s); by one row's trips where there are few (4 x 7168: 4.8 us).
template <int TYPE, int NT, bool WHOLE>
__global__ void __launch_bounds__(Worker<NT>::kThreads) norm_kernel(NormArgs p)
{
    __shared__ float lds[Worker<NT>::kLds];
    const int t = threadIdx.x % NT;
    const int64_t workers = (int64_t)gridDim.x * Worker<NT>::kPerGroup;
    const int64_t worker = (int64_t)blockIdx.x * Worker<NT>::kPerGroup + (NT == 64 ? threadIdx.x / 64 : 0);
    const int64_t share = p.rows / workers, more = p.rows % workers;
    int64_t row = worker * share + (worker < more ? worker : more);
    const int64_t end = row + share + (worker < more ? 1 : 0);
    if (row >= end)
        return;
    const float inv_n = 1.f / (float)p.cols;
    int turn = 0;
    float post[8], pre[8], gate[8];
    if (p.post)
        load_row(p.post_type, p.post, 0, p.cols, t, post);
    if (p.pre)
        load_row(p.pre_type, p.pre, 0, p.cols, t, pre);
    int64_t g = 0, left = 0;            // the gate row, and the rows before the next one's
    if (p.gate) {
        g = row / p.per_gate - 1;
        left = 0;
    }
    bool first = true;
    RawRow<TYPE, WHOLE> nx, nres;
    nx.load(p.x, row * p.ld_x, p.cols, t);
    nres.zero();
    if (p.residual)
        nres.load(p.residual, row * p.ld_res, p.cols, t);
    for (; row < end; ++row) {
        const RawRow<TYPE, WHOLE> x = nx, res = nres;
        if (p.gate && left-- == 0) {
            ++g;
            left = (first ? p.per_gate - row % p.per_gate : p.per_gate) - 1;
            first = false;
            load_row(p.gate_type, p.gate, g * p.ld_gate, p.cols, t, gate);
        }
        if (row + 1 < end) {
            nx.load(p.x, (row + 1) * p.ld_x, p.cols, t);
            if (p.residual)
                nres.load(p.residual, (row + 1) * p.ld_res, p.cols, t);
        }
        float v[8], sum[8];
        x.get(v);
        if (p.post) {
            const float rstd = centre<NT>(v, p, inv_n, lds, turn, t);
            times(v, rstd, post);
        }
        if (p.gate)
            times(v, 1.f, gate);
        res.get(sum);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum[i] += p.scale * v[i];
        RawRow<TYPE, WHOLE> out;
        out.put(sum);
        out.store(p.r, row * p.ld_r, p.cols, t);
        if (p.pre) {
            out.get(v);
            const float rstd = centre<NT>(v, p, inv_n, lds, turn, t);
            times(v, rstd, pre);
            out.put(v);
            out.store(p.y, row * p.ld_y, p.cols, t);
        }
    }
}

// Partial or whole sums of one gate row's gradient.
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
// norm_sums_kernel adds in order.  8192 x 4096 bfloat16 with everything and 8 gate
// rows: 430 MB, 25 of them partial rows, in 108 us (4.0 TB/s), and 7 for the sums.
// 128 registers hold no row ahead at this width, so that a row's loads and its
// arithmetic follow each other within a wave; its four trips over lanes and LDS
// merged into two took as long.
template <int TYPE, bool WHOLE>
struct NormInputs {
    RawRow<TYPE, WHOLE> dy, dr, x, r;
    __device__ __forceinline__ void load(const NormArgs& p, int64_t row, int t)
    {
        load_first(p, row, t);
        load_second(p, row, t);
    }
    __device__ __forceinline__ void load_first(const NormArgs& p, int64_t row, int t)
    {
        if (p.d_y) {
            dy.load(p.d_y, row * p.ld_dy, p.cols, t);
            r.load(p.r, row * p.ld_r, p.cols, t);
        }
    }
    __device__ __forceinline__ void load_second(const NormArgs& p, int64_t row, int t)
    {
        if (p.d_r)
            dr.load(p.d_r, row * p.ld_dr, p.cols, t);
        if (p.post || p.gate)
            x.load(p.x, row * p.ld_x, p.cols, t);
    }
};

template <int TYPE, int NT, bool WHOLE>
__global__ void __launch_bounds__(Worker<NT>::kThreads) __attribute__((amdgpu_waves_per_eu(NT == 64 ? 3 : 4)))
norm_backward_kernel(NormArgs p)
{
    // Sixteen waves per compute unit are 128 registers each.  Where they allow
    // it, the next row's loads go out a row ahead; where they do not even hold
    // a row of everything, half of it is loaded between the two norms.
    constexpr bool kAhead = TYPE != kFP32 && (NT == 64 || (TYPE == kBF16 && NT < 512));
    constexpr bool kHalves = TYPE == kFP32;
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
    float post[8], pre[8], gate[8], s_post[8], s_pre[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        s_post[i] = s_pre[i] = 0.f;
    if (p.post)
        load_row(p.post_type, p.post, 0, p.cols, t, post);
    if (p.pre)
        load_row(p.pre_type, p.pre, 0, p.cols, t, pre);
    for (int64_t u = u0; u < u1; ++u) {
        const int64_t g = u / p.units, first = (u - g * p.units) * p.per_unit;
        int64_t row = g * p.per_gate + first;
        const int64_t left = p.per_gate - first, end = row + (left < p.per_unit ? left : p.per_unit);
        float s_gate[8];
        NormInputs<TYPE, WHOLE> next;
        if constexpr (kAhead)
            next.load(p, row, t);
        if (p.gate) {
            load_row(p.gate_type, p.gate, g * p.ld_gate, p.cols, t, gate);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s_gate[i] = 0.f;
        }
        for (; row < end; ++row) {
            if constexpr (kHalves)
                next.load_first(p, row, t);
            else if constexpr (!kAhead)
                next.load(p, row, t);
            NormInputs<TYPE, WHOLE> in = next;
            if (kAhead && row + 1 < end)
                next.load(p, row + 1, t);
            float d[8], v[8];
            if (p.d_y) {
                in.dy.get(d);
                in.r.get(v);
                const float rstd = centre<NT>(v, p, inv_n, lds, turn, t);
                float s[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] *= rstd;
                    s_pre[i] += d[i] * v[i];
                    d[i] *= pre[i];
                    s[0] += d[i] * v[i];
                    s[1] += d[i];
                }
                row_sums<NT>(s, lds, turn, t);
                const float dot = s[0] * inv_n, mean = p.layer ? s[1] * inv_n : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = rstd * (d[i] - v[i] * dot - mean);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = 0.f;
            }
            if constexpr (kHalves)
                in.load_second(p, row, t);
            if (p.d_r) {
                in.dr.get(v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] += v[i];
            }
            RawRow<TYPE, WHOLE> out;
            if (p.d_residual) {
                out.put(d);
                out.store(p.d_residual, row * p.ld_dres, p.cols, t);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] *= p.scale;
            float rstd = 1.f;
            if (p.post || p.gate)
                in.x.get(v);
            if (p.post) {
                rstd = centre<NT>(v, p, inv_n, lds, turn, t);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] *= rstd;
            }
            if (p.gate) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s_gate[i] += d[i] * (p.post ? v[i] * post[i] : v[i]);
                    d[i] *= gate[i];
                }
            }
            if (p.post) {
                float s[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s_post[i] += d[i] * v[i];
                    d[i] *= post[i];
                    s[0] += d[i] * v[i];
                    s[1] += d[i];
                }
                row_sums<NT>(s, lds, turn, t);
                const float dot = s[0] * inv_n, mean = p.layer ? s[1] * inv_n : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = rstd * (d[i] - v[i] * dot - mean);
            }
            out.put(d);
            out.store(p.d_x, row * p.ld_dx, p.cols, t);
        }
        if (p.gate) {
            if (p.units == 1)
                store_gate(p, g, s_gate, t);
            else        // then a worker has one unit
                store_part(p, 2, worker, s_gate, t);
        }
    }
    if (p.post)
        store_part(p, 0, worker, s_post, t);
    if (p.pre)
        store_part(p, 1, worker, s_pre, t);
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

int norm_threads(int cols)
{
    return cols <= 512 ? 64 : cols <= 1024 ? 128 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : 1024;
}

template <int TYPE, int NT, bool WHOLE>
static void norm_launch(const NormArgs& a, bool backward, int cus, hipStream_t stream)
{
    typedef Worker<NT> W;
    if (backward) {
        hipLaunchKernelGGL((norm_backward_kernel<TYPE, NT, WHOLE>),
                           dim3((unsigned)((a.workers + W::kPerGroup - 1) / W::kPerGroup)), dim3(W::kThreads), 0, stream, a);
        return;
    }
    int64_t groups = (a.rows + W::kPerGroup - 1) / W::kPerGroup;
    // as many as a compute unit has waves for; their registers let five to seven
    // eighths of them be resident (three work-groups of 512 threads, one of 1024),
    // and the others follow
    const int64_t most = (int64_t)cus * (2048 / W::kThreads);
    groups = groups < most ? groups : most;
    hipLaunchKernelGGL((norm_kernel<TYPE, NT, WHOLE>), dim3((unsigned)groups), dim3(W::kThreads), 0, stream, a);
}

template <int TYPE, bool WHOLE>
static void norm_launch(const NormArgs& a, bool backward, int cus, hipStream_t stream)
{
    switch (norm_threads(a.cols)) {
    case 64: return norm_launch<TYPE, 64, WHOLE>(a, backward, cus, stream);
    case 128: return norm_launch<TYPE, 128, WHOLE>(a, backward, cus, stream);
    case 256: return norm_launch<TYPE, 256, WHOLE>(a, backward, cus, stream);
    case 512: return norm_launch<TYPE, 512, WHOLE>(a, backward, cus, stream);
    default: return norm_launch<TYPE, 1024, WHOLE>(a, backward, cus, stream);
    }
}

static hipError_t norm_any(const NormArgs& a, int type, bool backward, int cus, hipStream_t stream)
{
    if (a.cols % 8 == 0) {
        if (type == kBF16)
            norm_launch<kBF16, true>(a, backward, cus, stream);
        else if (type == kFP16)
            norm_launch<kFP16, true>(a, backward, cus, stream);
        else
            norm_launch<kFP32, true>(a, backward, cus, stream);
    } else {
        if (type == kBF16)
            norm_launch<kBF16, false>(a, backward, cus, stream);
        else if (type == kFP16)
            norm_launch<kFP16, false>(a, backward, cus, stream);
        else
            norm_launch<kFP32, false>(a, backward, cus, stream);
    }
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
