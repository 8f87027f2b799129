// Experts of each token and their weights, from the router's logits.
#include "block.h"
#include "element.h"
#include "wave.h"

namespace mxg {

// A wave takes one token at a time, expert 64 s + lane in slot s of a lane.
// Keys, the scores that a choice compares, are formed in 64 bits: scores of
// popular experts differ by less than an FP32 step often enough to change
// choices.  (Without bias and groups the logits themselves are compared.)  A
// key is held as the unsigned whole number of the same order; 0 is an expert
// that is never chosen (logit or key -infinity or NaN).  The next choice is a
// maximum of the upper words over the lanes, and of the lower ones only where
// several lanes have it.  16384 tokens of 256 experts, k 8: bound by these
// dependent steps, not by the 16 MB read.

__device__ __forceinline__ uint64_t ordered(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);       // -0 counts as 0
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double from_ordered(uint64_t u)
{
    return __builtin_bit_cast(double, u >> 63 ? u & 0x7FFFFFFFFFFFFFFFull : ~u);
}
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);
    return u >> 31 ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float route_logit(int type, const void* base, int64_t at)
{
    const float x = type == kFP32   ? static_cast<const float*>(base)[at]
                    : type == kFP16 ? Element<kFP16>::get(static_cast<const uint16_t*>(base)[at])
                                    : Element<kBF16>::get(static_cast<const uint16_t*>(base)[at]);
    return fminf(x, 3.402823466e38f) + (x != x ? x : 0.f);          // +infinity as the largest number; NaN stays
}

__device__ __forceinline__ bool can_choose(float logit) { return logit > -INFINITY; }

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp64(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL, ROWS>((uint32_t)(u >> 32)) << 32 | dpp<CTRL, ROWS>((uint32_t)u));
}
__device__ __forceinline__ uint64_t lane_value(uint64_t x, int lane)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(x >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((uint32_t)x, lane);
}
__device__ __forceinline__ double lane_value(double x, int lane)
{
    return __builtin_bit_cast(double, lane_value(__builtin_bit_cast(uint64_t, x), lane));
}
__device__ __forceinline__ double wave_sum(double x)
{
    x += dpp64<kDppSwap1>(x);
    x += dpp64<kDppSwap2>(x);
    x += dpp64<kDppHalfMirror>(x);
    x += dpp64<kDppMirror>(x);
    x += dpp64<kDppBcast15, 0xA>(x);
    x += dpp64<kDppBcast31, 0xC>(x);
    return lane_value(x, 63);
}

// Largest of x over the wave (-infinity where none can be chosen).
__device__ __forceinline__ float wave_max_logit(float x)
{
    const uint32_t m = wave_max(can_choose(x) ? ordered(x) : 0u);
    return m == 0 ? -INFINITY : __uint_as_float(m >> 31 ? m & 0x7FFFFFFFu : ~m);
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// Which experts' groups stay open: bit g of the result.  `keys`: the token's
// keys in LDS.  Lanes per group, each of which looks at every n-th of its keys.
__device__ __forceinline__ uint64_t open_groups(const RouteArgs& p, const uint64_t* keys, int lane)
{
    int n = 64;
    while (n > 1 && n * p.groups > 64)
        n >>= 1;
    const int g = lane / n, size = p.experts / p.groups;
    uint64_t a = 0, b = 0;              // the two largest
    if (g < p.groups)
        for (int i = lane % n; i < size; i += n) {
            const uint64_t x = keys[g * size + i];
            b = x > a ? a : x > b ? x : b;
            a = x > a ? x : a;
        }
    for (int d = 1; d < n; d <<= 1) {
        const uint64_t a1 = __shfl_xor(a, d), b1 = __shfl_xor(b, d);
        b = a1 > a ? (a > b1 ? a : b1) : (a1 > b ? a1 : b);
        a = a1 > a ? a1 : a;
    }
    // (a group of whom one can be chosen has that one's key)
    const uint64_t rank = a == 0 ? 0 : b == 0 ? a : ordered(from_ordered(a) + from_ordered(b));
    int ahead = 0;
    for (int h = 0; h < p.groups; ++h) {
        const uint64_t other = lane_value(rank, h * n);
        ahead += other > rank || (other == rank && h < g) ? 1 : 0;
    }
    const uint64_t open = __ballot(lane % n == 0 && g < p.groups && rank != 0 && ahead < p.top_groups);
    uint64_t mask = 0;
    for (int h = 0; h < p.groups; ++h)
        mask |= (open >> (h * n) & 1) << h;
    return mask;
}

template <int S, bool GROUPS>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs p)
{
    __shared__ uint64_t lds[GROUPS ? 4 * 64 * S : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool by_logit = !p.bias && !GROUPS;
    uint64_t* const keys = lds + (GROUPS ? wave * 64 * S : 0);
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < p.tokens; t += (int64_t)gridDim.x * 4) {
        const int64_t at = t * p.ld;
        float x[S];
        float top = -INFINITY;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = 64 * s + lane;
            x[s] = e < p.experts ? route_logit(p.type, p.logits, at + e) : -INFINITY;
            top = can_choose(x[s]) ? fmaxf(top, x[s]) : top;
        }
        // softmax over all experts, where the choice or the weights need it
        double total = 1.0;
        if (!p.sigmoid) {
            top = wave_max_logit(top);
            if (!by_logit || !p.normalize) {
                double sum = 0.0;
#pragma unroll
                for (int s = 0; s < S; ++s)
                    sum += can_choose(x[s]) ? exp((double)x[s] - (double)top) : 0.0;
                total = wave_sum(sum);
            }
        }
        uint64_t key[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = 64 * s + lane;
            if (by_logit) {
                key[s] = can_choose(x[s]) ? (uint64_t)ordered(x[s]) << 32 : 0;
            } else {
                double score = p.sigmoid ? sigmoid64(x[s]) : exp((double)x[s] - (double)top) / total;
                if (p.bias && e < p.experts)
                    score += (double)p.bias[e];
                key[s] = can_choose(x[s]) && score > -INFINITY ? ordered(score) : 0;
            }
        }
        if constexpr (GROUPS) {
            // (one wave reads only what it wrote itself, and its LDS
            // operations complete in order)
#pragma unroll
            for (int s = 0; s < S; ++s)
                keys[64 * s + lane] = key[s];
            __builtin_amdgcn_wave_barrier();
            const uint64_t open = open_groups(p, keys, lane);
            const int size = p.experts / p.groups;
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (!(open >> ((64 * s + lane) / size & 63) & 1))
                    key[s] = 0;
            __builtin_amdgcn_wave_barrier();
        }
        int mine = -1;                  // choice j in lane j
        for (int j = 0; j < p.k; ++j) {
            uint64_t best = key[0];
            int slot = 0;
#pragma unroll
            for (int s = 1; s < S; ++s) {
                slot = key[s] > best ? s : slot;
                best = key[s] > best ? key[s] : best;
            }
            const uint32_t hi = wave_max((uint32_t)(best >> 32));
            if (hi == 0)
                break;                  // nobody is left
            bool has = (uint32_t)(best >> 32) == hi;
            uint64_t who = __ballot(has);
            if (who & (who - 1)) {
                const uint32_t lo = wave_max(has ? (uint32_t)best : 0u);
                has = has && (uint32_t)best == lo;
                // the lowest index of equal ones
                const uint32_t first = ~wave_max(has ? ~(uint32_t)(64 * slot + lane) : 0u);
                has = has && (uint32_t)(64 * slot + lane) == first;
                who = __ballot(has);
            }
            const int from = __builtin_ctzll(who);
            const int e = __builtin_amdgcn_readlane(64 * slot + lane, from);
            mine = lane == j ? e : mine;
#pragma unroll
            for (int s = 0; s < S; ++s)
                key[s] = e == 64 * s + lane ? 0 : key[s];
        }
        const bool has = lane < p.k && mine >= 0;
        const float logit = has ? route_logit(p.type, p.logits, at + mine) : -INFINITY;
        double w = 0.0;
        if (p.sigmoid) {
            w = has ? sigmoid64(logit) : 0.0;
            if (p.normalize) {
                const double sum = wave_sum(w);
                w = sum > 0.0 ? w / sum : 0.0;
            }
        } else {
            const float base = p.normalize ? wave_max_logit(logit) : top;
            w = has ? exp((double)logit - (double)base) : 0.0;
            const double sum = p.normalize ? wave_sum(w) : total;
            w = has ? w / sum : 0.0;
        }
        if (lane < p.k) {
            p.ids[t * p.k + lane] = mine;
            p.weights[t * p.k + lane] = (float)(p.scale * w);
        }
    }
}

// Gradient to the logits, with g_j = scale d_weights_j and w the weights over
// their scale: normalised softmax w_j (g_j - <g w>); softmax s_e (g_e - <g s>)
// over all experts; sigmoid g_j s_j (1 - s_j), normalised with (g_j - <g w>) /
// sum s for g_j.  A wave takes a token; choice j in lane j.
template <int S>
__global__ void __launch_bounds__(256) route_backward_kernel(RouteArgs p)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < p.tokens; t += (int64_t)gridDim.x * 4) {
        const int64_t at = t * p.ld;
        int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
        id = id < p.experts ? id : -1;
        const float logit = id >= 0 ? route_logit(p.type, p.logits, at + id) : -INFINITY;
        const bool has = can_choose(logit);
        const double g = has ? (double)p.scale * (double)p.d_weights[t * p.k + lane] : 0.0;
        double d = 0.0, dot = 0.0, total = 1.0;
        float top = -INFINITY;
        float x[S];
        if (p.sigmoid) {
            const double s = has ? sigmoid64(logit) : 0.0, rest = has ? sigmoid64(-(double)logit) : 0.0;
            if (p.normalize) {
                const double sum = wave_sum(s), mean = sum > 0.0 ? wave_sum(g * s) / sum : 0.0;
                d = sum > 0.0 ? (g - mean) / sum * s * rest : 0.0;
            } else {
                d = g * s * rest;
            }
        } else if (p.normalize) {
            const float base = wave_max_logit(logit);
            const double s = has ? exp((double)logit - (double)base) : 0.0;
            const double sum = wave_sum(s), mean = wave_sum(g * s) / sum;
            d = has ? s / sum * (g - mean) : 0.0;
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int e = 64 * s + lane;
                x[s] = e < p.experts ? route_logit(p.type, p.logits, at + e) : -INFINITY;
                top = can_choose(x[s]) ? fmaxf(top, x[s]) : top;
            }
            top = wave_max_logit(top);
            double sum = 0.0;
#pragma unroll
            for (int s = 0; s < S; ++s)
                sum += can_choose(x[s]) ? exp((double)x[s] - (double)top) : 0.0;
            total = wave_sum(sum);
            d = g;
            const double term = has ? g * (exp((double)logit - (double)top) / total) : 0.0;
            dot = wave_sum(term);
        }
        double out[S];
#pragma unroll
        for (int s = 0; s < S; ++s)
            out[s] = 0.0;
        for (int j = 0; j < p.k; ++j) {
            const int e = __builtin_amdgcn_readlane(id, j);
            const double v = lane_value(d, j);
#pragma unroll
            for (int s = 0; s < S; ++s)
                out[s] += e == 64 * s + lane ? v : 0.0;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = 64 * s + lane;
            if (e >= p.experts)
                continue;
            if (!p.sigmoid && !p.normalize)
                out[s] = can_choose(x[s]) ? exp((double)x[s] - (double)top) / total * (out[s] - dot) : 0.0;
            const float v = (float)out[s];
            const int64_t to = t * p.ld_d + e;
            if (p.type == kFP32)
                static_cast<float*>(p.d_logits)[to] = v;
            else if (p.type == kFP16)
                static_cast<uint16_t*>(p.d_logits)[to] = Element<kFP16>::put(v);
            else
                static_cast<uint16_t*>(p.d_logits)[to] = Element<kBF16>::put(v);
        }
    }
}

// ----------------------------------------------------------------- launch --

template <int S>
static void route_launch(const RouteArgs& a, bool backward, hipStream_t stream)
{
    const int64_t need = (a.tokens + 3) / 4;
    const dim3 grid((unsigned)(need < (1 << 20) ? need : 1 << 20));
    if (backward)
        hipLaunchKernelGGL((route_backward_kernel<S>), grid, dim3(256), 0, stream, a);
    else if (a.groups > 1)
        hipLaunchKernelGGL((route_kernel<S, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((route_kernel<S, false>), grid, dim3(256), 0, stream, a);
}

static hipError_t route_any(const RouteArgs& a, bool backward, hipStream_t stream)
{
    if (a.experts <= 64)
        route_launch<1>(a, backward, stream);
    else if (a.experts <= 128)
        route_launch<2>(a, backward, stream);
    else if (a.experts <= 256)
        route_launch<4>(a, backward, stream);
    else if (a.experts <= 512)
        route_launch<8>(a, backward, stream);
    else
        route_launch<16>(a, backward, stream);
    return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) { return route_any(a, false, stream); }
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t stream) { return route_any(a, true, stream); }

}  // namespace mxg
