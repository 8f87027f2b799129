// Experts of each token and their weights, from the router's logits.
#include <type_traits>

#include "block.h"
#include "element.h"
#include "wave.h"

namespace mxg {

// A wave takes one token at a time, expert 64 s + lane in slot s of a lane.
// Keys, the scores that a choice compares, are formed in 64 bits: scores of
// popular experts differ by less than an FP32 step often enough to change
// choices.  (Without bias and groups the logits themselves are compared.)  The
// next choice is the largest of the keys rounded to FP32, as the unsigned whole
// numbers of the same order, over the lanes; only where several experts have it
// are the keys themselves compared.  0 stands for an expert that is not chosen
// (any more).  Few tokens are bound by one wave's chain of steps, k times a
// maximum over the lanes: 4 tokens of 128 experts, k 8, take 3.8 us.

__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);        // -0 counts as 0
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ float route_logit(int type, const void* base, int64_t at)
{
    const float x = type == kFP32   ? static_cast<const float*>(base)[at]
                    : type == kFP16 ? Element<kFP16>::get(static_cast<const uint16_t*>(base)[at])
                                    : Element<kBF16>::get(static_cast<const uint16_t*>(base)[at]);
    return x == INFINITY ? 3.402823466e38f : x;
}

__device__ __forceinline__ bool can_choose(float logit) { return logit > -INFINITY; }

// exp(x) to 1e-14: x = n ln 2 + r (ln 2 in two parts), the exponential series of
// |r| <= ln 2 / 2 to its eleventh power (the next is below 7e-15), times 2^n.
// Arguments beyond 709 count as 709.  N at a time, step by step: one chain alone
// waits for each of its twenty dependent operations.
template <int N>
__device__ __forceinline__ void exp64(double (&x)[N])
{
    constexpr double c[11] = {1.0 / 3628800, 1.0 / 362880, 1.0 / 40320, 1.0 / 5040, 1.0 / 720, 1.0 / 120,
                              1.0 / 24, 1.0 / 6, 0.5, 1.0, 1.0};
    double n[N], p[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = fmin(fmax(x[i], -746.0), 709.0);
        n[i] = rint(x[i] * 1.4426950408889634);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = fma(n[i], -0.6931471803691238, x[i]);
        x[i] = fma(n[i], -1.9082149292705877e-10, x[i]);
        p[i] = 1.0 / 39916800;
    }
#pragma unroll
    for (int k = 0; k < 11; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i)
            p[i] = fma(p[i], x[i], c[k]);
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = __builtin_amdgcn_ldexp(p[i], (int)n[i]);
}
__device__ __forceinline__ double exp64(double x)
{
    double v[1] = {x};
    exp64(v);
    return v[0];
}
// 1 / x by two Newton steps from the hardware's estimate; 0 < x < 1e305
__device__ __forceinline__ double reciprocal64(double x)
{
    double r = __builtin_amdgcn_rcp(x);
    r = fma(fma(-x, r, 1.0), r, r);
    return fma(fma(-x, r, 1.0), r, r);
}
// below -700: 0
template <int N>
__device__ __forceinline__ void sigmoid64(const float (&z)[N], double (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = -(double)z[i];
    exp64(v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const double s = reciprocal64(1.0 + v[i]);
        v[i] = z[i] < -700.f ? 0.0 : s;
    }
}
__device__ __forceinline__ double sigmoid64(float z)
{
    const float x[1] = {z};
    double v[1];
    sigmoid64(x, v);
    return v[0];
}

// Scores of N logits, before the softmax's division: sigmoid, or exp(x - top); 0
// for those that are not chosen.
template <int N>
__device__ __forceinline__ void scores64(bool sigmoid, const float (&x)[N], float top, double (&v)[N])
{
    if (sigmoid) {
        sigmoid64(x, v);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = (double)x[i] - (double)top;
        exp64(v);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = can_choose(x[i]) ? v[i] : 0.0;
}

// The same for S of them, a few at a time: enough chains to hide each other's
// waits, few enough for the registers.
template <int S>
__device__ __forceinline__ void scores_of(bool sigmoid, const float (&x)[S], float top, double (&v)[S])
{
    constexpr int N = S < 4 ? S : 4;
#pragma unroll
    for (int s = 0; s < S; s += N) {
        float z[N];
        double y[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            z[i] = x[s + i];
        scores64(sigmoid, z, top, y);
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[s + i] = y[i];
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp64(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL, ROWS>((uint32_t)(u >> 32)) << 32 | dpp<CTRL, ROWS>((uint32_t)u));
}
__device__ __forceinline__ double lane_value(double x, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(u >> 32), lane) << 32 |
                                          (uint32_t)__builtin_amdgcn_readlane((uint32_t)u, lane));
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

// Which experts' groups stay open: bit g of the result.  `keys`: the token's
// keys in LDS, -infinity where an expert is not chosen.  n lanes per group, each
// of which looks at every n-th of its keys.
__device__ __forceinline__ uint64_t open_groups(const RouteArgs& p, const double* keys, int n, int lane)
{
    const int g = lane / n, size = p.experts / p.groups;
    double a = -INFINITY, b = -INFINITY;        // the two largest
    if (g < p.groups)
        for (int i = lane & (n - 1); i < size; i += n) {
            const double x = keys[g * size + i];
            b = fmax(b, fmin(a, x));
            a = fmax(a, x);
        }
    for (int d = 1; d < n; d <<= 1) {
        const double a1 = __shfl_xor(a, d), b1 = __shfl_xor(b, d);
        b = fmax(fmax(b, b1), fmin(a, a1));
        a = fmax(a, a1);
    }
    // (a group of whom one can be chosen has that one's key)
    const double rank = b > -INFINITY ? a + b : a;
    int ahead = 0;
    for (int h = 0; h < p.groups; ++h) {
        const double other = lane_value(rank, h * n);
        ahead += other > rank || (other == rank && h < g) ? 1 : 0;
    }
    const uint64_t open = __ballot((lane & (n - 1)) == 0 && g < p.groups && rank > -INFINITY && ahead < p.top_groups);
    uint64_t mask = 0;
    for (int h = 0; h < p.groups; ++h)
        mask |= (open >> (h * n) & 1) << h;
    return mask;
}

// Lanes per group of experts, a power of two.
__device__ __forceinline__ int lanes_per_group(const RouteArgs& p)
{
    int n = 64;
    while (n > 1 && n * p.groups > 64)
        n >>= 1;
    return n;
}

// The choices of one token by a whole wave: choice j in lane j.  top and total:
// the largest logit and (where it was needed) the softmax's sum.  `keys`: the
// wave's LDS, 64 S keys, for groups.
template <int S, bool GROUPS>
__device__ __forceinline__ int choose_by_wave(const RouteArgs& p, int64_t at, int lane, int lanes, double* keys,
                                              float& top, double& total)
{
    const bool by_logit = !p.bias && !GROUPS;
    float x[S];
    top = -INFINITY;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int e = 64 * s + lane;
        x[s] = e < p.experts ? route_logit(p.type, p.logits, at + e) : -INFINITY;
        top = can_choose(x[s]) ? fmaxf(top, x[s]) : top;
    }
    // softmax over all experts, where the choice or the weights need it
    double key[S], part = 1.0;
    total = 1.0;
    if (!p.sigmoid)
        top = wave_max_logit(top);
    if (!by_logit || (!p.sigmoid && !p.normalize)) {
        scores_of<S>(p.sigmoid, x, top, key);
        if (!p.sigmoid) {
            double sum = 0.0;
#pragma unroll
            for (int s = 0; s < S; ++s)
                sum += key[s];
            total = wave_sum(sum);
            part = total > 0.0 ? reciprocal64(total) : 0.0;
        }
    }
    uint32_t near[S];               // the key to FP32, in whole numbers
    if (by_logit) {
#pragma unroll
        for (int s = 0; s < S; ++s)
            near[s] = can_choose(x[s]) ? ordered(x[s]) : 0;
    } else {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = 64 * s + lane;
            const double score = key[s] * part + (p.bias && e < p.experts ? (double)p.bias[e] : 0.0);
            key[s] = can_choose(x[s]) && score > -INFINITY ? score : -INFINITY;
        }
    }
    if constexpr (GROUPS) {
        // (one wave reads only what it wrote itself, and its LDS operations
        // complete in order)
#pragma unroll
        for (int s = 0; s < S; ++s)
            keys[64 * s + lane] = key[s];
        __builtin_amdgcn_wave_barrier();
        const uint64_t open = open_groups(p, keys, lanes, lane);
#pragma unroll
        for (int s = 0; s < S; ++s)
            key[s] = open >> ((64 * s + lane) / (p.experts / p.groups) & 63) & 1 ? key[s] : -INFINITY;
        __builtin_amdgcn_wave_barrier();
    }
    if (!by_logit) {
#pragma unroll
        for (int s = 0; s < S; ++s)
            near[s] = key[s] > -INFINITY ? ordered((float)key[s]) : 0;
    }
    int mine = -1;
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = near[0];
#pragma unroll
        for (int s = 1; s < S; ++s)
            best = max(best, near[s]);
        best = wave_max(best);
        if (best == 0)
            break;                  // nobody is left
        // the lowest index of those that have it, and how many
        int e = 0, n = 0;
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
            const uint64_t who = __ballot(near[s] == best);
            n += __builtin_popcountll(who);
            e = who ? 64 * s + __builtin_ctzll(who) : e;
        }
        if (n > 1 && !by_logit) {   // the largest key of these, then the lowest index
            uint64_t k64 = 0;
#pragma unroll
            for (int s = 0; s < S; ++s)
                k64 = near[s] == best ? max(k64, ordered(key[s])) : k64;
            const uint32_t hi = wave_max((uint32_t)(k64 >> 32));
            const uint32_t lo = wave_max((uint32_t)(k64 >> 32) == hi ? (uint32_t)k64 : 0u);
            const uint64_t most = (uint64_t)hi << 32 | lo;
#pragma unroll
            for (int s = S - 1; s >= 0; --s) {
                const uint64_t who = __ballot(near[s] == best && ordered(key[s]) == most);
                e = who ? 64 * s + __builtin_ctzll(who) : e;
            }
        }
        mine = lane == j ? e : mine;
#pragma unroll
        for (int s = 0; s < S; ++s)
            near[s] = e == 64 * s + lane ? 0 : near[s];
    }
    return mine;
}

template <int S, bool GROUPS>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs p)
{
    __shared__ double lds[GROUPS ? 4 * 64 * S : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double* const keys = lds + (GROUPS ? wave * 64 * S : 0);
    const int lanes = lanes_per_group(p);
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < p.tokens; t += (int64_t)gridDim.x * 4) {
        const int64_t at = t * p.ld;
        float top;
        double total;
        const int mine = choose_by_wave<S, GROUPS>(p, at, lane, lanes, keys, top, total);
        const bool has = lane < p.k && mine >= 0;
        const float logit = has ? route_logit(p.type, p.logits, at + mine) : -INFINITY;
        double w = 0.0;
        if (p.sigmoid) {
            const double score = sigmoid64(has ? logit : 0.f);
            w = has ? score : 0.0;
            if (p.normalize) {
                const double sum = wave_sum(w);
                w = sum > 0.0 ? w / sum : 0.0;
            }
        } else {
            const float base = p.normalize ? wave_max_logit(logit) : top;
            const double e = exp64(has ? (double)logit - (double)base : 0.0);
            w = has ? e : 0.0;
            const double sum = p.normalize ? wave_sum(w) : total;
            w = has ? w / sum : 0.0;
        }
        if (lane < p.k) {
            p.ids[t * p.k + lane] = mine;
            p.weights[t * p.k + lane] = (float)(p.scale * w);
        }
    }
}

// ------------------------------------------------- sixteen lanes per token --

// The same for up to 256 experts and 16 choices, four tokens to a wave: sixteen
// lanes share a token, lane l with experts e = n l .. n l + n - 1, n = ceil(E /
// 16), so that most of a choice's steps are done for four tokens at once.  Groups
// are whole lanes: a power of two of them each.  Keys are formed in FP32 first.
// Only where a choice hangs on less than they are good for, two keys or two
// groups' ranks nearer than `Near` says, does the wave choose by keys in 64 bits.
// 16384 tokens of 256 experts in 8 groups, sigmoid, bias, k 8: 22 to 25 us, where
// the 18 MB that move take 3.5.  They are one generation of four waves per SIMD,
// which wait 62% of their time for their own chains (of 65536 tokens, 68 us, each
// 16384 more take 15).  With the gradient's kernel of this kind 29 us, against 48
// with a wave to a token in both.
struct Near {
    float part, floor;
    __device__ __forceinline__ explicit Near(const RouteArgs& p)
    {
        // sigmoids are good to four steps; a softmax's exponents, differences of
        // logits down to -70, carry their own rounding: 70 2^-24 each.  A bias
        // may cancel a score, at most 1; without one, scores below 1e-30 are
        // all in doubt, since FP32 soon ends there.  In all, a sigmoid's key is off
        // by 6 2^-24 of the score and 2^-24 of itself at most, half a rank by half
        // of its two keys' errors and 2^-24 of itself; two of them by less than 16
        // 2^-24 = 2^-20 of 1 (or the score) and of the magnitudes in them.
        part = p.sigmoid ? 1.f / (1 << 20) : 1.f / (1 << 16);
        floor = p.bias ? 1.f : 1e-26f;
    }
    // a and b are sums of magnitudes up to `size` (also where both are infinite,
    // whose difference is none)
    __device__ __forceinline__ bool doubt(float a, float b, float size) const
    {
        return !(fabsf(a - b) > part * (size + floor));
    }
};

template <int CTRL>
__device__ __forceinline__ void top_two(float& a, float& b)
{
    const float a1 = dpp<CTRL>(a), b1 = dpp<CTRL>(b);
    b = fmaxf(fmaxf(b, b1), fminf(a, a1));
    a = fmaxf(a, a1);
}
// Half of a group's rank, from its lanes' two largest keys: the sum of two large
// biases would leave FP32's range.  (A group of whom one can be chosen has that
// one's key.)  size: the magnitudes in it, to which its error is relative: a large
// bias and its negative leave a small rank with a large error.
__device__ __forceinline__ float half_rank(int lanes, float a, float b, float& size)
{
    if (lanes >= 2)
        top_two<kDppSwap1>(a, b);
    if (lanes >= 4)
        top_two<kDppSwap2>(a, b);
    if (lanes >= 8)
        top_two<kDppHalfMirror>(a, b);
    const bool two = b > -INFINITY;
    size = 0.5f * fabsf(a) + (two ? 0.5f * fabsf(b) : 0.f);
    return two ? 0.5f * a + 0.5f * b : 0.5f * a;
}

__device__ __forceinline__ double row16_sum(double x)
{
    x += dpp64<kDppSwap1>(x);
    x += dpp64<kDppSwap2>(x);
    x += dpp64<kDppHalfMirror>(x);
    return x + dpp64<kDppMirror>(x);
}
__device__ __forceinline__ double row16_max(double x)
{
    x = fmax(x, dpp64<kDppSwap1>(x));
    x = fmax(x, dpp64<kDppSwap2>(x));
    x = fmax(x, dpp64<kDppHalfMirror>(x));
    return fmax(x, dpp64<kDppMirror>(x));
}
__device__ __forceinline__ float from_ordered(uint32_t u) { return __uint_as_float(u >> 31 ? u & 0x7FFFFFFFu : ~u); }
__device__ __forceinline__ float row16_max_logit(float x)
{
    const uint32_t m = row16_max(can_choose(x) ? ordered(x) : 0u);
    return m == 0 ? -INFINITY : from_ordered(m);
}

// exp(x) for x <= 0, or 1 / (1 + exp(-x)), to a few FP32 steps (the shared forms
// carry their argument's rounding): 2^h (1 + l ln 2), h and l the product with
// log2 e in two parts.
__device__ __forceinline__ float exp_near(float x)
{
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f, kLn2 = 0.693147181f;
    x = fminf(fmaxf(x, -150.f), 88.f);
    const float h = x * kHi, l = fmaf(x, kHi, -h) + x * kLo;
    const float e = __builtin_amdgcn_exp2f(h);
    return fmaf(e, l * kLn2, e);
}

// S consecutive logits from `at`, those from `count` on as -infinity.  whole: all
// are there.
template <int S, int TYPE>
__device__ __forceinline__ void load_logits(const void* base, int64_t at, int count, bool whole, float (&x)[S])
{
    const typename Element<TYPE>::T* p = static_cast<const typename Element<TYPE>::T*>(base) + at;
    if (whole) {
        Pack<TYPE, S> v;
        v.load(p);
#pragma unroll
        for (int s = 0; s < S; ++s)
            x[s] = v.get(s);
    } else {
#pragma unroll
        for (int s = 0; s < S; ++s)
            x[s] = s < count ? Element<TYPE>::get(p[s]) : -INFINITY;
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
        x[s] = x[s] == INFINITY ? 3.402823466e38f : x[s];
}

template <int S, bool GROUPS>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) route_rows_kernel(RouteArgs p)
{
    constexpr int kWide = S / 4;        // slots of a lane where the wave has one token
    __shared__ double lds[GROUPS ? 4 * 64 * kWide : 1];
    __shared__ int32_t chosen[16][16];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, row = lane >> 4, l = lane & 15;
    const bool by_logit = !p.bias && !GROUPS;
    const int per = (p.experts + 15) / 16, first = per * l;
    const int count = p.experts - first < per ? p.experts - first : per;        // of this lane's experts
    const int lanes = GROUPS ? p.experts / p.groups / per : 16;                 // of a group
    const bool whole = per == S && p.experts == 16 * S;
    const Near close(p);
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4; t0 < p.tokens; t0 += (int64_t)gridDim.x * 16) {
        const bool real = t0 + row < p.tokens;
        const int64_t t = real ? t0 + row : p.tokens - 1;
        uint32_t near[S];               // keys to FP32, in whole numbers; 0 is not chosen
        float top = -INFINITY;
        bool doubt = false;
        auto load = [&](float (&x)[S]) __attribute__((always_inline)) {
            if (p.type == kFP32)
                load_logits<S, kFP32>(p.logits, t * p.ld + first, count, whole, x);
            else if (p.type == kFP16)
                load_logits<S, kFP16>(p.logits, t * p.ld + first, count, whole, x);
            else
                load_logits<S, kBF16>(p.logits, t * p.ld + first, count, whole, x);
        };
        {
            float x[S];
            load(x);
            if (!p.sigmoid) {
#pragma unroll
                for (int s = 0; s < S; ++s)
                    top = can_choose(x[s]) ? fmaxf(top, x[s]) : top;
                top = row16_max_logit(top);
            }
            if (by_logit) {
#pragma unroll
                for (int s = 0; s < S; ++s)
                    near[s] = can_choose(x[s]) ? ordered(x[s]) : 0;
            } else {
                float key[S];
                if (p.sigmoid) {
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        key[s] = __builtin_amdgcn_rcpf(1.f + exp_near(-x[s]));
                } else {
                    float sum = 0.f;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        key[s] = can_choose(x[s]) ? exp_near(x[s] - top) : 0.f;
                        sum += key[s];
                    }
                    const float part = 1.f / row16_sum(sum);
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        key[s] *= part;
                }
                float a = -INFINITY, b = -INFINITY;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    if (p.bias)
                        key[s] += s < count ? p.bias[first + s] : 0.f;
                    key[s] = can_choose(x[s]) && key[s] > -INFINITY ? key[s] : -INFINITY;
                    if constexpr (GROUPS) {
                        b = fmaxf(b, fminf(a, key[s]));
                        a = fmaxf(a, key[s]);
                    }
                }
                bool open = true;
                if constexpr (GROUPS) {
                    float size;
                    const float rank = half_rank(lanes, a, b, size);
                    int ahead = 0;
#pragma unroll 1
                    for (int h = 0; h < p.groups; ++h) {
                        const float other = __shfl(rank, (threadIdx.x & 48) + h * lanes);
                        ahead += other > rank ? 1 : 0;
                        doubt |= h != l / lanes && rank > -INFINITY && close.doubt(rank, other, size);
                    }
                    open = ahead < p.top_groups;
                }
#pragma unroll
                for (int s = 0; s < S; ++s)
                    near[s] = open && key[s] > -INFINITY ? ordered(key[s]) : 0;
            }
        }
        int32_t* const list = chosen[4 * wave + row];       // choice j in place j
        list[l] = -1;
        __builtin_amdgcn_wave_barrier();
        uint32_t before = 0;
#pragma unroll 1
        for (int j = 0; j <= p.k; ++j) {
            uint32_t best = near[0];
#pragma unroll
            for (int s = 1; s < S; ++s)
                best = max(best, near[s]);
            best = row16_max(best);
            if (!by_logit && j > 0 && best != 0)
                doubt |= close.doubt(from_ordered(before), from_ordered(best), fabsf(from_ordered(before)));
            before = best;
            if (j == p.k)               // only whether the last choice is certain
                break;
            int slot = 64;
#pragma unroll
            for (int s = S - 1; s >= 0; --s)
                slot = near[s] == best ? s : slot;
            // the lowest index that has it: the first lane's
            const bool has = slot < 64 && best != 0;
            const uint32_t who = (uint32_t)(__ballot(has) >> (lane & 48));
            const bool wins = has && (who & ((1u << l) - 1)) == 0;
            if (wins)
                list[j] = first + slot;
            slot = wins ? slot : 64;
#pragma unroll
            for (int s = 0; s < S; ++s)
                near[s] = slot == s ? 0 : near[s];
        }
        __builtin_amdgcn_wave_barrier();
        int mine = list[l];
        __builtin_amdgcn_wave_barrier();
        // the tokens in doubt, one at a time by the whole wave
        uint64_t rows = by_logit ? 0 : __ballot(doubt);
        while (rows) {
            const int which = __builtin_ctzll(rows) >> 4;
            rows &= ~(0xFFFFull << (16 * which));
            const int64_t at = (t0 + which < p.tokens ? t0 + which : p.tokens - 1) * p.ld;
            float unused;
            double sum;
            const int e = choose_by_wave<kWide, GROUPS>(p, at, lane, lanes_per_group(p),
                                                        lds + (GROUPS ? wave * 64 * kWide : 0), unused, sum);
            const int moved = __shfl(e, l);
            mine = row == which ? moved : mine;
        }
        const bool has = l < p.k && mine >= 0;
        const float logit = has ? route_logit(p.type, p.logits, t * p.ld + mine) : -INFINITY;
        double w = 0.0;
        if (p.sigmoid) {
            const double score = sigmoid64(has ? logit : 0.f);
            w = has ? score : 0.0;
            if (p.normalize) {
                const double sum = row16_sum(w);
                w = sum > 0.0 ? w * reciprocal64(sum) : 0.0;
            }
        } else {
            const float base = p.normalize ? row16_max_logit(logit) : top;
            const double e = exp64(has ? (double)logit - (double)base : 0.0);
            w = has ? e : 0.0;
            double sum = w;
            if (!p.normalize) {         // the sum over all experts, from their logits once more
                float x[S];
                asm volatile("" ::: "memory");
                load(x);
                sum = 0.0;
#pragma unroll
                for (int s = 0; s < S; s += 2) {
                    const float z[2] = {x[s], x[s + 1]};
                    double v[2];
                    scores64(false, z, top, v);
                    sum += v[0] + v[1];
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            sum = row16_sum(sum);
            w = has ? w * reciprocal64(sum) : 0.0;
        }
        if (real && l < p.k) {
            p.ids[t0 * p.k + row * p.k + l] = mine;
            p.weights[t0 * p.k + row * p.k + l] = (float)(p.scale * w);
        }
    }
}

// --------------------------------------------------------------- gradient ----

// Gradient to the logits, with g_j = scale d_weights_j and w the weights over
// their scale: normalised softmax w_j (g_j - <g w>); softmax s_e (g_e - <g s>)
// over all experts; sigmoid g_j s_j (1 - s_j), normalised with (g_j - <g w>) /
// sum s for g_j.  In 64 bits: g - <g w> cancels where one choice has most weight.

// (g - <g w>) times the sum of scores, dot = <g score>: two products, not one and a
// multiply-add, so that nothing is left where one choice has all weight.
__device__ __forceinline__ double from_mean(double g, double all, double dot)
{
#pragma clang fp contract(off)
    return g * all - dot;
}

// The gradient of one choice: lane j of those that share a token has its logit,
// g_j and whether it was chosen; sums over them by `sum`, maximum by `largest`.
template <class Sum, class Max>
__device__ __forceinline__ double choice_gradient(const RouteArgs& p, float logit, bool has, double g, const Sum& sum,
                                                  const Max& largest)
{
    if (p.sigmoid) {
        const double e = exp64(has ? -(double)logit : 0.0), s = reciprocal64(1.0 + e);
        const double score = has && logit >= -700.f ? s : 0.0, slope = score * e * s;      // 1 - s = e s
        if (!p.normalize)
            return g * slope;
        const double all = sum(score), dot = sum(g * score), part = all > 0.0 ? reciprocal64(all) : 0.0;
        return from_mean(g, all, dot) * part * (part * slope);      // (1 / the sum may be 1e304)
    }
    const float base = largest(logit);
    const double e = exp64(has ? (double)logit - (double)base : 0.0), score = has ? e : 0.0;
    const double all = sum(score), dot = sum(g * score), part = all > 0.0 ? reciprocal64(all) : 0.0;
    return score * part * (from_mean(g, all, dot) * part);
}

// Where only the chosen logits have a gradient, sixteen lanes per token as above:
// choice j in lane j, whose gradient goes to the token's row in LDS one choice
// after the other (an index given twice counts twice), and the row from there to
// memory.  16384 tokens of 256 experts, k 8: 6.6 us, where 26 MB move (3.9 TB/s);
// 10.4 with runs of sixteen experts a lane, which met in a few of LDS's banks.
template <int S>
__global__ void __launch_bounds__(256) route_rows_backward_kernel(RouteArgs p)
{
    __shared__ __attribute__((aligned(16))) float lds[16][16 * S];
    const int l = threadIdx.x & 15, wave = threadIdx.x >> 6, row = (threadIdx.x & 63) >> 4;
    float* const mine = lds[4 * wave + row];
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4; t0 < p.tokens; t0 += (int64_t)gridDim.x * 16) {
        const bool real = t0 + row < p.tokens;
        const int64_t t = real ? t0 + row : p.tokens - 1;
        int id = l < p.k ? p.ids[t * p.k + l] : -1;
        id = id < p.experts ? id : -1;
        const float logit = id >= 0 ? route_logit(p.type, p.logits, t * p.ld + id) : -INFINITY;
        const bool has = can_choose(logit);
        const double g = has ? (double)p.scale * (double)p.d_weights[t * p.k + l] : 0.0;
        const float d = (float)choice_gradient(p, logit, has, g, [](double v) { return row16_sum(v); },
                                               [](float v) { return row16_max_logit(v); });
#pragma unroll
        for (int s = 0; s < S; s += 4)
            *reinterpret_cast<v4f*>(mine + 16 * s + 4 * l) = v4f{0.f, 0.f, 0.f, 0.f};
        // (the lanes of a wave meet only their own wave's rows, whose LDS
        // operations complete in order)
        __builtin_amdgcn_wave_barrier();
        for (int j = 0; j < p.k; ++j) {
            if (l == j && id >= 0)
                mine[id] += d;
            __builtin_amdgcn_wave_barrier();
        }
        // (four experts a lane, so that a token's lanes read and write a run)
        v4f out[S / 4];
#pragma unroll
        for (int s = 0; s < S / 4; ++s)
            out[s] = *reinterpret_cast<const v4f*>(mine + 64 * s + 4 * l);
        __builtin_amdgcn_wave_barrier();
        if (!real)
            continue;
        auto put = [&](auto tc) __attribute__((always_inline)) {
            constexpr int TYPE = decltype(tc)::value;
            typename Element<TYPE>::T* to = static_cast<typename Element<TYPE>::T*>(p.d_logits) + t * p.ld_d;
#pragma unroll
            for (int s = 0; s < S / 4; ++s) {
                const int c = 64 * s + 4 * l;
                if (c + 4 <= p.experts) {
                    Pack<TYPE, 4> v;
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        v.put(u, out[s][u]);
                    v.store(to + c);
                } else {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (c + u < p.experts)
                            to[c + u] = Element<TYPE>::put(out[s][u]);
                }
            }
        };
        if (p.type == kFP32)
            put(std::integral_constant<int, kFP32>());
        else if (p.type == kFP16)
            put(std::integral_constant<int, kFP16>());
        else
            put(std::integral_constant<int, kBF16>());
    }
}

// A wave takes a token; choice j in lane j.  ALL: every logit has a gradient
// (softmax that is not normalised).
template <int S, bool ALL>
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
        float out[S];
        if constexpr (ALL) {
            double score[S], sum = 0.0;
            float x[S], top = -INFINITY;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int e = 64 * s + lane;
                x[s] = e < p.experts ? route_logit(p.type, p.logits, at + e) : -INFINITY;
                top = can_choose(x[s]) ? fmaxf(top, x[s]) : top;
            }
            top = wave_max_logit(top);
            scores_of<S>(false, x, top, score);
#pragma unroll
            for (int s = 0; s < S; ++s)
                sum += score[s];
            const double total = wave_sum(sum), part = total > 0.0 ? 1.0 / total : 0.0;
            const double mine = exp64(has ? (double)logit - (double)top : 0.0) * part;
            const double dot = wave_sum(has ? g * mine : 0.0);
            double d[S];
#pragma unroll
            for (int s = 0; s < S; ++s)
                d[s] = -dot;
            for (int j = 0; j < p.k; ++j) {
                const int e = __builtin_amdgcn_readlane(id, j);
                const double v = lane_value(g, j);
#pragma unroll
                for (int s = 0; s < S; ++s)
                    d[s] += e == 64 * s + lane ? v : 0.0;
            }
#pragma unroll
            for (int s = 0; s < S; ++s)
                out[s] = (float)(score[s] * part * d[s]);
        } else {
            const double d = choice_gradient(p, logit, has, g, [](double v) { return wave_sum(v); },
                                             [](float v) { return wave_max_logit(v); });
            const float one = (float)d;
#pragma unroll
            for (int s = 0; s < S; ++s)
                out[s] = 0.f;
            // (an index given twice counts twice)
            for (int j = 0; j < p.k; ++j) {
                const int e = __builtin_amdgcn_readlane(id, j);
                const float v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(one), j));
#pragma unroll
                for (int s = 0; s < S; ++s)
                    out[s] += e == 64 * s + lane ? v : 0.f;
            }
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = 64 * s + lane;
            if (e >= p.experts)
                continue;
            const int64_t to = t * p.ld_d + e;
            if (p.type == kFP32)
                static_cast<float*>(p.d_logits)[to] = out[s];
            else if (p.type == kFP16)
                static_cast<uint16_t*>(p.d_logits)[to] = Element<kFP16>::put(out[s]);
            else
                static_cast<uint16_t*>(p.d_logits)[to] = Element<kBF16>::put(out[s]);
        }
    }
}

// ----------------------------------------------------------------- launch --

template <int S>
static void route_launch(const RouteArgs& a, bool backward, hipStream_t stream)
{
    const int64_t need = (a.tokens + 3) / 4;
    const dim3 grid((unsigned)(need < (1 << 20) ? need : 1 << 20));
    if (backward && !a.sigmoid && !a.normalize)
        hipLaunchKernelGGL((route_backward_kernel<S, true>), grid, dim3(256), 0, stream, a);
    else if (backward)
        hipLaunchKernelGGL((route_backward_kernel<S, false>), grid, dim3(256), 0, stream, a);
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

template <int S>
static void route_rows_launch(const RouteArgs& a, bool backward, hipStream_t stream)
{
    const int64_t need = (a.tokens + 15) / 16;
    const dim3 grid((unsigned)(need < (1 << 20) ? need : 1 << 20));
    if (backward)
        hipLaunchKernelGGL((route_rows_backward_kernel<S>), grid, dim3(256), 0, stream, a);
    else if (a.groups > 1)
        hipLaunchKernelGGL((route_rows_kernel<S, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((route_rows_kernel<S, false>), grid, dim3(256), 0, stream, a);
}

static hipError_t route_rows(const RouteArgs& a, bool backward, hipStream_t stream)
{
    const int per = (a.experts + 15) / 16;
    if (per <= 4)
        route_rows_launch<4>(a, backward, stream);
    else if (per <= 8)
        route_rows_launch<8>(a, backward, stream);
    else
        route_rows_launch<16>(a, backward, stream);
    return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream)
{
    const int per = (a.experts + 15) / 16, size = a.experts / a.groups, lanes = size / per;
    const bool whole = a.groups == 1 || (size % per == 0 && (lanes & (lanes - 1)) == 0);
    // Few tokens wait for one wave's steps, which are fewer where it has one
    // token.  A wave to a token / four tokens to a wave, k 8, us at 4096, 16384 and
    // 65536 tokens: 256 experts by their logits 6.7 / 6.7, 16.7 / 10.8, 57 / 33;
    // by sigmoid and bias 8.1 / 12.2, 21.0 / 19.7, 74 / 54; in 8 groups 10.7 /
    // 14.8, 29.5 / 23.9, 105 / 68; 64 experts in 4 groups, k 4, softmax and bias
    // 6.3 / 7.3, 15.5 / 9.3, 50 / 23.  Where many tokens are in doubt the second
    // catches up later: 16-bit logits in groups without a bias, whose equal keys
    // all are (256 experts in 8 groups 10.9 / 27.1, 29.4 / 36.2, 104 / 102), and 16
    // choices by softmax and bias (10.9 / 22.4, 28.0 / 33.7, 100 / 86).
    return a.experts <= 256 && a.k <= 16 && whole && a.tokens > 4096 ? route_rows(a, false, stream)
                                                                     : route_any(a, false, stream);
}
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t stream)
{
    const bool chosen = a.sigmoid || a.normalize;       // else every logit has a gradient
    return a.experts <= 256 && a.k <= 16 && chosen ? route_rows(a, true, stream) : route_any(a, true, stream);
}

}  // namespace mxg
