// FP8 codes with a float32 scale for each block of 128, along the rows, along
// the columns and in squares.
#include "activation.h"
#include "block.h"
#include "element.h"
#include "quant.h"
#include "segments.h"
#include "wave.h"

namespace mxg {

// A block's scale and what its elements are multiplied by.  The scale is the
// largest magnitude over the format's (7 2^6 or 7 2^13: times 1 / 7, in two
// parts), at least 2^-126 so that its reciprocal is a number; a block that holds
// a NaN or an infinity has a NaN scale and NaN codes, since no scale represents
// it.  The factor is the reciprocal of the scale before its rounding, in two
// parts, from the hardware's estimate and one Newton step: a code hangs on which
// side of a tie the quotient lies, and so only the quotient's own rounding
// counts.  (Divisions instead cost a fifth of all instructions.)
struct BlockScale {
    float s, mul, low;      // NaN, all three, for a block of NaN codes
};

template <int F>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits)
{
    constexpr float kUnit = F == kE5M2 ? 1.f / 8192 : 1.f / 64;
    constexpr float kHi = 0.142857149f * kUnit, kLo = -6.386212e-09f * kUnit;       // 1 / 7
    constexpr float kLow = 1.1754943508222875e-38f;     // 2^-126
    const float amax = __uint_as_float(amax_bits);
    BlockScale b;
    b.s = fmaf(amax, kHi, amax * kLo);
    float rest = fmaf(amax, kHi, -b.s) + amax * kLo;    // what the rounding of s left
    rest = b.s < kLow ? 0.f : rest;
    b.s = fmaxf(b.s, kLow);
    const float r = __builtin_amdgcn_rcpf(b.s), e = fmaf(-b.s, r, 1.f) - rest * r;
    b.mul = fmaf(e, r, r);
    b.low = fmaf(e, r, r - b.mul);
    if (amax_bits >= 0x7F800000u)
        b.s = b.mul = b.low = __uint_as_float(0x7FC00000u);
    return b;
}

// Codes of four elements, first in the low byte; round to nearest even.  (The
// quotient of the block's largest element may come out an FP32 step over fmax,
// which rounds to fmax.)
template <int F>
__device__ __forceinline__ uint32_t block_codes(const BlockScale& b, float x, float y, float z, float w)
{
    x = fmaf(x, b.mul, x * b.low);
    y = fmaf(y, b.mul, y * b.low);
    z = fmaf(z, b.mul, z * b.low);
    w = fmaf(w, b.mul, w * b.low);
    int c;
    if constexpr (F == kE5M2) {
        c = __builtin_amdgcn_cvt_pk_bf8_f32(x, y, 0, false);
        c = __builtin_amdgcn_cvt_pk_bf8_f32(z, w, c, true);
    } else {
        c = __builtin_amdgcn_cvt_pk_fp8_f32(x, y, 0, false);
        c = __builtin_amdgcn_cvt_pk_fp8_f32(z, w, c, true);
    }
    return isnan(b.mul) ? 0x7F7F7F7Fu : (uint32_t)c;
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// ------------------------------------------------------------------- tile ----

// A work-group of 256 threads takes a tile of 128 rows x 128 columns: lane
// group l = tid % 16 columns 8 l .. 8 l + 7, thread group r = tid / 16 rows
// 8 r .. 8 r + 7.  A block along the columns is then sixteen neighbouring
// lanes; one along the rows is the sixteen thread groups, whose maxima meet in
// LDS.  A thread's eight rows of a column are eight bytes of the transposed
// codes; the tile of those goes through LDS so that whole columns of 128 bytes
// are written.  y is read and formed once for both ways.  Bound by memory: 16384 x
// 4096 gated bfloat16 along the columns, 167 MB in 35 us (4.7 TB/s).
constexpr int kTile = 128;

struct TileLds {
    uint32_t amax[4][kTile];
    float2 factor[kTile + kTile / 8];
    uint8_t codes[kTile * kTile];
};

// Byte of (column, row) in the tile of transposed codes: rows of 128 bytes whose
// 16-byte chunks are swizzled, so that neither eight columns apart (the writes)
// nor whole columns (the reads) meet in a few banks.
__device__ __forceinline__ int code_at(int col, int row)
{
    return col * kTile + ((((row >> 4) ^ (col >> 3)) & 7) << 4) + (row & 15);
}

// Codes along the columns of N of a thread's rows [row, ..) below `end`, block tb
// of the row; those from `live` on are zero, codes and scales.
template <int F, int N>
__device__ __forceinline__ void put_rows8(const float (&v)[N][8], uint8_t* q, int64_t ld_q, float* s, int64_t ld_s,
                                          int64_t row, int64_t end, int64_t live, int tb, int tid)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            m = max(m, magnitude(v[i][u]));
        const BlockScale b = block_scale<F>(row16_max(m));
        if (row + i < end) {
            *reinterpret_cast<u32x2*>(q + (row + i) * ld_q + tb * kTile + 8 * (tid & 15)) =
                u32x2{block_codes<F>(b, v[i][0], v[i][1], v[i][2], v[i][3]),
                      block_codes<F>(b, v[i][4], v[i][5], v[i][6], v[i][7])};
            if ((tid & 15) == 0)
                s[tb * ld_s + row + i] = row + i < live ? b.s : 0.f;
        }
    }
}

// The eight columns' maxima over the wave's rows, for lds.amax.
template <int N>
__device__ __forceinline__ void column_max(const float (&v)[N][8], uint32_t* amax, int lane)
{
    uint32_t m[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        m[u] = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            m[u] = max(m[u], magnitude(v[i][u]));
        m[u] = max(m[u], (uint32_t)__shfl_xor((int)m[u], 16));
        m[u] = max(m[u], (uint32_t)__shfl_xor((int)m[u], 32));
    }
    if (lane < 16) {
        *reinterpret_cast<u32x4*>(amax + 8 * lane) = u32x4{m[0], m[1], m[2], m[3]};
        *reinterpret_cast<u32x4*>(amax + 8 * lane + 4) = u32x4{m[4], m[5], m[6], m[7]};
    }
}

// The factor of the thread's column u.  (One in nine places is empty: the
// sixteen threads of a row read eight columns apart, of which all would meet in
// an eighth of the banks.)
__device__ __forceinline__ BlockScale factor_of(const float2* factor, int u, int tid)
{
    const float2 f = factor[9 * (tid & 15) + u];
    return {0.f, f.x, f.y};
}

// N rows of the thread's column u, transposed, to the tile of codes.
template <int F, int N>
__device__ __forceinline__ void flip(const float (&v)[N][8], const BlockScale& b, int u, uint8_t* codes, int row, int tid)
{
    uint8_t* to = codes + code_at(8 * (tid & 15) + u, row);
    if constexpr (N == 8)
        *reinterpret_cast<u32x2*>(to) = u32x2{block_codes<F>(b, v[0][u], v[1][u], v[2][u], v[3][u]),
                                              block_codes<F>(b, v[4][u], v[5][u], v[6][u], v[7][u])};
    else
        *reinterpret_cast<uint32_t*>(to) = block_codes<F>(b, v[0][u], v[1][u], v[2][u], v[3][u]);
}

// The transposed codes out of LDS: column c of the tile, below `cols`, to row
// c of out, by NT threads.
template <int NT>
__device__ __forceinline__ void put_columns(const uint8_t* codes, uint8_t* out, int64_t ld, int cols, int tid)
{
#pragma unroll
    for (int k = 0; k < kTile * 8 / NT; ++k) {
        const int c = NT / 8 * k + (tid >> 3), at = 16 * (tid & 7);
        if (c < cols)
            *reinterpret_cast<u32x4*>(out + c * ld + at) = *reinterpret_cast<const u32x4*>(codes + code_at(c, at));
    }
}

// ----------------------------------------------------------- activations ----

// silu and its derivative a few roundings from exact: a code hangs on which side of
// a tie y lies, so errors of the shared, faster form (an exponential that carries
// its argument's rounding) show as codes that differ: twice as many from the exact
// ones' as this form has.  exp(-z) as 2^h (1 + l ln 2), h and l the product -z log2
// e in two parts; the reciprocal with one Newton step.  rest: 1 - the sigmoid, for
// z > 2 from the exponential, since the difference loses the sigmoid's rounding
// times z to the derivative (16 roundings of that at z = 16).  gelu and gelu_tanh
// keep the shared forms: another form of gelu spilled registers.
__device__ __forceinline__ float sigmoid_near(float z, float& rest)
{
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f, kLn2 = 0.693147181f;
    const float h = -z * kHi, l = fmaf(-z, kHi, -h) - z * kLo;
    float e = __builtin_amdgcn_exp2f(h);
    const float far = __builtin_amdgcn_rcpf(1.f + e);       // 0 or 1, or NaN
    e = fmaf(e, l * kLn2, e);
    const float d = 1.f + e, r = __builtin_amdgcn_rcpf(d);
    const bool near = fabsf(h) < 126.f;
    const float s = near ? fmaf(fmaf(-d, r, 1.f), r, r) : far;
    rest = near && z > 2.f ? e * s : 1.f - s;
    return s;
}

__device__ __forceinline__ void activate8(int act, float (&z)[8])
{
    if (act == kActSilu) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            float rest;
            z[u] *= sigmoid_near(z[u], rest);
        }
    } else {
        activate(act, z);
    }
}

// z becomes act'(z), y gets act(z)
__device__ __forceinline__ void activate_grads8(int act, float (&z)[8], float (&y)[8])
{
    if (act == kActSilu) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            float rest;
            const float s = sigmoid_near(z[u], rest);
            y[u] = z[u] * s;
            z[u] = s * fmaf(z[u], rest, 1.f);
        }
    } else {
        activate_grads(act, z, y);
    }
}

// Eight elements as loaded.
template <int TYPE>
struct Raw {
    uint32_t w[TYPE == kFP32 ? 8 : 4];
    __device__ __forceinline__ void load(const void* base, int64_t at)
    {
        __builtin_memcpy(w, static_cast<const typename Element<TYPE>::T*>(base) + at, sizeof(w));
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
};

template <int N>
__device__ __forceinline__ void clear(float (&v)[N][8])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[i][u] = 0.f;
}

// The thread's eight rows of y from `row` on, columns c .. c + 7, where a row
// comes in whole eights: the loads of kBatch rows go out before the first is
// used.  Rows from `live` and columns from C on are zero; what is loaded there
// is the last row, or the last eight columns, there is (a row below `live` must be
// one of the tile's).
template <int TYPE, bool BACK>
__device__ __forceinline__ void values8x8(const BlockQuantArgs& p, int64_t row, int64_t live, int c, float (&v)[8][8])
{
    constexpr int kBatch = TYPE == kFP32 || BACK ? 2 : 4;
    const int half = p.half;
    const bool up = BACK && half && c >= half;
    const int width = half ? half : p.C, at = up ? c - half : c;
    const int cc = at < width ? at : width - 8;
    const bool there = c < p.C;
#pragma unroll
    for (int i0 = 0; i0 < 8; i0 += kBatch) {
        Raw<TYPE> x[kBatch], x1[BACK ? 1 : kBatch];
        Raw<kBF16> z[BACK ? kBatch : 1], z1[BACK ? kBatch : 1];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            int64_t r = row + i0 + i;
            r = r < live ? r : live - 1;
            x[i].load(p.x, r * p.ld_x + cc);
            if constexpr (BACK) {
                z[i].load(p.z, r * p.ld_z + cc);
                if (half && !up)
                    z1[i].load(p.z, r * p.ld_z + half + cc);
            } else if (half) {
                x1[i].load(p.x, r * p.ld_x + half + cc);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float (&y)[8] = v[i0 + i];
            x[i].get(y);
            if constexpr (BACK) {
                float s[8], a[8];
                z[i].get(s);
                activate_grads8(p.act, s, a);
                if (up) {
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        y[u] *= a[u];
                } else {
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        y[u] *= s[u];
                    if (half) {
                        z1[i].get(a);
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            y[u] *= a[u];
                    }
                }
            } else {
                activate8(p.act, y);
                if (half) {
                    float u1[8];
                    x1[i].get(u1);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        y[u] *= u1[u];
                }
            }
            const bool ok = there && row + i0 + i < live;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                y[u] = ok ? y[u] : 0.f;
        }
    }
}

// Eight columns of one row of y, from column c on (zero past C).
template <int TYPE, bool BACK>
__device__ __forceinline__ void value8(const BlockQuantArgs& p, int64_t row, int c, float (&v)[8])
{
    const int half = p.half;
    if constexpr (!BACK) {
        if (!half) {
            load8<TYPE>(p.x, row * p.ld_x, c, p.C, v);
            activate8(p.act, v);
        } else {
            float u[8];
            load8<TYPE>(p.x, row * p.ld_x, c, half, v);
            load8<TYPE>(p.x, row * p.ld_x + half, c, half, u);
            activate8(p.act, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] *= u[i];
        }
    } else {
        // the columns as [first, first + 8) of one half; a piece that reaches
        // over the middle is taken a column at a time
        const bool up = half && c >= half;
        if (!half || up || c + 8 <= half) {
            const int width = half ? half : p.C, first = up ? c - half : c;
            float z[8], z1[8], y[8];
            load8<TYPE>(p.x, row * p.ld_x, first, width, v);
            load8<kBF16>(p.z, row * p.ld_z, first, width, z);
            if (half && !up)
                load8<kBF16>(p.z, row * p.ld_z + half, first, width, z1);
            activate_grads8(p.act, z, y);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] *= !half ? z[i] : up ? y[i] : z[i] * z1[i];
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 0.f;
#pragma unroll 1
        for (int i = 0; i < 8 && c + i < p.C; ++i) {
            const bool hi = c + i >= half;
            const int col = hi ? c + i - half : c + i;
            float d[8], z[8], z1[8], y[8];
            load8<TYPE>(p.x, row * p.ld_x, col, col + 1, d);
            load8<kBF16>(p.z, row * p.ld_z, col, col + 1, z);
            load8<kBF16>(p.z, row * p.ld_z + half, col, col + 1, z1);
            activate_grads8(p.act, z, y);
            const float one = d[0] * (hi ? y[0] : z[0] * z1[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = j == i ? one : v[j];
        }
    }
}

// By expert, what no segment holds is zero: the rows of dropped pairs, and
// the columns of qt past the last segment.
__device__ __forceinline__ void clear_rest(const BlockQuantArgs& p, int chunk, int tc)
{
    const int tid = threadIdx.x;
    const int64_t Cp = (p.C + kTile - 1) / kTile * kTile;
    if (p.qt && chunk < p.chunks) {
        const int cols = p.C - tc * kTile < kTile ? p.C - tc * kTile : kTile;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = 32 * k + (tid >> 3);
            if (c < cols)
                *reinterpret_cast<u32x4*>(p.qt + (tc * kTile + c) * p.ld_qt + (int64_t)chunk * kTile + 16 * (tid & 7)) =
                    u32x4{0, 0, 0, 0};
        }
        if (tid < cols)
            p.st[(int64_t)chunk * p.C + tc * kTile + tid] = 0.f;
    }
    if (!p.q || p.rows == 0)
        return;
    // the chunks past the last segment share the dropped rows
    int first = p.k_offsets[p.groups], live = p.offsets[p.groups];
    first = first < 0 ? 0 : (first + kTile - 1) / kTile;
    first = first < p.chunks ? first : p.chunks;
    live = live < 0 ? 0 : live;
    const int64_t stride = (int64_t)(p.chunks + 1 - first) * 32;
    for (int64_t row = live + (int64_t)(chunk - first) * 32 + (tid >> 3); row < p.rows; row += stride) {
        *reinterpret_cast<u32x4*>(p.q + row * Cp + tc * kTile + 16 * (tid & 7)) = u32x4{0, 0, 0, 0};
        if ((tid & 7) == 0)
            p.s[(int64_t)tc * p.rows + row] = 0.f;
    }
}

// VEC: rows of whole eights.
template <int F, int TYPE, bool BACK, bool VEC>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) block_quant_kernel(BlockQuantArgs p)
{
    __shared__ TileLds lds;
    const int tid = threadIdx.x, tc = blockIdx.x, chunk = blockIdx.y;
    int row0 = chunk * kTile, end = p.rows, live = p.rows;
    if (!p.qt) {        // rows in any order: no segments, the dropped ones last
        if (p.offsets)
            live = min(max(p.offsets[p.groups], 0), p.rows);
    } else {
        if (p.rows == 0 || !segment_rows(p, chunk, row0, end)) {   // (no row may be read)
            clear_rest(p, chunk, tc);
            return;
        }
        live = end;
    }
    const int c = tc * kTile + 8 * (tid & 15);
    const int64_t row = row0 + 8 * (tid >> 4);
    float v[8][8];
    if constexpr (VEC) {
        if (row0 < live)
            values8x8<TYPE, BACK>(p, row, live, c, v);
        else            // of a tile of dropped rows nothing is read
            clear(v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (row + i < live) {
                value8<TYPE, BACK>(p, row + i, c, v[i]);
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[i][u] = 0.f;
            }
        }
    }
    if (p.q)
        put_rows8<F>(v, p.q, (int64_t)(p.C + kTile - 1) / kTile * kTile, p.s, p.rows, row, end, live, tc, tid);
    if (!p.qt)
        return;
    column_max(v, lds.amax[tid >> 6], tid & 63);
    __syncthreads();
    if (tid < kTile) {
        const BlockScale b = block_scale<F>(max(max(lds.amax[0][tid], lds.amax[1][tid]),
                                                max(lds.amax[2][tid], lds.amax[3][tid])));
        lds.factor[tid + tid / 8] = make_float2(b.mul, b.low);
        if (tc * kTile + tid < p.C)
            p.st[(int64_t)chunk * p.C + tc * kTile + tid] = b.s;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 8; ++u)
        flip<F>(v, factor_of(lds.factor, u, tid), u, lds.codes, 8 * (tid >> 4), tid);
    __syncthreads();
    put_columns<256>(lds.codes, p.qt + (int64_t)tc * kTile * p.ld_qt + (int64_t)chunk * kTile, p.ld_qt, p.C - tc * kTile,
                     tid);
}

// A gated gradient whose halves are whole blocks: a work-group of 512 threads
// takes the tile's columns of both halves, [x u act'(g), x act(g)], so that x, g
// and u are read and the activation is evaluated once; a thread has four rows.
// 8002 x 4096 in ragged segments, both ways: 175 MB in 44 us (4.0 TB/s), against
// 56 with a work-group for each half; the rest is its instructions.
struct PairLds {
    uint32_t amax[2][8][kTile];
    float2 factor[2][kTile + kTile / 8];
    uint8_t codes[2][kTile * kTile];
};

template <int F, int TYPE>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(TYPE == kFP32 ? 2 : 4)))
block_quant_pair_kernel(BlockQuantArgs p)
{
    __shared__ PairLds lds;
    const int tid = threadIdx.x, tc = blockIdx.x, chunk = blockIdx.y, tiles = p.half / kTile;
    int row0 = chunk * kTile, end = p.rows, live = p.rows;
    if (!p.qt) {        // rows in any order: no segments, the dropped ones last
        if (p.offsets)
            live = min(max(p.offsets[p.groups], 0), p.rows);
    } else {
        if (p.rows == 0 || !segment_rows(p, chunk, row0, end)) {   // (no row may be read)
            if (tid < 256) {
                clear_rest(p, chunk, tc);
                clear_rest(p, chunk, tc + tiles);
            }
            return;
        }
        live = end;
    }
    const int c = tc * kTile + 8 * (tid & 15);
    const int64_t row = row0 + 4 * (tid >> 4);
    float v[4][8], w[4][8];
    constexpr int kBatch = TYPE == kFP32 ? 1 : 2;       // rows whose loads go out together
    if (row0 >= live) {         // of a tile of dropped rows nothing is read
        clear(v);
        clear(w);
    } else {
#pragma unroll
        for (int i0 = 0; i0 < 4; i0 += kBatch) {
            Raw<TYPE> x[kBatch];
            Raw<kBF16> g[kBatch], u[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                int64_t r = row + i0 + i;
                r = r < live ? r : live - 1;
                x[i].load(p.x, r * p.ld_x + c);
                g[i].load(p.z, r * p.ld_z + c);
                u[i].load(p.z, r * p.ld_z + p.half + c);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float d[8], s[8], a[8], y[8];
                x[i].get(d);
                g[i].get(s);
                u[i].get(y);
                activate_grads8(p.act, s, a);
                const bool ok = row + i0 + i < live;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    v[i0 + i][k] = ok ? d[k] * s[k] * y[k] : 0.f;
                    w[i0 + i][k] = ok ? d[k] * a[k] : 0.f;
                }
            }
        }
    }
    if (p.q) {
        put_rows8<F>(v, p.q, p.C, p.s, p.rows, row, end, live, tc, tid);
        put_rows8<F>(w, p.q, p.C, p.s, p.rows, row, end, live, tc + tiles, tid);
    }
    if (!p.qt)
        return;
    column_max(v, lds.amax[0][tid >> 6], tid & 63);
    column_max(w, lds.amax[1][tid >> 6], tid & 63);
    __syncthreads();
    if (tid < 2 * kTile) {
        const int h = tid / kTile, k = tid % kTile;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, lds.amax[h][i][k]);
        const BlockScale b = block_scale<F>(m);
        lds.factor[h][k + k / 8] = make_float2(b.mul, b.low);
        p.st[(int64_t)chunk * p.C + h * p.half + tc * kTile + k] = b.s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        flip<F>(v, factor_of(lds.factor[0], k, tid), k, lds.codes[0], 4 * (tid >> 4), tid);
        flip<F>(w, factor_of(lds.factor[1], k, tid), k, lds.codes[1], 4 * (tid >> 4), tid);
    }
    __syncthreads();
    uint8_t* const out = p.qt + (int64_t)tc * kTile * p.ld_qt + (int64_t)chunk * kTile;
    put_columns<512>(lds.codes[0], out, p.ld_qt, kTile, tid);
    put_columns<512>(lds.codes[1], out + p.half * p.ld_qt, p.ld_qt, kTile, tid);
}

// ---------------------------------------------------------------- squares ----

// One scale for the tile.  24 x 2048 x 2048 bfloat16, both ways: 403 MB in 81 us
// (5.0 TB/s).
template <int F, int TYPE>
__global__ void __launch_bounds__(256) square_quant_kernel(SquareQuantArgs p)
{
    __shared__ TileLds lds;
    const int tid = threadIdx.x, tk = blockIdx.x, tn = blockIdx.y;
    const int64_t e = blockIdx.z;
    const int kb = gridDim.x, nb = gridDim.y;
    const int c = tk * kTile + 8 * (tid & 15), row = tn * kTile + 8 * (tid >> 4);
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (row + i < p.N) {
            load8<TYPE>(p.w, e * p.group + (row + i) * p.ld, c, p.K, v[i]);
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[i][u] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int u = 0; u < 8; ++u)
            m = max(m, magnitude(v[i][u]));
    m = wave_max(m);
    if ((tid & 63) == 0)
        lds.amax[0][tid >> 6] = m;
    __syncthreads();
    m = max(max(lds.amax[0][0], lds.amax[0][1]), max(lds.amax[0][2], lds.amax[0][3]));
    const BlockScale b = block_scale<F>(m);
    if (tid == 0) {
        p.s[(e * nb + tn) * kb + tk] = b.s;
        if (p.qt)
            p.st[(e * kb + tk) * nb + tn] = b.s;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (row + i < p.N)
            *reinterpret_cast<u32x2*>(p.q + ((e * p.N + row + i) * kb + tk) * kTile + 8 * (tid & 15)) =
                u32x2{block_codes<F>(b, v[i][0], v[i][1], v[i][2], v[i][3]),
                      block_codes<F>(b, v[i][4], v[i][5], v[i][6], v[i][7])};
    if (!p.qt)
        return;
#pragma unroll
    for (int u = 0; u < 8; ++u)
        flip<F>(v, b, u, lds.codes, 8 * (tid >> 4), tid);
    __syncthreads();
    const int64_t ld = (int64_t)nb * kTile;
    put_columns<256>(lds.codes, p.qt + (e * p.K + (int64_t)tk * kTile) * ld + (int64_t)tn * kTile, ld, p.K - tk * kTile,
                     tid);
}

// ----------------------------------------------------------------- launch --

template <int F, int TYPE>
static void quant_launch(const BlockQuantArgs& a, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.C + kTile - 1) / kTile), (unsigned)a.chunks + (a.qt && a.offsets ? 1 : 0));
    const bool vec = (a.half ? a.half : a.C) % 8 == 0;
    if (a.z && a.half && a.half % kTile == 0)
        hipLaunchKernelGGL((block_quant_pair_kernel<F, TYPE>), dim3(a.half / kTile, grid.y), dim3(512), 0, stream, a);
    else if (a.z && vec)
        hipLaunchKernelGGL((block_quant_kernel<F, TYPE, true, true>), grid, dim3(256), 0, stream, a);
    else if (a.z)
        hipLaunchKernelGGL((block_quant_kernel<F, TYPE, true, false>), grid, dim3(256), 0, stream, a);
    else if (vec)
        hipLaunchKernelGGL((block_quant_kernel<F, TYPE, false, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((block_quant_kernel<F, TYPE, false, false>), grid, dim3(256), 0, stream, a);
}

template <int F>
static hipError_t quant_launch(const BlockQuantArgs& a, hipStream_t stream)
{
    if (a.type == kBF16)
        quant_launch<F, kBF16>(a, stream);
    else if (a.type == kFP16)
        quant_launch<F, kFP16>(a, stream);
    else
        quant_launch<F, kFP32>(a, stream);
    return hipGetLastError();
}

hipError_t launch_block_quant(const BlockQuantArgs& a, hipStream_t stream)
{
    return a.fmt == kE5M2 ? quant_launch<kE5M2>(a, stream) : quant_launch<kE4M3>(a, stream);
}

template <int F>
static hipError_t square_launch(const SquareQuantArgs& a, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.K + kTile - 1) / kTile), (unsigned)((a.N + kTile - 1) / kTile), (unsigned)a.batch);
    if (a.type == kBF16)
        hipLaunchKernelGGL((square_quant_kernel<F, kBF16>), grid, dim3(256), 0, stream, a);
    else if (a.type == kFP16)
        hipLaunchKernelGGL((square_quant_kernel<F, kFP16>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((square_quant_kernel<F, kFP32>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_square_quant(const SquareQuantArgs& a, hipStream_t stream)
{
    return a.fmt == kE5M2 ? square_launch<kE5M2>(a, stream) : square_launch<kE4M3>(a, stream);
}

}  // namespace mxg
