// The MXFP8 product with a fused epilogue, dense and by expert, templated on
// the FP8 formats of its operands.  Each format pair is instantiated in its
// own translation unit.
#pragma once

#include "activation.h"
#include "element.h"
#include "gemm_impl.h"
#include "linear.h"
#include "quant.h"

namespace mxg {

// A wave-uniform pointer as a scalar (the copies' base register).
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p)
{
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint8_t*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

// ------------------------------------------------------------- work items --

// What a work-group computes: rows [m0, end) of the product (at most the
// tile's height), columns from column tile tn, of expert e; K-steps
// [k0, k0 + steps).  zero: rows that belong to no expert.
struct LinItem {
    int m0, end, tn, e, k0, steps;
    int ks;             // K split
    bool zero;
};

// The list of all experts' row tiles: expert e has ceil(rows of e / BM) of
// them, and the rows past the last expert come as one expert more.  A round
// takes 256 experts, four per lane (so up to 255 experts are one round of
// loads); the offsets are clamped to the rows there are.  All 64 lanes of the
// wave take part.
template <int BM>
struct RowTiles {
    int at[5], n[4], sum, inc;      // the lane's row ranges and tiles; tiles of the round up to it

    __device__ __forceinline__ void scan(const LinArgs& p, int g0, int lane)
    {
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const int g = g0 + 4 * lane + i;
            at[i] = g <= p.groups ? p.offsets[g] : p.rows;
        }
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const int lo = i ? at[i - 1] : 0;
            at[i] = at[i] < lo ? lo : at[i] > p.rows ? p.rows : at[i];
        }
        sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            n[i] = (at[i + 1] - at[i] + BM - 1) / BM;
            sum += n[i];
        }
        inc = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int x = __shfl_up(inc, d);
            inc += lane >= d ? x : 0;
        }
    }
    __device__ __forceinline__ int tiles() const { return __builtin_amdgcn_readlane(inc, 63); }
    // tile tm of this round's (0 <= tm < tiles())
    __device__ __forceinline__ void find(const LinArgs& p, int g0, int tm, int lane, LinItem& it) const
    {
        const int l = __builtin_ctzll(__ballot(inc > tm));
        int first = inc - sum, lo = at[0], hi = at[1], e = g0 + 4 * lane;
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (tm >= first + n[i - 1] && e == g0 + 4 * lane + i - 1) {
                first += n[i - 1];
                lo = at[i];
                hi = at[i + 1];
                ++e;
            }
        it.e = __builtin_amdgcn_readfirstlane(__shfl(e, l));
        it.m0 = __builtin_amdgcn_readfirstlane(__shfl(lo + (tm - first) * BM, l));
        it.end = __builtin_amdgcn_readfirstlane(__shfl(hi, l));
        it.zero = it.e == p.groups;
    }
};

// By rows, the grid is the most tiles there could be; the ones there are go
// to the XCDs in equal, contiguous shares (shares of the grid would leave
// whole XCDs without work: 1.2 times the time at 32 experts of about 512
// rows).  False where this work-group has none.
template <int BM>
__device__ __forceinline__ bool lin_item_rows(const LinArgs& p, int lane, LinItem& it)
{
    RowTiles<BM> round;
    round.scan(p, 0, lane);
    int tiles = round.tiles();
    for (int g0 = 256; g0 <= p.groups; g0 += 256) {
        RowTiles<BM> more;
        more.scan(p, g0, lane);
        tiles += more.tiles();
    }
    const int work = tiles * p.tiles_n;
    const int x = blockIdx.x % kNumXcd, i = blockIdx.x / kNumXcd;
    const int share = work / kNumXcd, extra = work % kNumXcd;
    if (i >= share + (x < extra ? 1 : 0))
        return false;
    const TileCoord tc = decode_work(x * share + (x < extra ? x : extra) + i, tiles, p.tiles_n, 1, p.group_n);
    it.tn = tc.tn;
    it.ks = 0;
    int tm = tc.tm, g0 = 0;
    while (tm >= round.tiles()) {       // past the first 256 experts
        tm -= round.tiles();
        g0 += 256;
        round.scan(p, g0, lane);
    }
    round.find(p, g0, tm, lane, it);
    return true;
}

template <int BM>
__device__ __forceinline__ bool lin_item(const LinArgs& p, int lane, LinItem& it)
{
    it.k0 = 0;
    it.steps = p.K / kBK;
    it.zero = false;
    it.e = 0;
    it.end = p.rows;
    if (p.mode == kByRows)
        return lin_item_rows<BM>(p, lane, it);
    int w = remap_block(blockIdx.x, gridDim.x);
    if (p.mode == kByInner) {
        // Each XCD has an equal share of the tiles, of every expert: their
        // inner ranges differ, so whole experts would be unequal shares.
        // Within it expert after expert, whose operands it then shares.
        const int tiles = p.tiles_m * p.tiles_n, share = (tiles + kNumXcd - 1) / kNumXcd;
        const int x = blockIdx.x % kNumXcd, i = blockIdx.x / kNumXcd;
        it.e = i / share;
        w = x * share + i % share;
        if (w >= tiles || it.e >= p.groups)
            return false;
        int lo = p.offsets[it.e], hi = p.offsets[it.e + 1];
        lo = lo < 0 ? 0 : lo > p.K ? p.K : lo;
        hi = hi < lo ? lo : hi > p.K ? p.K : hi;
        it.k0 = lo / kBK;
        it.steps = hi / kBK - it.k0;
    }
    const TileCoord tc = decode_work(w, p.tiles_m, p.tiles_n, p.split, p.group_n);
    it.tn = tc.tn;
    it.m0 = tc.tm * BM;
    it.ks = tc.ks;
    if (p.split > 1) {      // K-steps in even runs, the first ones a step longer
        const int share = it.steps / p.split, more = it.steps % p.split;
        it.k0 = tc.ks * share + (tc.ks < more ? tc.ks : more);
        it.steps = share + (tc.ks < more ? 1 : 0);
    }
    return true;
}

// ---------------------------------------------------------------- epilogue --

// The bits of eight consecutive columns [c, c + 8) of a 16- or 32-bit row of
// n, as loaded.  Loading early and converting late keeps the loads' latency
// out of the way.  Columns past the row give some of its own elements (never
// used): no lane branches, and every access is inside the row.
struct Raw8 {
    u32x4 v[2];
};

__device__ __forceinline__ Raw8 raw8(int type, const void* base, int64_t at, int c, int n)
{
    Raw8 r;
    r.v[0] = r.v[1] = u32x4{0, 0, 0, 0};
    if ((n & 7) == 0) {
        const int64_t i = at + (c < n ? c : n - 8);
        if (type == kFP32) {
            __builtin_memcpy(&r.v[0], static_cast<const float*>(base) + i, 16);
            __builtin_memcpy(&r.v[1], static_cast<const float*>(base) + i + 4, 16);
        } else {
            __builtin_memcpy(&r.v[0], static_cast<const uint16_t*>(base) + i, 16);
        }
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t i = at + (c + u < n ? c + u : n - 1);
            if (type == kFP32)
                r.v[u >> 2][u & 3] = __float_as_uint(static_cast<const float*>(base)[i]);
            else
                r.v[0][u >> 1] |= (uint32_t)static_cast<const uint16_t*>(base)[i] << (16 * (u & 1));
        }
    }
    return r;
}

template <int TYPE, int N>
__device__ __forceinline__ void add_raw(const Raw8 (&r)[N], float (&v)[8 * N])
{
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t w = r[k].v[0][u >> 1];
            if constexpr (TYPE == kFP32)
                v[8 * k + u] += __uint_as_float(r[k].v[u >> 2][u & 3]);
            else if constexpr (TYPE == kFP16)
                v[8 * k + u] += Element<kFP16>::get((uint16_t)(w >> (16 * (u & 1))));
            else
                v[8 * k + u] += __uint_as_float(u & 1 ? w & 0xFFFF0000u : w << 16);
        }
}

template <int N>
__device__ __forceinline__ void add_raw(int type, const Raw8 (&r)[N], float (&v)[8 * N])
{
    if (type == kBF16)
        add_raw<kBF16>(r, v);
    else if (type == kFP16)
        add_raw<kFP16>(r, v);
    else
        add_raw<kFP32>(r, v);
}

// Bias of columns [c, c + 8) of `cols` (gated: of both halves), as FP32.
template <bool GATED>
struct Bias8 {
    float v[GATED ? 2 : 1][8];
    __device__ __forceinline__ void load(const LinArgs& p, int e, int c, int cols)
    {
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[h][u] = 0.f;
            if (p.bias) {
                const Raw8 r[1] = {raw8(p.bias_type, p.bias, (int64_t)e * p.N + h * cols, c, cols)};
                add_raw(p.bias_type, r, v[h]);
            }
        }
    }
};

__device__ __forceinline__ int residual_type(const LinArgs& p) { return p.out_type > kFP32 ? kBF16 : p.out_type; }

// Residual of row `row` (or of the last row `end` - 1), columns [c, c + 8).
__device__ __forceinline__ Raw8 residual8(const LinArgs& p, int row, int end, int c, int cols)
{
    Raw8 r;
    r.v[0] = r.v[1] = u32x4{0, 0, 0, 0};
    if (p.residual)
        r = raw8(residual_type(p), p.residual, (row < end ? row : end - 1) * p.ld_res, c, cols);
    return r;
}

// Eight consecutive elements from v[FIRST] to columns [c, c + 8) of the row
// of n at p, those past n dropped.
template <int TYPE, int FIRST, int N>
__device__ __forceinline__ void put8(typename Element<TYPE>::T* p, int c, int n, const float (&v)[N])
{
    constexpr int kWords = TYPE == kFP32 ? 8 : 4;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if constexpr (TYPE == kFP32)
            w[i] = __float_as_uint(v[FIRST + i]);
        else if constexpr (TYPE == kBF16)
            w[i] = pack_bf16x2(v[FIRST + 2 * i], v[FIRST + 2 * i + 1]);
        else
            w[i] = Element<TYPE>::put(v[FIRST + 2 * i]) | (uint32_t)Element<TYPE>::put(v[FIRST + 2 * i + 1]) << 16;
    }
    if ((n & 7) == 0) {         // the first column exists, so all eight do
        __builtin_memcpy(p, w, sizeof(w));
        return;
    }
    // one element at a time, moved down from the next: small, not fast
#pragma unroll 1
    for (int u = 0; u < 8 && c + u < n; ++u) {
        if constexpr (TYPE == kFP32)
            p[u] = __uint_as_float(w[0]);
        else
            p[u] = (uint16_t)w[0];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint32_t next = i + 1 < kWords ? w[i + 1] : 0;
            w[i] = TYPE == kFP32 ? next : (w[i] >> 16) | (next << 16);
        }
    }
}

// f(LO), .., f(HI - 1) with constant arguments.
template <int LO, int HI, class F>
__device__ __forceinline__ void static_for(const F& f)
{
    if constexpr (LO < HI) {
        f(std::integral_constant<int, LO>());
        static_for<LO + 1, HI>(f);
    }
}

// Columns [c, c + 8) of N rows, `first`, first + STEP, ..: row k is stored
// where bit k of `ok` is set.
template <int TYPE, int N, int STEP>
__device__ __forceinline__ void put_rows(void* base, int64_t ld, int first, int c, int cols, uint32_t ok,
                                         const float (&v)[8 * N])
{
    typename Element<TYPE>::T* p = static_cast<typename Element<TYPE>::T*>(base) + first * ld + c;
    static_for<0, N>([&](auto kc) __attribute__((always_inline)) {
        constexpr int k = decltype(kc)::value;
        if (ok >> k & 1)
            put8<TYPE, 8 * k>(p + k * STEP * ld, c, cols, v);
        __builtin_amdgcn_sched_barrier(0);
    });
}

template <int FMT, int N, int STEP>
__device__ __forceinline__ void put_mx(const LinArgs& p, int first, int c, uint32_t ok, const float (&v)[8 * N],
                                       int lane)
{
    static_for<0, N>([&](auto kc) __attribute__((always_inline)) {
        constexpr int k = decltype(kc)::value;
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            m = max(m, __float_as_uint(v[8 * k + u]) & 0x7FFFFFFFu);
        const MxScale s = mx_scale<FMT>(quad_max(m));
        const int64_t row = first + k * STEP;
        if (ok >> k & 1) {      // whole blocks are in or out
            *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(p.out) + row * p.ld_out + c) =
                u32x2{mx_codes<FMT>(s, v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3]),
                      mx_codes<FMT>(s, v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7])};
            if ((lane & 3) == 0)
                p.out_s[row * p.ld_out_s + (c >> 5)] = s.byte;
        }
        __builtin_amdgcn_sched_barrier(0);
    });
}

// Columns [c, c + 8) of `cols` of N rows of the output, `first`, first +
// STEP, .., from z (and, gated, the up half's z1).  Everything is FP32 until
// the one rounding of the store (the bfloat16 copy of z, kept for the
// gradient, is rounded by itself).  With MXFP8 output four consecutive lanes
// hold one block of 32; every lane of the wave calls, and bit k of `ok` says
// whether row k and the first column exist.  Each step is one branch for all
// the values: with one wave per SIMD the epilogue is bound by instructions.
template <bool GATED, int N, int STEP>
__device__ __forceinline__ void finish(const LinArgs& p, int e, int first, int c, int cols, uint32_t ok,
                                       float (&z)[8 * N], float (&z1)[GATED ? 8 * N : 1], const Bias8<GATED>& bias,
                                       const Raw8 (&residual)[N], int lane)
{
    if (p.bias) {
#pragma unroll
        for (int u = 0; u < 8 * N; ++u) {
            z[u] += bias.v[0][u & 7];
            if constexpr (GATED)
                z1[u] += bias.v[1][u & 7];
        }
    }
    if (p.z) {
        put_rows<kBF16, N, STEP>(p.z, p.ld_z, first, c, cols, ok, z);
        if constexpr (GATED)
            put_rows<kBF16, N, STEP>(p.z + cols, p.ld_z, first, c, cols, ok, z1);
    }
    activate(p.act, z);
    if constexpr (GATED) {
#pragma unroll
        for (int u = 0; u < 8 * N; ++u)
            z[u] *= z1[u];
    }
    if (p.residual)
        add_raw(residual_type(p), residual, z);
    void* out = p.out;
    if (p.mode == kByInner)
        out = static_cast<char*>(out) + e * p.out_group * (p.out_type == kFP32 ? 4 : 2);
    if (p.out_type == kBF16)
        put_rows<kBF16, N, STEP>(out, p.ld_out, first, c, cols, ok, z);
    else if (p.out_type == kFP16)
        put_rows<kFP16, N, STEP>(out, p.ld_out, first, c, cols, ok, z);
    else if (p.out_type == kFP32)
        put_rows<kFP32, N, STEP>(out, p.ld_out, first, c, cols, ok, z);
    else if (p.out_type == kMxE4M3)
        put_mx<kE4M3, N, STEP>(p, first, c, ok, z, lane);
    else
        put_mx<kE5M2, N, STEP>(p, first, c, ok, z, lane);
}

// Zero rows [m0, end) of the tile's columns (rows of no expert).
template <int BM, int BN>
__device__ __forceinline__ void zero_rows(const LinArgs& p, const LinItem& it)
{
    const int cols = p.gated ? p.N / 2 : p.N;
    const int width = p.gated ? BN / 2 : BN;
    const int end = it.end - it.m0 < BM ? it.end : it.m0 + BM;
    for (int i = threadIdx.x; i < (end - it.m0) * width; i += blockDim.x) {
        const int row = it.m0 + i / width, c = it.tn * width + i % width;
        if (c >= cols)
            continue;
        const int64_t at = row * p.ld_out + c;
        if (p.out_type >= kMxE4M3) {
            static_cast<uint8_t*>(p.out)[at] = 0;
            if (c % 32 == 0)
                p.out_s[row * p.ld_out_s + c / 32] = 0;
        } else if (p.out_type == kFP32) {
            static_cast<float*>(p.out)[at] = 0.f;
        } else {
            static_cast<uint16_t*>(p.out)[at] = 0;
        }
        if (p.z) {
            p.z[row * p.ld_z + c] = 0;
            if (p.gated)
                p.z[row * p.ld_z + cols + c] = 0;
        }
    }
}

// A slab of 32 rows x 64 columns of the product in LDS, FP32: row r holds
// its sixteen 16-byte chunks XOR-swizzled by r, so neither the accumulators'
// writes (32 rows, one chunk) nor the row-wise reads pile onto a few banks.
constexpr int kSlabBytes = 32 * 64 * 4;

__device__ __forceinline__ int slab_at(int r, int chunk) { return r * 256 + ((chunk ^ (r & 15)) * 16); }

template <int GB>
__device__ __forceinline__ void slab_write(uint8_t* buf, const v16f (&acc)[GB], int g0, int lane)
{
    const int lr = lane & 31, lq = lane >> 5;
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const v16f& a = acc[g0 + g];
            *reinterpret_cast<v4f*>(buf + slab_at(lr, 8 * g + 2 * q + lq)) =
                v4f{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
        }
}

// Columns [8 c, 8 c + 8) of row r, summed over COPIES slabs in order.
template <int COPIES, int FIRST, int N>
__device__ __forceinline__ void slab_read8(const uint8_t* buf, int r, int c, float (&v)[N])
{
    v4f x[COPIES][2];
#pragma unroll
    for (int k = 0; k < COPIES; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            x[k][h] = *reinterpret_cast<const v4f*>(buf + k * kSlabBytes + slab_at(r, 2 * c + h));
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        v[FIRST + u] = x[0][u >> 2][u & 3];
#pragma unroll
        for (int k = 1; k < COPIES; ++k)
            v[FIRST + u] += x[k][u >> 2][u & 3];
    }
}

// Rows of a slab as a wave finishes them: eight lanes per row (gated: four, the
// tile holding gate and up columns in alternating blocks of 32).
template <bool GATED>
struct SlabRows {
    static constexpr int kPer = GATED ? 4 : 8;          // lanes per row
    static constexpr int kStep = 64 / kPer;             // rows per pass
    // first output column of the lane in a slab whose first product column is col0
    __device__ static __forceinline__ int column(int col0, int lane)
    {
        return (GATED ? col0 / 2 : col0) + 8 * (lane % kPer);
    }
};

// The slab's rows [r0, r0 + rows), at most PASSES kStep of them, from
// product row row0 + r0 on.
template <bool GATED, int PASSES, int COPIES>
__device__ __forceinline__ void finish_rows(const LinArgs& p, const uint8_t* buf, const Bias8<GATED>& bias,
                                            const Raw8 (&res)[PASSES], int row0, int end, int col0, int cols, int e,
                                            int r0, int rows, int lane)
{
    typedef SlabRows<GATED> S;
    float z[8 * PASSES], z1[GATED ? 8 * PASSES : 1];
    const int c = S::column(col0, lane), first = r0 + lane / S::kPer;
    uint32_t ok = 0;
    static_for<0, PASSES>([&](auto kc) __attribute__((always_inline)) {
        constexpr int k = decltype(kc)::value;
        const int r = first + k * S::kStep, rr = r < r0 + rows ? r : r0;
        slab_read8<COPIES, 8 * k>(buf, rr, lane % S::kPer, z);
        if constexpr (GATED)
            slab_read8<COPIES, 8 * k>(buf, rr, 4 + lane % S::kPer, z1);
        ok |= r < r0 + rows && row0 + r < end && c < cols ? 1u << k : 0;
    });
    finish<GATED, PASSES, S::kStep>(p, e, row0 + first, c, cols, ok, z, z1, bias, res, lane);
}

// ------------------------------------------------------------------ copies --

// Column `c` of a tile -> row of w, relative to the tile's first one.  Gated:
// blocks of 32 columns alternate between the halves.  Columns past the edge
// give the last row there is; their results are not stored.
__device__ __forceinline__ int64_t lin_wrow(const LinArgs& p, int n0, int c)
{
    if (!p.gated)
        return n0 + c < p.N ? c : p.N - 1 - n0;
    const int half = p.N / 2, o = (c >> 6) * 32 + (c & 31);
    const int col = n0 / 2 + o < half ? o : half - 1 - n0 / 2;
    return ((c >> 5) & 1) ? (int64_t)half + col : col;
}

// As copy_offsets, for rows at a plain stride: offsets are relative to rows
// m0 of a and (gated: half of) n0 of w.
template <int BM, int BN, int NW>
__device__ __forceinline__ void lin_copy_offsets(const LinArgs& p, int m0, int end, int n0, int wave, int lane,
                                                 CopyOffsets<BM, BN, NW, 32>& o)
{
    typedef StageGeom<BM, BN, NW> G;
    const int last = end - 1 - m0;
#pragma unroll
    for (int j = 0; j < G::JA; ++j) {
        const int t = wave + j * NW;
        const int row = 8 * (t < G::IA ? t : G::IA - 1) + (lane >> 3);
        o.a[j] = (uint32_t)((row < last ? row : last) * (uint32_t)p.lda) + swz_t<32>(row, lane & 7) * 16;
    }
#pragma unroll
    for (int j = 0; j < G::JB; ++j) {
        const int t = wave + j * NW;
        const int row = 8 * (t < G::IB ? t : G::IB - 1) + (lane >> 3);
        o.b[j] = (uint32_t)(lin_wrow(p, n0, row) * p.ldw) + swz_t<32>(row, lane & 7) * 16;
    }
#pragma unroll
    for (int j = 0; j < G::KSA; ++j) {
        const int t = wave + j * NW;
        int row = 64 * (t < G::ISA ? t : G::ISA - 1) + lane;
        row = row < BM ? row : BM - 1;
        o.as[j] = (uint32_t)((row < last ? row : last) * (uint32_t)p.ldas);
    }
#pragma unroll
    for (int j = 0; j < G::KSB; ++j) {
        const int t = wave + j * NW;
        int row = 64 * (t < G::ISB ? t : G::ISB - 1) + lane;
        row = row < BN ? row : BN - 1;
        o.bs[j] = (uint32_t)(lin_wrow(p, n0, row) * p.ldws);
    }
}

// ------------------------------------------------------- native K loop ------

// LDS of the native loop: two stages of one K-step (rows of 128 bytes, A then
// B), then two slots of scale words, sixteen bytes per row: the words of four
// K-steps, copied at once.  (One copy of four bytes per row and K-step made a
// third of all L2 requests, which bound the 256 x 256 tile; so did stages of
// 64 K, whose copies ask the L2 for 64 bytes at a time and not for a line.)
template <int BM, int BN, int NW>
struct PairGeom {
    static constexpr int A_BYTES = BM * kBK, STAGE = (BM + BN) * kBK;
    static constexpr int SCALES = 16 * (BM + BN);
    static constexpr int BYTES = 2 * STAGE + 2 * SCALES + 1024;             // and 1 KB nobody reads
    static constexpr int JA = BM / 8 / NW, JB = BN / 8 / NW;                // 1 KB copies per wave and stage
    static constexpr int IS = (BM + BN) / 64, JS = (IS + NW - 1) / NW;      // 1 KB copies of scale words
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0,
                  "every wave copies as much as any other");
};

// A wave's copies: source offsets relative to rows m0 of a and (gated: half
// of) n0 of w.  A scale copy takes 64 of the tile's A rows followed by its B
// rows.
template <int BM, int BN, int NW>
struct PairCopies {
    typedef PairGeom<BM, BN, NW> G;
    uint32_t a[G::JA], b[G::JB], s[G::JS];

    __device__ __forceinline__ void init(const LinArgs& p, int m0, int end, int n0, int wave, int lane)
    {
        const int last = end - 1 - m0;
#pragma unroll
        for (int j = 0; j < G::JA; ++j) {
            const int row = 8 * (wave + j * NW) + (lane >> 3);
            a[j] = (uint32_t)((row < last ? row : last) * (uint32_t)p.lda) + swz_t<32>(row, lane & 7) * 16;
        }
#pragma unroll
        for (int j = 0; j < G::JB; ++j) {
            const int row = 8 * (wave + j * NW) + (lane >> 3);
            b[j] = (uint32_t)(lin_wrow(p, n0, row) * p.ldw) + swz_t<32>(row, lane & 7) * 16;
        }
#pragma unroll
        for (int j = 0; j < G::JS; ++j)
            s[j] = scale_row(p, last, n0, 64 * piece(wave, j) + lane);
    }
    // a wave with no scale piece left repeats the last one
    __device__ static __forceinline__ int piece(int wave, int j)
    {
        return wave + j * NW < G::IS ? wave + j * NW : G::IS - 1;
    }
    __device__ static __forceinline__ uint32_t scale_row(const LinArgs& p, int last, int n0, int row)
    {
        return row < BM ? (uint32_t)((row < last ? row : last) * (uint32_t)p.ldas)
                        : (uint32_t)(lin_wrow(p, n0, row - BM) * p.ldws);
    }
    // copy t of a stage's codes
    __device__ __forceinline__ void issue(const StepSrc& src, uint8_t* stage, int wave, int t) const
    {
#pragma unroll
        for (int j = 0; j < G::JA; ++j)
            if (t == j)
                dma16_at(uniform(src.a), a[j], stage + (wave + j * NW) * 1024);
#pragma unroll
        for (int j = 0; j < G::JB; ++j)
            if (t == G::JA + j)
                dma16_at(uniform(src.b), b[j], stage + G::A_BYTES + (wave + j * NW) * 1024);
    }
    // scale copy j: sixteen bytes of every row, from src; with `rows` zero,
    // the first row's sixty-four times over (one request), to `idle`
    __device__ __forceinline__ void issue_scales(const StepSrc& src, uint8_t* slot, uint8_t* idle, uint32_t rows,
                                                 int wave, int j) const
    {
        const int k = piece(wave, j);
        dma16_at(uniform(64 * k < BM ? src.as : src.bs), s[j] & rows, rows ? slot + k * 1024 : idle);
    }
    // the same where rows hold fewer than sixteen: `words` words of four
    // bytes, the last repeated
    __device__ static __forceinline__ void issue_short_scales(const LinArgs& p, const StepSrc& src, int words,
                                                              uint8_t* slot, int m0, int end, int n0, int wave,
                                                              int lane)
    {
        const int word = (lane & 3) < words ? lane & 3 : words - 1;
        for (int k = wave; k < (BM + BN) / 16; k += NW)
            dma4_at(uniform(16 * k < BM ? src.as : src.bs),
                    scale_row(p, end - 1 - m0, n0, 16 * k + (lane >> 2)) + 4 * word, slot + k * 256);
    }
};

template <int I, class T>
__device__ __forceinline__ T& pick(T& a, T& b)
{
    if constexpr (I == 0)
        return a;
    else
        return b;
}

// Task i where c tasks 0 .. c - 1 and r tasks c .. c + r - 1 take turns.
constexpr int take_turns(int i, int c, int r)
{
    const int both = 2 * (c < r ? c : r);
    return i < both ? (i & 1 ? c + i / 2 : i / 2) : c < r ? i : i - r;
}

// K loop on the scaled FP8 MFMA (32 x 32 x 64), software-pipelined.  A
// K-step (128 K) is two sub-steps m of 64 K.  While the GA x GB MFMAs of a
// sub-step run, the fragments of the next one are read from LDS into the
// other register set, so no MFMA waits for a read.  The one barrier of a
// K-step comes three quarters through sub-step 0: by then step s + 1 has
// landed and every wave holds all of step s in registers, so the copies of
// step s + 2 are issued into its stage at once and have a whole K-step to
// land.  (8192 x 8192 x 8192: 466 us; with the barrier between the sub-steps
// 474, and there with all copies before the fragments' reads 486.)  Large wave tiles
// keep the LDS reads per MFMA low: a 128 x 128 wave tile reads each byte for
// 128 outputs, and four of them read 128 KB per 256 x 256 x 128 step (1024
// clocks at 128 bytes per clock, plus 512 for the copies' writes, against
// 2048 clocks of MFMA), where eight waves of 128 x 64 read 192 KB.
// In all 2.36 PFLOP/s, at 2.2 GHz; the MFMAs alone would take 240 us there.
// Scale bytes: a lane reads the four of its row as one word, shifted so that
// byte 2 m is its block's in sub-step m.
// src: sources of the loop's first K-step, of `valid` ones; nsteps: the
// barriers to meet (valid or one more).  scale_bytes: bytes of a row's scales
// from src on (at least 4 valid), short_rows: whole rows have fewer than 16.
template <int BM, int BN, int WGM, int WGN, int WGK, int FA, int FB>
__device__ __forceinline__ void native_mainloop(const LinArgs& p, uint8_t* stages,
                                                const PairCopies<BM, BN, WGM * WGN>& co, const StepSrc& src,
                                                int nsteps, int valid, int scale_bytes, bool short_rows, int m0,
                                                int end, int n0, int wl, int lane,
                                                v16f (&acc)[BM / WGM / 32][BN / WGN / 32])
{
    constexpr int MW = 32;
    typedef PairGeom<BM, BN, WGM * WGN> G;
    constexpr int TM = BM / WGM, TN = BN / WGN;
    constexpr int GA = TM / MW, GB = TN / MW;
    constexpr int NF = GA + GB;
    constexpr int NU = GA * GB;                    // MFMAs of a sub-step
    constexpr int NC = G::JA + G::JB;
    const int wm = wl / WGN, wn = wl % WGN;
    const int lr = lane & 31, lq = lane >> 5;
    uint8_t* const scales = stages + 2 * G::STAGE;

    const int a_row = (wm * TM + lr) * kBK, b_row = G::A_BYTES + (wn * TN + lr) * kBK;
    auto frag_off = [&](int f) { return f < GA ? a_row + f * MW * kBK : b_row + (f - GA) * MW * kBK; };
    auto scale_off = [&](int f) { return 16 * (f < GA ? wm * TM + f * MW + lr : BM + wn * TN + (f - GA) * MW + lr); };
    auto chunk_off = [&](int m, int h) { return swz_t<MW>(lr, 4 * m + 2 * h + lq) * 16; };

    const int last = valid > 0 ? valid - 1 : 0;
    auto src_at = [&](int s) {
        const int64_t k = s < last ? s : last;      // past the end: the last K-step again
        return StepSrc{src.a + k * kBK, src.b + k * kBK, nullptr, nullptr};
    };
    // the scale words of K-steps 4 g .. 4 g + 3: from where they start, or
    // from sixteen bytes before the rows end
    auto scale_at = [&](int g) { return 16 * g + 16 <= scale_bytes ? 16 * g : scale_bytes - 16; };
    auto scale_src = [&](int g) { return StepSrc{nullptr, nullptr, src.as + scale_at(g), src.bs + scale_at(g)}; };
    // place of K-step s's words
    auto scale_slot = [&](int s) {
        const int g = s >> 2;
        return scales + (g & 1) * G::SCALES + (short_rows ? 4 * s : 4 * s - scale_at(g));
    };

    u32x4 fr0[NF][2], fr1[NF][2];  // fragments of sub-steps 0 and 1
    uint32_t sw[NF];               // scale words of the current K-step
    auto operand = [](const u32x4(&fr)[2]) __attribute__((always_inline)) {
        const u32x4 lo = fr[0], hi = fr[1];
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };

    if (short_rows)
        co.issue_short_scales(p, src, last + 1, scales, m0, end, n0, wl, lane);
    else
#pragma unroll
        for (int j = 0; j < G::JS; ++j)
            co.issue_scales(scale_src(0), scales, nullptr, ~0u, wl, j);
#pragma unroll
    for (int t = 0; t < NC; ++t)
        co.issue(src_at(0), stages, wl, t);
#pragma unroll
    for (int t = 0; t < NC; ++t)
        co.issue(src_at(1), stages + G::STAGE, wl, t);
    wait_copies<NC>();
    __syncthreads();
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        sw[f] = *reinterpret_cast<const uint32_t*>(scale_slot(0) + scale_off(f)) >> (8 * lq);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            fr0[f][h] = *reinterpret_cast<const u32x4*>(stages + frag_off(f) + chunk_off(0, h));
    }
    // One K-step per iteration: with two unrolled and one left over, the
    // compiler spilled 192 registers of the 256 x 256 tile.
    for (int s = 0; s < nsteps; ++s) {
        if (WGK > 1 && s >= valid) {        // a group without this step meets the barrier
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            continue;
        }
        uint8_t* const cur = stages + (s & 1) * G::STAGE;
        const uint8_t* const nxt = stages + (~s & 1) * G::STAGE;
        const StepSrc src2 = src_at(s + 2);
        const uint8_t* const next_scales = scale_slot(s < last ? s + 1 : last);
        // every fourth step copies the next four's scale words.  (The others
        // go through the same copies idly: a branch here let the compiler
        // move sub-step 0's MFMAs behind the barrier.)
        const bool more = (s & 3) == 0 && s + 4 < valid;
        const int group = more ? (s >> 2) + 1 : 0;
        const StepSrc ssrc = short_rows ? StepSrc{nullptr, nullptr, src.a, src.b} : scale_src(group);
        uint8_t* const next_slot = scales + (group & 1) * G::SCALES;
        uint32_t swn[NF];
        static_for<0, 2>([&](auto mc) __attribute__((always_inline)) {
            constexpr int m = decltype(mc)::value;
            const uint8_t* from = m == 0 ? cur : nxt;
            auto& now = pick<m>(fr0, fr1);
            auto& then = pick<1 - m>(fr0, fr1);
            // Beside the MFMAs.  m = 0: the fragments of sub-step 1 and the
            // next K-step's scale words in the first half, so that the
            // barrier's wait for them is short; after the barrier the first
            // copies of step s + 2.  m = 1: the other copies and the
            // next K-step's fragments in turns (the load unit takes about one
            // copy of each wave per MFMA, and fragments read last would be
            // waited for).
            constexpr int kEarly = NU / 4;      // MFMAs, and copies, of sub-step 0 after the barrier
            constexpr int ncopy = m == 1 ? NC - kEarly : 0, nscale = m == 1 ? G::JS : 0;
            constexpr int reads = ncopy + nscale, words = reads + 2 * NF;
            constexpr int ntask = words + (m == 0 ? NF : 0), over = m == 0 ? NU / 2 : NU;
            static_for<0, NU>([&](auto uc) __attribute__((always_inline)) {
                constexpr int u = decltype(uc)::value, i = u / GB, g = u % GB;
                if constexpr (m == 0 && u == NU - kEarly) {
                    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    __syncthreads();
                }
                acc[i][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    operand(now[GA + g]), operand(now[i]), acc[i][g], FB, FA, 2 * m, (int)sw[GA + g], 2 * m, (int)sw[i]);
                constexpr int t0 = u < over ? u * ntask / over : ntask, t1 = u < over ? (u + 1) * ntask / over : ntask;
                if constexpr (m == 0 && u >= NU - kEarly)
                    co.issue(src2, cur, wl, u - (NU - kEarly));
                static_for<t0, t1>([&](auto tc) __attribute__((always_inline)) {
                    constexpr int i0 = decltype(tc)::value;
                    constexpr int t = m == 0 ? i0 : take_turns(i0, reads, 2 * NF);
                    if constexpr (t < ncopy) {
                        co.issue(src2, cur, wl, t + kEarly);
                    } else if constexpr (t < reads) {
                        co.issue_scales(ssrc, next_slot, scales + 2 * G::SCALES, more ? ~0u : 0u, wl, t - ncopy);
                    } else if constexpr (t < words) {
                        // first the B fragments, which every row of MFMAs uses
                        constexpr int r = t - reads, f = (r / 2 + GA) % NF, h = r & 1;
                        then[f][h] = *reinterpret_cast<const u32x4*>(from + frag_off(f) + chunk_off(m ^ 1, h));
                    } else {
                        constexpr int f = t - words;
                        swn[f] = *reinterpret_cast<const uint32_t*>(next_scales + scale_off(f));
                    }
                });
                __builtin_amdgcn_sched_barrier(0);
            });
        });
#pragma unroll
        for (int f = 0; f < NF; ++f)
            sw[f] = swn[f] >> (8 * lq);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy outlives the work-group
}

// ------------------------------------------------------------ tile kernel ---

// How a tile's epilogue has its residual.  Loads and stores share one counter,
// so a load waited for between two slabs waits for the slab before to be
// written; a 16-bit residual of aligned rows is therefore copied to LDS whole
// before the first store.  Others are loaded slab by slab.
enum { kNoResidual, kLdsResidual, kDirectResidual };

__device__ __forceinline__ int residual_path(const LinArgs& p)
{
    if (!p.residual)
        return kNoResidual;
    const int cols = p.gated ? p.N / 2 : p.N;
    return p.out_type != kFP32 && (cols & 7) == 0 && (p.ld_res & 7) == 0 && p.ld_res < (1 << 22) &&
                   (reinterpret_cast<uintptr_t>(p.residual) & 15) == 0
               ? kLdsResidual
               : kDirectResidual;
}

// The wave's accumulators (rows from row0, product columns from col0) through
// LDS and the epilogue, one slab at a time.  `mem`: the wave's LDS, a slab and
// (kLdsResidual) the wave tile's residual, 32 GA rows of kResRow bytes.
template <bool GATED, int RES, int GA, int GB>
__device__ __forceinline__ void tile_epilogue(const LinArgs& p, uint8_t* mem, v16f (&acc)[GA][GB], const LinItem& it,
                                              int row0, int col0, int cols, int lane)
{
    typedef SlabRows<GATED> S;
    constexpr int kSlabs = GA * GB / 2;
    constexpr int kOuts = GATED ? GB * 16 : GB * 32;    // output columns of the wave tile
    constexpr int kResRow = kOuts * 2;
    uint8_t* const res_lds = mem + kSlabBytes;
    if constexpr (RES == kLdsResidual) {
        constexpr int kPieces = kResRow / 16, kRowsPer = 64 / kPieces;      // 1 KB copies of whole rows
        const int c = (GATED ? col0 / 2 : col0) + 8 * (lane % kPieces);
        const int cc = c < cols ? c : cols - 8;
        const int top = row0 < it.end ? row0 : it.end - 1;
        const uint8_t* base = uniform(static_cast<const uint8_t*>(p.residual) + top * p.ld_res * 2);
#pragma unroll
        for (int i = 0; i < 32 * GA / kRowsPer; ++i) {
            const int row = i * kRowsPer + lane / kPieces, last = it.end - 1 - top;
            dma16_at(base, ((row < last ? row : last) * (uint32_t)p.ld_res + cc) * 2, res_lds + i * 1024);
        }
    }
    Bias8<GATED> bias[GB / 2];
#pragma unroll
    for (int g = 0; g < GB / 2; ++g)
        bias[g].load(p, it.e, S::column(col0 + 64 * g, lane), cols);
    if constexpr (RES == kLdsResidual)
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    // one copy of the finishing code: only the slab's accumulators and bias
    // are picked by its number
#pragma unroll 1
    for (int t = 0; t < kSlabs; ++t) {
        Bias8<GATED> b = bias[0];
#pragma unroll
        for (int n = 0; n < kSlabs; ++n)
            if (t == n) {
                slab_write<GB>(mem, acc[n % GA], n / GA * 2, lane);
                b = bias[n / GA];
            }
        const int r0 = 32 * (t % GA), slab_col = col0 + 64 * (t / GA);
        // LDS operations of one wave complete in order, and the wave reads
        // back only what it wrote itself
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
        for (int r = 0; r < 32; r += 2 * S::kStep) {
            Raw8 res[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int rr = r0 + r + k * S::kStep + lane / S::kPer;
                if constexpr (RES == kLdsResidual)
                    res[k].v[0] = *reinterpret_cast<const u32x4*>(res_lds + rr * kResRow + (t / GA) * (kOuts * 4 / GB) +
                                                                  16 * (lane % S::kPer));
                else if constexpr (RES == kDirectResidual)
                    res[k] = residual8(p, row0 + rr, it.end, S::column(slab_col, lane), cols);
            }
            finish_rows<GATED, 2, 1>(p, mem, b, res, row0 + r0, it.end, slab_col, cols, it.e, r, 2 * S::kStep, lane);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// Several K groups of one wave each share a 64 x 64 block: every group leaves
// its sums, and each wave adds up and finishes its share of the rows.
template <bool GATED, int WGK>
__device__ __forceinline__ void groups_epilogue(const LinArgs& p, uint8_t* lds, v16f (&acc)[2][2], const LinItem& it,
                                                int col0, int cols, int wave, int lane)
{
    constexpr int kRows = 32 / WGK;
    typedef SlabRows<GATED> S;
    Raw8 res[2][1];
    Bias8<GATED> bias;
    const int c = S::column(col0, lane);
    bias.load(p, it.e, c, cols);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        res[i][0] = residual8(p, it.m0 + 32 * i + wave * kRows + lane / S::kPer, it.end, c, cols);
        slab_write<2>(lds + (i * WGK + wave) * kSlabBytes, acc[i], 0, lane);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        finish_rows<GATED, 1, WGK>(p, lds + i * WGK * kSlabBytes, bias, res[i], it.m0 + 32 * i, it.end, col0, cols,
                                   it.e, wave * kRows, kRows, lane);
}

// The same with K split over work-groups: the sums go to the workspace,
// [split][rows][N] in FP32, gated columns still in the product's order.
template <int WGK>
__device__ __forceinline__ void groups_partial(const LinArgs& p, uint8_t* lds, v16f (&acc)[2][2], const LinItem& it,
                                               int n0, int wave, int lane)
{
    constexpr int kRows = 32 / WGK;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        slab_write<2>(lds + (i * WGK + wave) * kSlabBytes, acc[i], 0, lane);
    __syncthreads();
    const int c8 = lane & 7;
    // gated tiles hold 32 gate columns, then 32 up columns
    const int half = p.N / 2;
    const int c = !p.gated ? n0 + 8 * c8 : n0 / 2 + 8 * (c8 & 3);
    const int n = !p.gated ? p.N : half;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = wave * kRows + (lane >> 3), row = it.m0 + 32 * i + r;
        float z[8];
        slab_read8<WGK, 0>(lds + i * WGK * kSlabBytes, r, c8, z);
        if (row >= it.end)
            continue;
        float* out = p.part + ((int64_t)it.ks * p.rows + row) * p.N + c + (p.gated && c8 >= 4 ? half : 0);
        if (c + 8 <= n) {
            __builtin_memcpy(out, z, 32);
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (c + u < n)
                    out[u] = z[u];
        }
    }
}

// One BM x BN tile of the product per work-group, WGK K groups of WGM x WGN
// waves (each a run of the K-steps; a group whose steps run out one early
// only meets the last barrier).  After the K loop the stages are
// free: the accumulators go through LDS in slabs of 32 rows x 64 columns, so
// that bias, activation, residual and the stores run on whole rows; the K
// groups' slabs are added there in group order.  Measured, with what bounds
// them: 256 x 256 native, 8192 x 8192 x 8192 with bias, silu and residual, 475
// us (the K loop; its copies are about 100 us of it, the epilogue 5%); 128 x 128 native by expert, 16384
// rows of 4096 x 4096 over 32 experts, gated silu to MXFP8, 395 us, 1.40
// PFLOP/s (the same copies, twice the bytes per product, and tiles that end
// early: 11% of their rows); by inner range, exact, 24 experts of 384 tokens,
// 2048 x 2048, 135 us (the writes of 201 MB, 60 us, and the K loop at 1.03
// PFLOP/s one after the other); 64 x 64 split over all compute units, exact,
// 64 x 2048 x 7168, 11.5 us (latency: seven K-steps per work-group).
// WGS work-groups share a compute unit.
template <int BM, int BN, int WGM, int WGN, int WGK, int WGS, bool EXACT, int FA, int FB>
__global__ void __launch_bounds__(WGM * WGN * WGK * 64)
    __attribute__((amdgpu_waves_per_eu(WGM * WGN * WGK * WGS / 4, WGM * WGN * WGK * WGS / 4)))
linear_kernel(LinArgs p)
{
    constexpr int NWG = WGM * WGN;
    constexpr int TM = BM / WGM, TN = BN / WGN;
    constexpr int GA = TM / 32, GB = TN / 32;
    static_assert(TN % 64 == 0, "slabs of 64 columns; gated blocks come in pairs");
    typedef StageGeom<BM, BN, NWG> G;
    typedef PairGeom<BM, BN, NWG> R;
    constexpr int kWaveEpilogue = kSlabBytes + TM * TN * 2;      // a slab and a 16-bit residual
    constexpr int kLoop = WGK * (EXACT ? 2 * G::STAGE : R::BYTES);
    constexpr int kLds = WGK == 1 && NWG * kWaveEpilogue > kLoop ? NWG * kWaveEpilogue : kLoop;
    static_assert(WGS * kLds <= 160 * 1024, "LDS of a compute unit");

    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave / NWG, wl = wave % NWG;
    const int wm = wl / WGN, wn = wl % WGN;

    LinItem it;
    if (!lin_item<BM>(p, lane, it))
        return;
    if (it.zero) {
        zero_rows<BM, BN>(p, it);
        return;
    }
    const int n0 = it.tn * BN;
    v16f acc[GA][GB];
#pragma unroll
    for (int i = 0; i < GA; ++i)
#pragma unroll
        for (int g = 0; g < GB; ++g)
            acc[i][g] = v16f{};
    if (it.steps > 0) {
        const int64_t wrow = p.gated ? n0 / 2 : n0;
        const int64_t e = p.mode == kByRows ? it.e : 0;
        // K group wk: a run of K-steps, one more for the first groups where
        // they do not divide evenly
        const int share = it.steps / WGK, more = it.steps % WGK;
        const int nsteps = share + (more ? 1 : 0), valid = share + (wk < more ? 1 : 0);
        int first = it.k0 + wk * share + (wk < more ? wk : more);
        if (WGK > 1 && valid == 0)
            first = it.k0;                  // copied, never multiplied
        const StepSrc src0 = {p.a + it.m0 * p.lda + (int64_t)first * kBK,
                              p.w + e * p.w_group + wrow * p.ldw + (int64_t)first * kBK,
                              p.as + it.m0 * p.ldas + first * 4, p.ws + e * p.ws_group + wrow * p.ldws + first * 4};
        if constexpr (EXACT) {
            CopyOffsets<BM, BN, NWG, 32> co;
            lin_copy_offsets<BM, BN, NWG>(p, it.m0, it.end, n0, wl, lane, co);
            const int last = valid > 0 ? valid - 1 : 0;
            auto src_of = [&](int s) {
                const int k = WGK == 1 || s < last ? s : last;
                return StepSrc{uniform(src0.a + (int64_t)k * kBK), uniform(src0.b + (int64_t)k * kBK),
                               uniform(src0.as + k * 4), uniform(src0.bs + k * 4)};
            };
            exact_mainloop<BM, BN, WGM, WGN, WGK, FA, FB, (WGK > 1), true>(lds, lds + WGK * G::STAGE, co, src_of, nsteps,
                                                                     valid, wk, wl, lane, acc);
        } else {
            PairCopies<BM, BN, NWG> co;
            co.init(p, it.m0, it.end, n0, wl, lane);
            native_mainloop<BM, BN, WGM, WGN, WGK, FA, FB>(p, lds + wk * R::BYTES, co, src0, nsteps, valid,
                                                           p.K / 32 - 4 * first, p.K < 16 * 32, it.m0, it.end, n0,
                                                           wl, lane, acc);
        }
    }
    const int cols = p.gated ? p.N / 2 : p.N;
    __syncthreads();        // every wave has read its last fragments
    if constexpr (WGK > 1) {
        static_assert(NWG == 1 && GA == 2 && GB == 2 && 2 * WGK * kSlabBytes <= kLds, "two sets of slabs");
        if (p.split > 1)
            groups_partial<WGK>(p, lds, acc, it, n0, wave, lane);
        else if (p.gated)
            groups_epilogue<true, WGK>(p, lds, acc, it, n0, cols, wave, lane);
        else
            groups_epilogue<false, WGK>(p, lds, acc, it, n0, cols, wave, lane);
    } else {
        const int row0 = it.m0 + wm * TM, col0 = n0 + wn * TN;
        uint8_t* const mem = lds + wave * kWaveEpilogue;
        const int res = residual_path(p);
        if (p.gated) {
            if (res == kNoResidual)
                tile_epilogue<true, kNoResidual, GA, GB>(p, mem, acc, it, row0, col0, cols, lane);
            else if (res == kLdsResidual)
                tile_epilogue<true, kLdsResidual, GA, GB>(p, mem, acc, it, row0, col0, cols, lane);
            else
                tile_epilogue<true, kDirectResidual, GA, GB>(p, mem, acc, it, row0, col0, cols, lane);
        } else {
            if (res == kNoResidual)
                tile_epilogue<false, kNoResidual, GA, GB>(p, mem, acc, it, row0, col0, cols, lane);
            else if (res == kLdsResidual)
                tile_epilogue<false, kLdsResidual, GA, GB>(p, mem, acc, it, row0, col0, cols, lane);
            else
                tile_epilogue<false, kDirectResidual, GA, GB>(p, mem, acc, it, row0, col0, cols, lane);
        }
    }
}

// ------------------------------------------------- few rows: skinny kernel --

// Sums of the waves, in order, and the epilogue of a BM x BN tile.
template <bool GATED, int BM, int BN, int NW>
__device__ __forceinline__ void skinny_epilogue(const LinArgs& p, const float* red, const LinItem& it, int c0,
                                                int cols, int tid, int lane)
{
    constexpr int LD = BN + 4;
    constexpr int kPer = (GATED ? BN / 2 : BN) / 8;     // eights of outputs per row
    constexpr int kTotal = BM * kPer;
#pragma unroll
    for (int i0 = 0; i0 < kTotal; i0 += NW * 64) {
        const int i = i0 + tid;
        if (i - lane >= kTotal)             // whole waves
            return;
        const int r = i < kTotal ? i / kPer : BM - 1, c8 = i < kTotal ? i % kPer : 0;
        const int row = it.m0 + r, c = c0 + 8 * c8;
        const bool ok = i < kTotal && row < it.end && c < cols;
        Bias8<GATED> bias;
        bias.load(p, it.e, c, cols);
        const Raw8 res[1] = {residual8(p, row, it.end, c, cols)};
        float z[8], z1[GATED ? 8 : 1];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            z[u] = 0.f;
            if constexpr (GATED)
                z1[u] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const float* src = red + (k * BM + r) * LD + 8 * c8;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                z[u] += src[u];
            if constexpr (GATED) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    z1[u] += src[BN / 2 + u];
            }
        }
        finish<GATED, 1, 1>(p, it.e, row, c, cols, ok ? 1 : 0, z, z1, bias, res, lane);
    }
}

// Up to 16 RT rows: the weights' bytes are the cost, and no row of w is used
// by a second wave, so they go straight from memory to registers in the
// MFMA's operand layout (lane l: row l % 16, K [16 q, +16) and [64 + 16 q,
// +16), q = l / 16), without LDS.  A work-group of NW waves takes NB blocks
// of 16 columns (gated: the first NB / 2 gate, the others up) and splits K
// over its waves in runs of K-steps; the loads of U steps are in flight per
// wave.  The waves' sums are added in wave order through LDS, where the
// epilogue reads them row-wise.  Bound by memory: 64 pairs over 43 of 128
// experts, gated 1536 x 2048 weights to MXFP8 37 us (3.8 TB/s), 2048 x 768
// weights 18.4 us (3.8 TB/s).
template <int RT, int NB, int NW, int U, bool EXACT, int FA, int FB>
__global__ void __launch_bounds__(NW * 64) linear_skinny_kernel(LinArgs p)
{
    constexpr int BM = 16 * RT, BN = 16 * NB;
    constexpr int LD = BN + 4;              // floats per row of the sums (4: spreads the rows over the banks)
    __shared__ __attribute__((aligned(16))) float red[NW * BM * LD];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lr = lane & 15, lq = lane >> 4;
    LinItem it;
    if (!lin_item<BM>(p, lane, it))
        return;
    if (it.zero) {
        zero_rows<BM, BN>(p, it);
        return;
    }
    const int cols = p.gated ? p.N / 2 : p.N;
    const int width = p.gated ? BN / 2 : BN;
    const int c0 = it.tn * width;
    const int64_t e = p.mode == kByRows ? it.e : 0;
    const int64_t kofs = (int64_t)it.k0 * kBK + 16 * lq;
    const uint8_t *wp[NB], *wsp[NB], *ap[RT], *asp[RT];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int half = p.gated && 2 * b >= NB;
        int c = c0 + 16 * (half ? b - NB / 2 : b) + lr;
        c = c < cols ? c : cols - 1;
        const int64_t n = half ? (int64_t)cols + c : c;
        wp[b] = p.w + e * p.w_group + n * p.ldw + kofs;
        wsp[b] = p.ws + e * p.ws_group + n * p.ldws + it.k0 * 4;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = it.m0 + 16 * r + lr;
        const int64_t m = row < it.end ? row : it.end - 1;
        ap[r] = p.a + m * p.lda + kofs;
        asp[r] = p.as + m * p.ldas + it.k0 * 4;
    }
    v4f acc[RT][NB], tot[RT][NB];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            acc[r][b] = tot[r][b] = v4f{0.f, 0.f, 0.f, 0.f};

    const int per = (it.steps + NW - 1) / NW;
    const int lo = wave * per, hi = lo + per < it.steps ? lo + per : it.steps;
    u32x4 wv[U][NB][2], av[U][RT][2];
    uint32_t wsv[U][NB], asv[U][RT];
    auto load = [&](auto uc, int s) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            wv[u][b][0] = *reinterpret_cast<const u32x4*>(wp[b] + (int64_t)s * kBK);
            wv[u][b][1] = *reinterpret_cast<const u32x4*>(wp[b] + (int64_t)s * kBK + 64);
            wsv[u][b] = *reinterpret_cast<const uint32_t*>(wsp[b] + (int64_t)s * 4);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            av[u][r][0] = *reinterpret_cast<const u32x4*>(ap[r] + (int64_t)s * kBK);
            av[u][r][1] = *reinterpret_cast<const u32x4*>(ap[r] + (int64_t)s * kBK + 64);
            asv[u][r] = *reinterpret_cast<const uint32_t*>(asp[r] + (int64_t)s * 4);
        }
    };
    auto multiply = [&](auto uc, int s) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        __builtin_amdgcn_sched_barrier(0);      // one step's conversions at a time
        if constexpr (EXACT) {
            // as in mxgemm_kernel's 16-wide exact form: half h of the
            // step is the lane's chunk h, scaled by MX block 2 h + q / 2
            const int shift = 8 * (lq >> 1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    v8bf bb[NB], ab[RT];
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const u32x4 x = wv[u][b][h];
                        bb[b] = fp8x8_to_bf16<FB>(m ? u32x2{x.z, x.w} : u32x2{x.x, x.y},
                                                  e8m0_to_f32(wsv[u][b] >> (shift + 16 * h)));
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const u32x4 x = av[u][r][h];
                        ab[r] = fp8x8_to_bf16<FA>(m ? u32x2{x.z, x.w} : u32x2{x.x, x.y},
                                                  e8m0_to_f32(asv[u][r] >> (shift + 16 * h)));
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            acc[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bb[b], ab[r], acc[r][b], 0, 0, 0);
                }
            // fresh sums per pair of K-steps, as in the other exact forms
            if (((s - lo) & 1) == 1 || s == hi - 1) {
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        tot[r][b] += acc[r][b];
                        acc[r][b] = v4f{0.f, 0.f, 0.f, 0.f};
                    }
            }
        } else {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const u32x4 x0 = wv[u][b][0], x1 = wv[u][b][1], y0 = av[u][r][0], y1 = av[u][r][1];
                    tot[r][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        v8i{(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w, (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w},
                        v8i{(int)y0.x, (int)y0.y, (int)y0.z, (int)y0.w, (int)y1.x, (int)y1.y, (int)y1.z, (int)y1.w},
                        tot[r][b], FB, FA, 0, (int)(wsv[u][b] >> (8 * lq)), 0, (int)(asv[u][r] >> (8 * lq)));
                }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // The loads of U steps are always on their way: a step's registers are
    // loaded again, U steps on, as soon as it is multiplied.
    static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
        if (lo + decltype(uc)::value < hi)
            load(uc, lo + decltype(uc)::value);
    });
    int s0 = lo;
    for (; s0 + 2 * U <= hi; s0 += U)
        static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value;
            multiply(uc, s0 + u);
            load(uc, s0 + u + U);
        });
    static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        if (s0 + u < hi) {
            multiply(uc, s0 + u);
            if (s0 + u + U < hi)
                load(uc, s0 + u + U);
        }
    });
    static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        if (s0 + u + U < hi)
            multiply(uc, s0 + u + U);
    });
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            *reinterpret_cast<v4f*>(red + (wave * BM + 16 * r + lr) * LD + 16 * b + 4 * lq) = tot[r][b];
    __syncthreads();
    if (p.gated)
        skinny_epilogue<true, BM, BN, NW>(p, red, it, c0, cols, tid, lane);
    else
        skinny_epilogue<false, BM, BN, NW>(p, red, it, c0, cols, tid, lane);
}

// ------------------------------------------------------------------ launch --

template <int BM, int BN, int WGM, int WGN, int WGK, int WGS, int FA, int FB>
static hipError_t launch_lin_tile(bool exact, const LinArgs& a, hipStream_t stream)
{
    if (exact) {
        if constexpr ((BM / WGM) * (BN / WGN) <= 64 * 64) {
            hipLaunchKernelGGL((linear_kernel<BM, BN, WGM, WGN, WGK, WGS, true, FA, FB>), dim3(a.total_work),
                               dim3(WGM * WGN * WGK * 64), 0, stream, a);
            return hipGetLastError();
        } else {
            return hipErrorInvalidValue;    // never planned
        }
    }
    hipLaunchKernelGGL((linear_kernel<BM, BN, WGM, WGN, WGK, WGS, false, FA, FB>), dim3(a.total_work),
                       dim3(WGM * WGN * WGK * 64), 0, stream, a);
    return hipGetLastError();
}

template <int RT, int NB, int NW, int U, int FA, int FB>
static hipError_t launch_lin_skinny(bool exact, const LinArgs& a, hipStream_t stream)
{
    if (exact)
        hipLaunchKernelGGL((linear_skinny_kernel<RT, NB, NW, U, true, FA, FB>), dim3(a.total_work), dim3(NW * 64), 0,
                           stream, a);
    else
        hipLaunchKernelGGL((linear_skinny_kernel<RT, NB, NW, U, false, FA, FB>), dim3(a.total_work), dim3(NW * 64), 0,
                           stream, a);
    return hipGetLastError();
}

// Skinny tiles: blocks of 16 columns per tile and waves per work-group by the
// plan's choice.  Measured (exact): experts' 2048 x 768 weights, 64 pairs over
// 128 experts, 22 / 26 / 39 us with 2 / 4 / 8 waves; 4096 x 4096 weights, 512
// pairs over 64, 373 / 357 / 362 us; one row x 8192 x 8192, 20.7 / 16.6 / 16.0 us.
template <int RT, int FA, int FB>
static hipError_t launch_lin_rows(bool exact, const LinArgs& a, hipStream_t stream)
{
    switch (a.skinny) {
    case kSkinnyNarrow: return launch_lin_skinny<RT, 1, 16, 2, FA, FB>(exact, a, stream);
    case kSkinny2: return launch_lin_skinny<RT, 2, 2, 2, FA, FB>(exact, a, stream);
    case kSkinny4: return launch_lin_skinny<RT, 2, 4, 2, FA, FB>(exact, a, stream);
    case kSkinny8: return launch_lin_skinny<RT, 2, 8, 2, FA, FB>(exact, a, stream);
    case kSkinnyWide: return launch_lin_skinny<RT, 4, 4, 1, FA, FB>(exact, a, stream);
    default: return hipErrorInvalidValue;
    }
}

template <int FA, int FB>
hipError_t launch_linear_fmt(int cfg, bool exact, const LinArgs& a, hipStream_t stream)
{
    switch (cfg) {
    case kLin256x256: return launch_lin_tile<256, 256, 2, 2, 1, 1, FA, FB>(exact, a, stream);
    case kLin128x128: return launch_lin_tile<128, 128, 2, 2, 1, 2, FA, FB>(exact, a, stream);
    case kLin64x64: return launch_lin_tile<64, 64, 1, 1, 4, 1, FA, FB>(exact, a, stream);
    case kLinRows32: return launch_lin_rows<2, FA, FB>(exact, a, stream);
    case kLinRows16: return launch_lin_rows<1, FA, FB>(exact, a, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace mxg
