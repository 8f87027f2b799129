// The FP8 product with a float32 scale for each block of 128, dense and by
// expert, templated on the FP8 formats of its operands.  Each format pair is
// instantiated in its own translation unit.
//
//   out[m][n] = sum over blocks b of sa[m][b] sw[n][b] (sum over k in b of a[m][k] w[n][k])
//
// One MFMA K-step is one block: the inner sum is formed in fresh accumulators,
// on the FP8 matrix unit (native) or on the BF16 one from exactly converted
// codes (exact), and added to the running totals times its scale, in FP32.
// So no sum runs over more than 128 products at one magnitude, and the vector
// unit's one multiply-add per output and block goes beside the matrix unit's
// 128: a 32 x 32 block takes 16 of them in 64 clocks, beside 128 clocks of FP8
// MFMA.
#pragma once

#include "block.h"
#include "linear_impl.h"

namespace mxg {

// E8M0 1.0 in every byte: the scaled MFMA's own scales are not used.
constexpr int kUnitScale = 0x7F7F7F7F;

// ------------------------------------------------------------------ copies --

// LDS of a K loop: stages of one K-step, rows of 128 bytes, A then W, then as
// many slots of the step's scales, a float per row.
template <int BM, int BN, int NW, int STAGES>
struct BlockGeom {
    static constexpr int A_BYTES = BM * kBK, CODES = (BM + BN) * kBK, SCALES = 4 * (BM + BN);
    static constexpr int BYTES = STAGES * (CODES + SCALES);
    static constexpr int JA = BM / 8 / NW, JB = BN / 8 / NW;        // 1 KB copies per wave and stage
    static constexpr int IS = (BM + BN) / 64, JS = (IS + NW - 1) / NW;      // copies of 64 scales
    static constexpr int COPIES = JA + JB + JS;
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && (BM + BN) % 64 == 0 && BM % 64 == 0,
                  "every wave copies as much as any other");
};

struct BlockSrc {
    const uint8_t *a, *w, *as, *ws;
};

// A wave's copies: source offsets relative to rows m0 of a and n0 of w, rows
// past the edge the last one there is (their results are not stored).
template <int BM, int BN, int NW, int STAGES>
struct BlockCopies {
    typedef BlockGeom<BM, BN, NW, STAGES> G;
    uint32_t a[G::JA], b[G::JB], s[G::JS];

    __device__ __forceinline__ void init(const BlockLinArgs& p, int m0, int end, int n0, int wave, int lane)
    {
        const int last = end - 1 - m0, edge = p.N - 1 - n0;
#pragma unroll
        for (int j = 0; j < G::JA; ++j) {
            const int row = 8 * (wave + j * NW) + (lane >> 3);
            a[j] = (uint32_t)((row < last ? row : last) * (uint32_t)p.lda) + swz_t<32>(row, lane & 7) * 16;
        }
#pragma unroll
        for (int j = 0; j < G::JB; ++j) {
            const int row = 8 * (wave + j * NW) + (lane >> 3);
            b[j] = (uint32_t)((row < edge ? row : edge) * (uint32_t)p.ldw) + swz_t<32>(row, lane & 7) * 16;
        }
#pragma unroll
        for (int j = 0; j < G::JS; ++j) {
            int row = 64 * piece(wave, j) + lane;
            if (row < BM) {
                s[j] = (uint32_t)(row < last ? row : last) * (uint32_t)p.as_row * 4;
            } else {
                row -= BM;
                row = row < edge ? row : edge;
                s[j] = (uint32_t)(p.squares ? (n0 + row) / kScaleBlock - n0 / kScaleBlock : row) *
                       (uint32_t)p.ws_row * 4;
            }
        }
    }
    // a wave with no piece of the scales left repeats the last one
    __device__ static __forceinline__ int piece(int wave, int j)
    {
        return wave + j * NW < G::IS ? wave + j * NW : G::IS - 1;
    }
    // copy t of a K-step to stage number `stage`
    __device__ __forceinline__ void issue(const BlockSrc& src, uint8_t* lds, int stage, int wave, int t) const
    {
        uint8_t* const codes = lds + stage * G::CODES;
#pragma unroll
        for (int j = 0; j < G::JA; ++j)
            if (t == j)
                dma16_at(uniform(src.a), a[j], codes + (wave + j * NW) * 1024);
#pragma unroll
        for (int j = 0; j < G::JB; ++j)
            if (t == G::JA + j)
                dma16_at(uniform(src.w), b[j], codes + G::A_BYTES + (wave + j * NW) * 1024);
#pragma unroll
        for (int j = 0; j < G::JS; ++j)
            if (t == G::JA + G::JB + j) {
                const int k = piece(wave, j);
                dma4_at(uniform(64 * k < BM ? src.as : src.ws), s[j],
                        lds + STAGES * G::CODES + stage * G::SCALES + k * 256);
            }
    }
    __device__ __forceinline__ void issue_all(const BlockSrc& src, uint8_t* lds, int stage, int wave) const
    {
#pragma unroll
        for (int t = 0; t < G::COPIES; ++t)
            issue(src, lds, stage, wave, t);
    }
};

// -------------------------------------------------------------- one K-step --

// The wave's block of the tile: rows from r0, columns from c0 of the stage.
// Fragments as in the MXFP8 loops: lane l has row l % 32 and, with q = l / 32,
// the 16-byte chunks 2 c + q of its 128 bytes.  The result of a 32 x 32 block
// has row l % 32 of a and column 8 (v / 4) + 4 q + v % 4 of w in element v.
typedef float v8f __attribute__((ext_vector_type(8)));

template <int GA, int GB, bool SQUARES>
struct BlockScales {
    float a[GA], w[GB][SQUARES ? 1 : 16];
    __device__ __forceinline__ void load(const float* rows, const float* cols, int lane)
    {
        const int lr = lane & 31, lq = lane >> 5;
#pragma unroll
        for (int i = 0; i < GA; ++i)
            a[i] = rows[32 * i + lr];
#pragma unroll
        for (int g = 0; g < GB; ++g) {
            if constexpr (SQUARES) {
                w[g][0] = cols[32 * g];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v4f x = *reinterpret_cast<const v4f*>(cols + 32 * g + 8 * q + 4 * lq);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        w[g][4 * q + u] = x[u];
                }
            }
        }
    }
    // (whole vectors: element by element, the largest tiles' totals went to scratch)
    __device__ __forceinline__ void add(v16f& total, const v16f& part, int i, int g) const
    {
        if constexpr (SQUARES) {
            total += part * (a[i] * w[g][0]);
        } else {
            const v16f y = {w[g][0], w[g][1], w[g][2], w[g][3], w[g][4], w[g][5], w[g][6], w[g][7],
                            w[g][8], w[g][9], w[g][10], w[g][11], w[g][12], w[g][13], w[g][14], w[g][15]};
            total += part * (y * a[i]);
        }
    }
    // elements [8 HALF, 8 HALF + 8) of block (i, g)
    template <int HALF>
    __device__ __forceinline__ void add_half(v8f& total, const v16f& part, int i, int g) const
    {
        v8f x;
        if constexpr (HALF == 0)
            x = __builtin_shufflevector(part, part, 0, 1, 2, 3, 4, 5, 6, 7);
        else
            x = __builtin_shufflevector(part, part, 8, 9, 10, 11, 12, 13, 14, 15);
        if constexpr (SQUARES) {
            total += x * (a[i] * w[g][0]);
        } else {
            constexpr int f = 8 * HALF;
            const v8f y = {w[g][f], w[g][f + 1], w[g][f + 2], w[g][f + 3], w[g][f + 4], w[g][f + 5], w[g][f + 6], w[g][f + 7]};
            total += x * (y * a[i]);
        }
    }
};

template <int GA, int GB, bool EXACT, bool SQUARES, int FA, int FB>
__device__ __forceinline__ void block_step(const uint8_t* a, const uint8_t* w, const float* rows, const float* cols,
                                           int lane, v16f (&acc)[GA][GB])
{
    const int lr = lane & 31, lq = lane >> 5;
    auto chunk = [&](const uint8_t* base, int row, int c) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4*>(base + (row + lr) * kBK + swz_t<32>(lr, 2 * c + lq) * 16);
    };
    BlockScales<GA, GB, SQUARES> s;
    s.load(rows, cols, lane);
    if constexpr (EXACT) {
        v16f part[GA][GB];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u32x4 ar[GA], wr[GB];
#pragma unroll
            for (int i = 0; i < GA; ++i)
                ar[i] = chunk(a, 32 * i, c);
#pragma unroll
            for (int g = 0; g < GB; ++g)
                wr[g] = chunk(w, 32 * g, c);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v8bf ab[GA], wb[GB];
#pragma unroll
                for (int i = 0; i < GA; ++i)
                    ab[i] = fp8x8_to_bf16<FA>(h ? u32x2{ar[i].z, ar[i].w} : u32x2{ar[i].x, ar[i].y}, 1.f);
#pragma unroll
                for (int g = 0; g < GB; ++g)
                    wb[g] = fp8x8_to_bf16<FB>(h ? u32x2{wr[g].z, wr[g].w} : u32x2{wr[g].x, wr[g].y}, 1.f);
#pragma unroll
                for (int i = 0; i < GA; ++i)
#pragma unroll
                    for (int g = 0; g < GB; ++g)
                        part[i][g] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            wb[g], ab[i], c == 0 && h == 0 ? v16f{} : part[i][g], 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < GA; ++i)
#pragma unroll
            for (int g = 0; g < GB; ++g)
                s.add(acc[i][g], part[i][g], i, g);
    } else {
        auto operand = [](const u32x4& lo, const u32x4& hi) __attribute__((always_inline)) {
            return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
        };
        u32x4 wr[GB][4];
#pragma unroll
        for (int g = 0; g < GB; ++g)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                wr[g][c] = chunk(w, 32 * g, c);
#pragma unroll
        for (int i = 0; i < GA; ++i) {
            u32x4 ar[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                ar[c] = chunk(a, 32 * i, c);
#pragma unroll
            for (int g = 0; g < GB; ++g) {
                v16f part = v16f{};
                part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(wr[g][0], wr[g][1]), operand(ar[0], ar[1]),
                                                                       part, FB, FA, 0, kUnitScale, 0, kUnitScale);
                part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(wr[g][2], wr[g][3]), operand(ar[2], ar[3]),
                                                                       part, FB, FA, 0, kUnitScale, 0, kUnitScale);
                s.add(acc[i][g], part, i, g);
            }
        }
    }
}

// ------------------------------------------------------------ native K loop --

// The K loop of tiles of several waves on the FP8 matrix unit, in slots of one
// MFMA (32 x 32 x 64; two of them, one on the other, make a block's inner
// sum).  While a slot's MFMA runs, the wave issues eight multiply-adds of the
// sum before, and its share of the LDS reads and copies: the next 32 rows'
// fragments of a, and, past the one barrier of a K-step, which comes before
// the last 32 rows' MFMAs (by then every wave holds all of step s in
// registers, and step s + 1 has landed), the first fragments and the scales of
// step s + 1 and the copies of step s + 2.  So neither the barrier nor an LDS
// read's latency stands between two MFMAs of a wave, and with two waves per
// SIMD the other one's fill what is left.  8192 x 8192 x 8192: 466 us (2.36
// PFLOP/s), against 521 for a loop that reads, multiplies and adds in turn.  A
// wave whose MFMA is due goes before the other's multiply-adds (without the
// priority 478); a copy to a slot, since two held up its LDS reads (474).  The
// matrix unit is busy 62% of the time at the clock it then runs at; without the
// copies the loop takes 419, without the multiply-adds 430.
template <int GA, int GB, bool SQUARES, int FA, int FB, class Copies, class Src>
__device__ __forceinline__ void native_block_loop(const Copies& co, const Src& src_at, uint8_t* lds, int nsteps, int wl,
                                                  int a_row, int w_row, bool idle, int lane, v16f (&acc)[GA][GB])
{
    typedef typename Copies::G G;
    constexpr int kSlots = GA * GB * 2, kRow = GB * 2;      // MFMAs of a K-step, of 32 rows
    constexpr int kBarrier = kSlots - kRow;                 // the barrier is before this one
    const int lr = lane & 31, lq = lane >> 5;
    const int last = nsteps - 1;
    const float* const scales = reinterpret_cast<const float*>(lds + 2 * G::CODES);
    constexpr int kScales = G::SCALES / 4;
    const int a_rows = G::A_BYTES / kBK;                    // scales: a's rows, then w's

    auto frag = [&](int stage, int row, int c) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4*>(lds + stage * G::CODES + (row + lr) * kBK + swz_t<32>(lr, 2 * c + lq) * 16);
    };
    auto operand = [](const u32x4& lo, const u32x4& hi) __attribute__((always_inline)) {
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    u32x4 w[GB][4], a[2][4];
    BlockScales<GA, GB, SQUARES> now, next;
    co.issue_all(src_at(0), lds, 0, wl);
    co.issue_all(src_at(last < 1 ? last : 1), lds, 1, wl);
    wait_copies<G::COPIES>();
    __syncthreads();
    if (idle) {         // copies and barriers only; the SIMD's other wave has its matrix unit
        for (int s = 0; s < nsteps; ++s) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            co.issue_all(src_at(s + 2 < last ? s + 2 : last), lds, s & 1, wl);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        return;
    }
#pragma unroll
    for (int g = 0; g < GB; ++g)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            w[g][c] = frag(0, a_rows + w_row + 32 * g, c);
#pragma unroll
    for (int c = 0; c < 4; ++c)
        a[0][c] = frag(0, a_row, c);
    next.load(scales + a_row, scales + a_rows + w_row, lane);
    now = next;

    v16f part[2];               // the sum being formed and the one before
    part[1] = v16f{};           // (the first slots add zero to the last block)
    v8f total[GA][GB][2];
#pragma unroll
    for (int i = 0; i < GA; ++i)
#pragma unroll
        for (int g = 0; g < GB; ++g)
            total[i][g][0] = total[i][g][1] = v8f{};
    for (int s = 0; s < nsteps; ++s) {
        const int cur = s & 1, nxt = cur ^ 1;
        const BlockSrc src1 = src_at(s + 1 < last ? s + 1 : last), src2 = src_at(s + 2 < last ? s + 2 : last);
        static_for<0, kSlots>([&](auto uc) __attribute__((always_inline)) {
            constexpr int u = decltype(uc)::value, i = u / kRow, g = u % kRow / 2, m = u % 2, pair = u / 2;
            if constexpr (u == kBarrier) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                __syncthreads();
            }
            v16f& sum = part[pair & 1];
            __builtin_amdgcn_s_setprio(1);
            sum = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                operand(w[g][2 * m], w[g][2 * m + 1]), operand(a[i & 1][2 * m], a[i & 1][2 * m + 1]),
                m == 0 ? v16f{} : sum, FB, FA, 0, kUnitScale, 0, kUnitScale);
            __builtin_amdgcn_s_setprio(0);
            // the multiply-adds of the pair before
            constexpr int before = (pair + GA * GB - 1) % (GA * GB), bi = before / GB, bg = before % GB;
            if constexpr (u == 2)
                now = next;     // (the last pair of the step before had its own until here)
            now.template add_half<m>(total[bi][bg][m], part[(pair & 1) ^ 1], bi, bg);
            // copies: from the barrier on, the last ones in the next step's
            // first slots (then of what was step s + 2)
            constexpr int t = u >= kBarrier ? u - kBarrier : u + kRow;
            if constexpr (t < G::COPIES) {
                if constexpr (u >= kBarrier)
                    co.issue(src2, lds, cur, wl, t);
                else        // (of the second step again, in the first one)
                    co.issue(src1, lds, nxt, wl, t);
            }
            // fragments
            if constexpr (i + 1 < GA) {
                if constexpr (GB == 2)
                    a[(i + 1) & 1][u % kRow] = frag(cur, a_row + 32 * (i + 1), u % kRow);
            } else {
                if constexpr (m == 1) {
                    w[g][0] = frag(nxt, a_rows + w_row + 32 * g, 0);
                    w[g][1] = frag(nxt, a_rows + w_row + 32 * g, 1);
                    w[g][2] = frag(nxt, a_rows + w_row + 32 * g, 2);
                    w[g][3] = frag(nxt, a_rows + w_row + 32 * g, 3);
                }
                if constexpr (u % kRow < 2) {
                    constexpr int c = 2 * (u % kRow);
                    a[GA & 1][c] = frag(nxt, a_row, c);
                    a[GA & 1][c + 1] = frag(nxt, a_row, c + 1);
                }
                if constexpr (u % kRow == 2)
                    next.load(scales + nxt * kScales + a_row, scales + nxt * kScales + a_rows + w_row, lane);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    now.template add_half<0>(total[GA - 1][GB - 1][0], part[1], GA - 1, GB - 1);
    now.template add_half<1>(total[GA - 1][GB - 1][1], part[1], GA - 1, GB - 1);
#pragma unroll
    for (int i = 0; i < GA; ++i)
#pragma unroll
        for (int g = 0; g < GB; ++g)
            acc[i][g] = __builtin_shufflevector(total[i][g][0], total[i][g][1], 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12,
                                                13, 14, 15);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy outlives the work-group
}

// ---------------------------------------------------------------- epilogue --

// N consecutive elements of the output's type from v, to columns [c, c + N) of a
// row of n at p (any element alignment); those past n are dropped.  FP32 outputs
// (weights' gradients, read much later) are written past the caches, so that
// beside them the operands stay there: 24 experts of 384 tokens, 2048 x 2048,
// 145 us exact and 106 native, against 170 and 143 through the caches.  That takes
// whole lines per store: with 32 bytes of a row per lane the writes alone took
// 174 us, against 70.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));

template <int TYPE, int N>
__device__ __forceinline__ void put_out(void* base, int64_t at, int c, int n, const float (&v)[N])
{
    typename Element<TYPE>::T* p = static_cast<typename Element<TYPE>::T*>(base) + at + c;
    static_assert(N * sizeof(*p) == 16, "one store");
    if (c + N <= n) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == kFP32)
                w[i] = __float_as_uint(v[i]);
            else if constexpr (TYPE == kBF16)
                w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            else
                w[i] = Element<TYPE>::put(v[2 * i]) | (uint32_t)Element<TYPE>::put(v[2 * i + 1]) << 16;
        }
        if constexpr (TYPE == kFP32)
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4_a2*>(p));
        else
            *reinterpret_cast<u32x4_a2*>(p) = w;
    } else {
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (c + u < n)
                p[u] = Element<TYPE>::put(v[u]);
    }
}

// The wave's totals (rows from row0, columns from col0) through LDS in slabs of
// 32 rows x 64 columns, so that eight neighbouring lanes write whole lines of a
// row.  `mem`: the wave's LDS, a slab.
template <int GA>
__device__ __forceinline__ void block_epilogue(const BlockLinArgs& p, uint8_t* mem, const v16f (&acc)[GA][2],
                                               const LinItem& it, int row0, int col0, int lane)
{
    const int l = lane & 7;
    void* out = p.out;
    if (p.mode == kByInner)
        out = static_cast<char*>(out) + it.e * p.out_group * (p.out_type == kFP32 ? 4 : 2);
#pragma unroll 1
    for (int t = 0; t < GA; ++t) {
#pragma unroll
        for (int i = 0; i < GA; ++i)
            if (t == i)
                slab_write<2>(mem, acc[i], 0, lane);
        // LDS operations of one wave complete in order, and the wave reads
        // back only what it wrote itself
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 2
        for (int r0 = 0; r0 < 32; r0 += 8) {
            const int r = r0 + (lane >> 3), row = row0 + 32 * t + r;
            const bool wide = p.out_type == kFP32;      // its 256 bytes of a row are two lines
            const v4f x0 = *reinterpret_cast<const v4f*>(mem + slab_at(r, wide ? l : 2 * l));
            const v4f x1 = *reinterpret_cast<const v4f*>(mem + slab_at(r, wide ? l + 8 : 2 * l + 1));
            if (row >= it.end)
                continue;
            const int64_t at = row * p.ld_out;
            if (wide) {
                const float a[4] = {x0[0], x0[1], x0[2], x0[3]}, b[4] = {x1[0], x1[1], x1[2], x1[3]};
                put_out<kFP32>(out, at, col0 + 4 * l, p.N, a);
                put_out<kFP32>(out, at, col0 + 32 + 4 * l, p.N, b);
            } else {
                const float a[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
                if (p.out_type == kBF16)
                    put_out<kBF16>(out, at, col0 + 8 * l, p.N, a);
                else
                    put_out<kFP16>(out, at, col0 + 8 * l, p.N, a);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// ------------------------------------------------------------------ kernel --

// One BM x BN tile per work-group, WGK K groups of WGM x WGN waves.  Two
// stages: while a K-step is multiplied, the next one's copies are on their
// way.  A K group is a run of the K-steps with stages of its own; one of a
// single wave reads only what it copied itself and needs no barrier.
//
// Tiles of 128 x 128 keep the simple loop: two work-groups on a compute unit fill
// each other's waits (8192 x 8192 x 8192 native 562 us, 572 with the loop above;
// exact 935, 1.18 PFLOP/s, where a plain BF16 product reaches 1.25).  More stages
// with one work-group (256 x 128 in three, 592; 128 x 128 in four, 959, with eight
// waves 743, with fragments read a step ahead 909) or eight waves in each of two
// (567) did no better.  Where work-groups are alone (256 x 4096 x 4096 native, 64
// of them: 26 us) the copies by themselves take 22 and the arithmetic 20.
template <int BM, int BN, int WGM, int WGN, int WGK, int WGS, bool EXACT, bool SQUARES, int FA, int FB>
__global__ void __launch_bounds__(WGM * WGN * WGK * 64)
    __attribute__((amdgpu_waves_per_eu(WGM * WGN * WGK * WGS / 4, WGM * WGN * WGK * WGS / 4)))
block_linear_kernel(BlockLinArgs p)
{
    constexpr int NWG = WGM * WGN;
    constexpr int TM = BM / WGM, TN = BN / WGN;
    constexpr int GA = TM / 32, GB = TN / 32;
    static_assert(TN == 64, "slabs of 64 columns, within one square");
    typedef BlockCopies<BM, BN, NWG, 2> Copies;
    typedef typename Copies::G G;
    constexpr int kLoop = WGK * G::BYTES, kSlabs = NWG * kSlabBytes;
    constexpr int kLds = kLoop > kSlabs ? kLoop : kSlabs;
    static_assert(WGS * kLds <= 160 * 1024, "LDS of a compute unit");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];

    const int tid = threadIdx.x, lane = tid & 63;
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
        const int64_t e = p.mode == kByRows ? it.e : 0;
        const int share = it.steps / WGK, more = it.steps % WGK;
        const int nsteps = share + (wk < more ? 1 : 0);
        const int first = it.k0 + wk * share + (wk < more ? wk : more);
        uint8_t* const mem = lds + wk * G::BYTES;
        const float* const scales = reinterpret_cast<const float*>(mem + 2 * G::CODES);
        // a wave whose rows (or columns) all lie past the edge multiplies nothing
        const bool idle = it.m0 + wm * TM >= it.end || n0 + wn * TN >= p.N;
        Copies co;
        co.init(p, it.m0, it.end, n0, wl, lane);
        const BlockSrc src0 = {
            p.a + it.m0 * p.lda + (int64_t)first * kBK,
            p.w + e * p.w_group + n0 * p.ldw + (int64_t)first * kBK,
            reinterpret_cast<const uint8_t*>(p.a_scale + it.m0 * p.as_row + first * p.as_k),
            reinterpret_cast<const uint8_t*>(p.w_scale + e * p.w_scale_group +
                                             (SQUARES ? n0 / kScaleBlock : n0) * p.ws_row + first * p.ws_k)};
        auto src_at = [&](int s) {
            return BlockSrc{src0.a + (int64_t)s * kBK, src0.w + (int64_t)s * kBK, src0.as + s * p.as_k * 4,
                            src0.ws + s * p.ws_k * 4};
        };
        if constexpr (BM == 256) {
            native_block_loop<GA, GB, SQUARES, FA, FB>(co, src_at, mem, nsteps, wl, wm * TM, wn * TN, idle, lane,
                                                       acc);
        } else {
            // the first two steps' copies go out together (short inner ranges wait
            // for little else)
            if (nsteps > 0)
                co.issue_all(src_at(0), mem, 0, wl);
            if (nsteps > 1)
                co.issue_all(src_at(1), mem, 1, wl);
            for (int s = 0; s < nsteps; ++s) {
                if (s == 0 && nsteps > 1)
                    wait_copies<G::COPIES>();
                else
                    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                if constexpr (NWG > 1)
                    __syncthreads();        // step s has landed; step s - 1 is read
                if (s > 0 && s + 1 < nsteps)
                    co.issue_all(src_at(s + 1), mem, (s + 1) & 1, wl);
                const uint8_t* const codes = mem + (s & 1) * G::CODES;
                const float* const sc = scales + (s & 1) * (BM + BN);
                if (!idle)
                    block_step<GA, GB, EXACT, SQUARES, FA, FB>(codes + wm * TM * kBK, codes + G::A_BYTES + wn * TN * kBK,
                                                           sc + wm * TM, sc + BM + wn * TN, lane, acc);
                if constexpr (NWG == 1)
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // read before it is copied over
            }
        }
    }
    __syncthreads();        // every wave has read its last fragments
    if constexpr (WGK > 1) {
        static_assert(NWG == 1 && GA == 2 && GB == 2 && 2 * WGK * kSlabBytes <= kLds, "two sets of slabs");
        if (p.split > 1)
            groups_partial<WGK>(p, lds, acc, it, n0, wave, lane);
        else
            groups_epilogue<false, WGK>(p, lds, acc, it, n0, p.N, wave, lane);
    } else {
        // (the largest tile has not a register left in its K loop: its epilogue is
        // the one that adds none)
        if constexpr (BM == 256)
            tile_epilogue<false, kNoResidual, GA, GB>(p, lds + wave * kSlabBytes, acc, it, it.m0 + wm * TM, n0 + wn * TN,
                                                      p.N, lane);
        else
            block_epilogue<GA>(p, lds + wave * kSlabBytes, acc, it, it.m0 + wm * TM, n0 + wn * TN, lane);
    }
}

// ------------------------------------------------- few rows: skinny kernel --

// Up to 16 RT rows: the weights' bytes are the cost, and no row of w is used
// by a second wave, so they go straight from memory to registers in the
// MFMA's operand layout (lane l: row l % 16, K [16 q, +16) and [64 + 16 q,
// +16), q = l / 16), without LDS.  A work-group of NW waves takes 16 NB
// columns (of one square) and splits K over its waves in runs of K-steps; the
// loads of U steps are in flight per wave.  The waves' sums are added in wave
// order through LDS, where the epilogue reads them row-wise.  64 x 2048 x 7168
// exact: 9.9 us again and again on the same operands, 14.5 in turn with others;
// the weights' 15 MB, which both row tiles read, each on an XCD of its own (30.1
// MB), are 6 of these, the rest a few loads' latency, one after the other, and the
// sums.  64 rows over 128 experts of 1536 x 2048, 118 MB of weights that have rows:
// 26 us (4.6 TB/s).
template <int RT, int NB, int NW, int U, bool EXACT, int FA, int FB>
__global__ void __launch_bounds__(NW * 64) block_skinny_kernel(BlockLinArgs p)
{
    constexpr int BM = 16 * RT, BN = 16 * NB;
    constexpr int LD = BN + 4;              // floats per row of the sums (4: spreads the rows over the banks)
    static_assert(kScaleBlock % BN == 0, "one square");
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
    const int c0 = it.tn * BN;
    const int64_t e = p.mode == kByRows ? it.e : 0;
    const int64_t kofs = (int64_t)it.k0 * kBK + 16 * lq;
    const uint8_t *wp[NB], *ap[RT];
    const float* asp[RT];
    const float* wsp = p.w_scale + e * p.w_scale_group + c0 / kScaleBlock * p.ws_row + it.k0 * p.ws_k;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        int c = c0 + 16 * b + lr;
        c = c < p.N ? c : p.N - 1;
        wp[b] = p.w + e * p.w_group + c * p.ldw + kofs;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = it.m0 + 16 * r + lr;
        const int64_t m = row < it.end ? row : it.end - 1;
        ap[r] = p.a + m * p.lda + kofs;
        asp[r] = p.a_scale + m * p.as_row + it.k0 * p.as_k;
    }
    v4f tot[RT][NB];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            tot[r][b] = v4f{0.f, 0.f, 0.f, 0.f};

    const int per = (it.steps + NW - 1) / NW;
    const int lo = wave * per, hi = lo + per < it.steps ? lo + per : it.steps;
    u32x4 wv[U][NB][2], av[U][RT][2];
    float wsv[U], asv[U][RT];
    auto load = [&](auto uc, int s) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            wv[u][b][0] = *reinterpret_cast<const u32x4*>(wp[b] + (int64_t)s * kBK);
            wv[u][b][1] = *reinterpret_cast<const u32x4*>(wp[b] + (int64_t)s * kBK + 64);
        }
        wsv[u] = wsp[s * p.ws_k];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            av[u][r][0] = *reinterpret_cast<const u32x4*>(ap[r] + (int64_t)s * kBK);
            av[u][r][1] = *reinterpret_cast<const u32x4*>(ap[r] + (int64_t)s * kBK + 64);
            asv[u][r] = asp[r][s * p.as_k];
        }
    };
    auto multiply = [&](auto uc) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        __builtin_amdgcn_sched_barrier(0);      // one step's conversions at a time
        v4f part[RT][NB];
        if constexpr (EXACT) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    v8bf bb[NB], ab[RT];
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const u32x4 x = wv[u][b][h];
                        bb[b] = fp8x8_to_bf16<FB>(m ? u32x2{x.z, x.w} : u32x2{x.x, x.y}, 1.f);
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const u32x4 x = av[u][r][h];
                        ab[r] = fp8x8_to_bf16<FA>(m ? u32x2{x.z, x.w} : u32x2{x.x, x.y}, 1.f);
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            part[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                bb[b], ab[r], h == 0 && m == 0 ? v4f{0.f, 0.f, 0.f, 0.f} : part[r][b], 0, 0, 0);
                }
        } else {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const u32x4 x0 = wv[u][b][0], x1 = wv[u][b][1], y0 = av[u][r][0], y1 = av[u][r][1];
                    part[r][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        v8i{(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w, (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w},
                        v8i{(int)y0.x, (int)y0.y, (int)y0.z, (int)y0.w, (int)y1.x, (int)y1.y, (int)y1.z, (int)y1.w},
                        v4f{0.f, 0.f, 0.f, 0.f}, FB, FA, 0, kUnitScale, 0, kUnitScale);
                }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float f = asv[u][r] * wsv[u];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    tot[r][b][v] += part[r][b][v] * f;
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
            multiply(uc);
            load(uc, s0 + decltype(uc)::value + U);
        });
    static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        if (s0 + u < hi) {
            multiply(uc);
            if (s0 + u + U < hi)
                load(uc, s0 + u + U);
        }
    });
    static_for<0, U>([&](auto uc) __attribute__((always_inline)) {
        if (s0 + decltype(uc)::value + U < hi)
            multiply(uc);
    });
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            *reinterpret_cast<v4f*>(red + (wave * BM + 16 * r + lr) * LD + 16 * b + 4 * lq) = tot[r][b];
    __syncthreads();
    skinny_epilogue<false, BM, BN, NW>(p, red, it, c0, p.N, tid, lane);
}

// ------------------------------------------------------------------ launch --

template <int BM, int BN, int WGM, int WGN, int WGK, int WGS, bool EXACT, int FA, int FB>
static hipError_t launch_block_tile(const BlockLinArgs& a, hipStream_t stream)
{
    const dim3 grid(a.total_work), block(WGM * WGN * WGK * 64);
    if (a.squares)
        hipLaunchKernelGGL((block_linear_kernel<BM, BN, WGM, WGN, WGK, WGS, EXACT, true, FA, FB>), grid, block, 0, stream,
                           a);
    else if constexpr (BM < 256)        // (the largest tile has no registers for a scale per column; never planned)
        hipLaunchKernelGGL((block_linear_kernel<BM, BN, WGM, WGN, WGK, WGS, EXACT, false, FA, FB>), grid, block, 0, stream,
                           a);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

template <int RT, int NB, int NW, int U, int FA, int FB>
static hipError_t launch_block_skinny(bool exact, const BlockLinArgs& a, hipStream_t stream)
{
    const dim3 grid(a.total_work), block(NW * 64);
    if (exact)
        hipLaunchKernelGGL((block_skinny_kernel<RT, NB, NW, U, true, FA, FB>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((block_skinny_kernel<RT, NB, NW, U, false, FA, FB>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <int RT, int FA, int FB>
static hipError_t launch_block_rows(bool exact, const BlockLinArgs& a, hipStream_t stream)
{
    switch (a.skinny) {
    case kSkinnyNarrow: return launch_block_skinny<RT, 1, 16, 2, FA, FB>(exact, a, stream);
    case kSkinny2: return launch_block_skinny<RT, 2, 2, 2, FA, FB>(exact, a, stream);
    case kSkinny4: return launch_block_skinny<RT, 2, 4, 2, FA, FB>(exact, a, stream);
    case kSkinny8: return launch_block_skinny<RT, 2, 8, 2, FA, FB>(exact, a, stream);
    default: return hipErrorInvalidValue;
    }
}

template <int FA, int FB>
hipError_t launch_block_fmt(int cfg, bool exact, const BlockLinArgs& a, hipStream_t stream)
{
    switch (cfg) {
    case kBlock256x256:
        return exact ? hipErrorInvalidValue : launch_block_tile<256, 256, 2, 4, 1, 1, false, FA, FB>(a, stream);
    case kBlock128x128:
        return exact ? launch_block_tile<128, 128, 2, 2, 1, 2, true, FA, FB>(a, stream)
                     : launch_block_tile<128, 128, 2, 2, 1, 2, false, FA, FB>(a, stream);
    case kBlock64x64:
        return exact ? launch_block_tile<64, 64, 1, 1, 4, 1, true, FA, FB>(a, stream)
                     : launch_block_tile<64, 64, 1, 1, 4, 1, false, FA, FB>(a, stream);
    case kBlockRows32: return launch_block_rows<2, FA, FB>(exact, a, stream);
    case kBlockRows16: return launch_block_rows<1, FA, FB>(exact, a, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace mxg
