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

// ------------------------------------------------------------- work items --

// What a work-group computes: rows [m0, end) of the product (at most the
// tile's height), columns from column tile tn, of expert e; K-steps
// [k0, k0 + steps).  zero: rows that belong to no expert.
struct LinItem {
    int m0, end, tn, e, k0, steps;
    bool zero;
};

// Row tile tm of the list of all experts' row tiles: expert e has
// ceil(rows of e / BM) of them, and the rows past the last expert come as one
// expert more.  All 64 lanes of the wave take part; the offsets are clamped
// to the rows there are.  False past the end of the list.
template <int BM>
__device__ __forceinline__ bool find_rows(const LinArgs& p, int tm, int lane, LinItem& it)
{
    int before = 0;
    for (int g0 = 0; g0 <= p.groups; g0 += 64) {
        const int g = g0 + lane;
        int lo = 0, hi = 0;
        if (g <= p.groups) {
            lo = p.offsets[g];
            hi = g < p.groups ? p.offsets[g + 1] : p.rows;
            lo = lo < 0 ? 0 : lo > p.rows ? p.rows : lo;
            hi = hi < lo ? lo : hi > p.rows ? p.rows : hi;
        }
        const int n = (hi - lo + BM - 1) / BM;
        int inc = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int x = __shfl_up(inc, d);
            inc += lane >= d ? x : 0;
        }
        const uint64_t past = __ballot(before + inc > tm);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int first = before + __shfl(inc - n, l);
            it.e = __builtin_amdgcn_readfirstlane(g0 + l);
            it.m0 = __builtin_amdgcn_readfirstlane(__shfl(lo, l) + (tm - first) * BM);
            it.end = __builtin_amdgcn_readfirstlane(__shfl(hi, l));
            it.zero = it.e == p.groups;
            return true;
        }
        before += __shfl(inc, 63);
    }
    return false;
}

template <int BM>
__device__ __forceinline__ bool lin_item(const LinArgs& p, int lane, LinItem& it)
{
    const int w = remap_block(blockIdx.x, gridDim.x);
    it.k0 = 0;
    it.steps = p.K / kBK;
    it.zero = false;
    it.e = 0;
    it.end = p.rows;
    int rest = w;
    if (p.mode == kByInner) {
        const int per = p.tiles_m * p.tiles_n;
        it.e = w / per;
        rest = w - it.e * per;
        int lo = p.offsets[it.e], hi = p.offsets[it.e + 1];
        lo = lo < 0 ? 0 : lo > p.K ? p.K : lo;
        hi = hi < lo ? lo : hi > p.K ? p.K : hi;
        it.k0 = lo / kBK;
        it.steps = hi / kBK - it.k0;
    }
    const TileCoord tc = decode_work(rest, p.tiles_m, p.tiles_n, 1, p.group_n);
    it.tn = tc.tn;
    it.m0 = tc.tm * BM;
    if (p.mode == kByRows)
        return find_rows<BM>(p, tc.tm, lane, it);
    return true;
}

// ---------------------------------------------------------------- epilogue --

// Eight columns [c, c + 8) of a bias or residual row, as FP32; columns past
// n are left alone.
template <int TYPE>
__device__ __forceinline__ void add8_t(const void* base, int64_t at, int c, int n, float (&v)[8])
{
    const typename Element<TYPE>::T* p = static_cast<const typename Element<TYPE>::T*>(base) + at + c;
    if (c + 8 <= n) {
        Pack<TYPE, 8> x;
        x.load(p);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] += x.get(u);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (c + u < n)
                v[u] += Element<TYPE>::get(p[u]);
    }
}

__device__ __forceinline__ void add8(int type, const void* base, int64_t at, int c, int n, float (&v)[8])
{
    if (type == kBF16)
        add8_t<kBF16>(base, at, c, n, v);
    else if (type == kFP16)
        add8_t<kFP16>(base, at, c, n, v);
    else
        add8_t<kFP32>(base, at, c, n, v);
}

template <int TYPE>
__device__ __forceinline__ void put8(void* base, int64_t at, int c, int n, const float (&v)[8])
{
    typename Element<TYPE>::T* p = static_cast<typename Element<TYPE>::T*>(base) + at + c;
    if (c + 8 <= n) {
        Pack<TYPE, 8> x;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            x.put(u, v[u]);
        x.store(p);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (c + u < n)
                p[u] = Element<TYPE>::put(v[u]);
    }
}

// Eight outputs of one row: columns [c, c + 8) of `cols`, from z (and, gated,
// the up half's z1).  Everything is FP32 until the one rounding of the store
// (the bfloat16 copy of z, kept for the gradient, is rounded by itself).
// With MXFP8 output four consecutive lanes hold one block of 32; every lane
// of the wave calls, `ok` says whether the row and the first column exist.
__device__ __forceinline__ void finish8(const LinArgs& p, int e, int row, int c, int cols, bool ok,
                                        float (&z)[8], float (&z1)[8], int lane)
{
    if (ok) {
        if (p.bias) {
            add8(p.bias_type, p.bias, (int64_t)e * p.N, c, cols, z);
            if (p.gated)
                add8(p.bias_type, p.bias, (int64_t)e * p.N + cols, c, cols, z1);
        }
        if (p.z) {
            put8<kBF16>(p.z, row * p.ld_z, c, cols, z);
            if (p.gated)
                put8<kBF16>(p.z, row * p.ld_z + cols, c, cols, z1);
        }
    }
    activate8(p.act, z);
    if (p.gated) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            z[u] *= z1[u];
    }
    if (ok && p.residual)
        add8(p.out_type > kFP32 ? kBF16 : p.out_type, p.residual, row * p.ld_res, c, cols, z);
    const int64_t at = (p.mode == kByInner ? e * p.out_group : 0) + row * p.ld_out;
    if (p.out_type >= kMxE4M3) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            m = max(m, __float_as_uint(z[u]) & 0x7FFFFFFFu);
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        u32x2 code;
        uint8_t byte;
        if (p.out_type == kMxE4M3) {
            const MxScale s = mx_scale<kE4M3>(m);
            code = u32x2{mx_codes<kE4M3>(s, z[0], z[1], z[2], z[3]), mx_codes<kE4M3>(s, z[4], z[5], z[6], z[7])};
            byte = s.byte;
        } else {
            const MxScale s = mx_scale<kE5M2>(m);
            code = u32x2{mx_codes<kE5M2>(s, z[0], z[1], z[2], z[3]), mx_codes<kE5M2>(s, z[4], z[5], z[6], z[7])};
            byte = s.byte;
        }
        if (ok) {       // cols is a multiple of 32: whole blocks are in or out
            *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(p.out) + at + c) = code;
            if ((lane & 3) == 0)
                p.out_s[row * p.ld_out_s + (c >> 5)] = byte;
        }
        return;
    }
    if (!ok)
        return;
    if (p.out_type == kBF16)
        put8<kBF16>(p.out, at, c, cols, z);
    else if (p.out_type == kFP16)
        put8<kFP16>(p.out, at, c, cols, z);
    else
        put8<kFP32>(p.out, at, c, cols, z);
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

// Columns [8 c, 8 c + 8) of row r, summed over `copies` slabs in order.
__device__ __forceinline__ void slab_read8(const uint8_t* buf, int copies, int stride, int r, int c, float (&v)[8])
{
    const v4f lo = *reinterpret_cast<const v4f*>(buf + slab_at(r, 2 * c));
    const v4f hi = *reinterpret_cast<const v4f*>(buf + slab_at(r, 2 * c + 1));
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        v[u] = lo[u];
        v[4 + u] = hi[u];
    }
    for (int k = 1; k < copies; ++k) {
        const v4f l2 = *reinterpret_cast<const v4f*>(buf + k * stride + slab_at(r, 2 * c));
        const v4f h2 = *reinterpret_cast<const v4f*>(buf + k * stride + slab_at(r, 2 * c + 1));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v[u] += l2[u];
            v[4 + u] += h2[u];
        }
    }
}

// Rows [r0, r1) of a slab (whose first row is `row0` of the product and
// first product column `col0`), finished and stored row-wise by one wave.
// Gated tiles hold gate and up columns in alternating blocks of 32.
__device__ __forceinline__ void slab_finish(const LinArgs& p, const uint8_t* buf, int copies, int stride, int r0,
                                            int r1, int row0, int end, int col0, int e, int lane)
{
    const int cols = p.gated ? p.N / 2 : p.N;
    const int per = p.gated ? 4 : 8;            // lanes per row
    const int cl = lane & (per - 1), rl = p.gated ? lane >> 2 : lane >> 3;
    const int c = (p.gated ? col0 / 2 : col0) + 8 * cl;
#pragma unroll 1
    for (int r = r0 + rl; r - rl < r1; r += 64 / per) {
        float z[8], z1[8];
        const int rr = r < r1 ? r : r1 - 1;
        slab_read8(buf, copies, stride, rr, cl, z);
        if (p.gated)
            slab_read8(buf, copies, stride, rr, 4 + cl, z1);
        finish8(p, e, row0 + r, c, cols, r < r1 && row0 + r < end && c < cols, z, z1, lane);
    }
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

// K loop on the scaled FP8 MFMA (32 x 32 x 64), software-pipelined.  A
// K-step (128 K) is two sub-steps m of 64 K.  While the GA x GB MFMAs of a
// sub-step run, the fragments of the next one are read from LDS into the
// other register set, one read after each MFMA or two, so no MFMA waits for
// a read.  The one barrier of a K-step opens sub-step 1: by then every wave
// has read all of the current stage, so the copies of step s + 2 are issued
// into it during sub-step 1 and have a whole K-step to land, and sub-step 1
// reads the first fragments of step s + 1.  Large wave tiles keep the LDS
// reads per MFMA low: a 128 x 128 wave tile reads each byte for 128 outputs,
// and four of them read 128 KB per 256 x 256 x 128 step (1024 clocks at 128
// bytes per clock, plus 512 for the copies' writes, against 2048 clocks of
// MFMA), where eight waves of 128 x 64 read 192 KB.
// Scale bytes: a lane reads the four of its row as one word, shifted so that
// byte 2 m is its block's.
template <int BM, int BN, int WGM, int WGN, int WGK, int FA, int FB, class Src>
__device__ __forceinline__ void native_mainloop(uint8_t* stage0, uint8_t* stage1,
                                                const CopyOffsets<BM, BN, WGM * WGN, 32>& co, const Src& src_of,
                                                int nsteps, int valid, int wk, int wl, int lane,
                                                v16f (&acc)[BM / WGM / 32][BN / WGN / 32])
{
    constexpr int MW = 32;
    constexpr int NWG = WGM * WGN;
    constexpr int TM = BM / WGM, TN = BN / WGN;
    constexpr int GA = TM / MW, GB = TN / MW;
    constexpr int NF = GA + GB;
    typedef StageGeom<BM, BN, NWG> G;
    constexpr int NCOPY = G::JA + G::JB + G::KSA + G::KSB;
    constexpr int NU = GA * GB;                    // MFMAs of a sub-step
    const int wm = wl / WGN, wn = wl % WGN;
    const int lr = lane & 31, lq = lane >> 5;
    const int ksub = wk * G::STAGE;

    const int a_row = ksub + (wm * TM + lr) * kBK;
    const int b_row = ksub + G::A_BYTES + (wn * TN + lr) * kBK;
    const int sa_row = ksub + G::SA_OFF + (wm * TM + lr) * 4;
    const int sb_row = ksub + G::SB_OFF + (wn * TN + lr) * 4;
    auto frag_off = [&](int f) { return f < GA ? a_row + f * MW * kBK : b_row + (f - GA) * MW * kBK; };
    auto scale_off = [&](int f) { return f < GA ? sa_row + f * MW * 4 : sb_row + (f - GA) * MW * 4; };
    auto chunk_off = [&](int m, int h) { return swz_t<MW>(lr, 4 * m + 2 * h + lq) * 16; };

#pragma unroll
    for (int i = 0; i < GA; ++i)
#pragma unroll
        for (int g = 0; g < GB; ++g)
            acc[i][g] = v16f{};

    u32x4 fr[2][NF][2];            // fragments by sub-step
    uint32_t sw[NF];               // scale words of the current K-step

    copy_issue(co, src_of(0), stage0 + ksub, wl);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (nsteps > 1)
        copy_issue(co, src_of(1), stage1 + ksub, wl);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        sw[f] = *reinterpret_cast<const uint32_t*>(stage0 + scale_off(f)) >> (8 * lq);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            fr[0][f][h] = *reinterpret_cast<const u32x4*>(stage0 + frag_off(f) + chunk_off(0, h));
    }

    auto operand = [&](int m, int f) {
        const u32x4 lo = fr[m][f][0], hi = fr[m][f][1];
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    auto kstep = [&](int s, const uint8_t* __restrict__ cur, uint8_t* __restrict__ nxt) {
        // past the last K-step the copies repeat the last one, into the
        // stage just released: no branches here
        const StepSrc src2 = src_of(s + 2 < nsteps ? s + 2 : nsteps - 1);
        uint32_t swn[NF];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (m == 1) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                __syncthreads();
            }
            const uint8_t* src = m == 0 ? cur : nxt;
            // the sub-step's other work, in this order: 2 NF fragment reads
            // of the next sub-step; at m = 1 the scale words of step s + 1
            // and the copies of step s + 2
            constexpr int kReads = 2 * NF;
            const int ntask = m == 0 ? kReads : kReads + NF + NCOPY;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int i = u / GB, g = u % GB;
                if (m == 0)
                    acc[i][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        operand(0, GA + g), operand(0, i), acc[i][g], FB, FA, 0, (int)sw[GA + g], 0, (int)sw[i]);
                else
                    acc[i][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        operand(1, GA + g), operand(1, i), acc[i][g], FB, FA, 2, (int)sw[GA + g], 2, (int)sw[i]);
                const int t0 = u * ntask / NU, t1 = (u + 1) * ntask / NU;
#pragma unroll
                for (int t = 0; t < kReads + NF + NCOPY; ++t) {
                    if (t < t0 || t >= t1)
                        continue;
                    if (t < kReads) {
                        // first the B fragments, which every MFMA row uses
                        const int f = (t / 2 + GA) % NF, h = t & 1;
                        fr[m ^ 1][f][h] = *reinterpret_cast<const u32x4*>(src + frag_off(f) + chunk_off(m ^ 1, h));
                    } else if (t < kReads + NF) {
                        const int f = t - kReads;
                        swn[f] = *reinterpret_cast<const uint32_t*>(nxt + scale_off(f)) >> (8 * lq);
                    } else {
                        copy_one(co, src2, const_cast<uint8_t*>(cur) + ksub, wl, 0, 1, t - kReads - NF);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int f = 0; f < NF; ++f)
            sw[f] = swn[f];
    };
    auto idle = [&]() {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    };
    for (int s = 0; s < nsteps; s += 2) {
        if (WGK == 1 || s < valid)
            kstep(s, stage0, stage1);
        else
            idle();
        if (s + 1 < nsteps) {
            if (WGK == 1 || s + 1 < valid)
                kstep(s + 1, stage1, stage0);
            else
                idle();
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ------------------------------------------------------------ tile kernel ---

// One BM x BN tile of the product per work-group, WGK K groups of WGM x WGN
// waves (group k takes K-steps k, k + WGK, ...; a group whose steps run out
// one early only meets the last barrier).  After the K loop the stages are
// free: the accumulators go through LDS in slabs of 32 rows x 64 columns, so
// that bias, activation, residual and the stores run on whole rows; the K
// groups' slabs are added there in group order.
template <int BM, int BN, int WGM, int WGN, int WGK, bool EXACT, int FA, int FB>
__global__ void __launch_bounds__(WGM * WGN * WGK * 64)
    __attribute__((amdgpu_waves_per_eu(WGM * WGN * WGK / 4, WGM * WGN * WGK / 4)))
linear_kernel(LinArgs p)
{
    constexpr int NWG = WGM * WGN;
    constexpr int TM = BM / WGM, TN = BN / WGN;
    constexpr int GA = TM / 32, GB = TN / 32;
    static_assert(TN % 64 == 0, "slabs of 64 columns; gated blocks come in pairs");
    typedef StageGeom<BM, BN, NWG> G;

    __shared__ __attribute__((aligned(1024))) uint8_t stage0[WGK * G::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t stage1[WGK * G::STAGE];

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
    if (it.steps > 0) {
        CopyOffsets<BM, BN, NWG, 32> co;
        lin_copy_offsets<BM, BN, NWG>(p, it.m0, it.end, n0, wl, lane, co);
        const int64_t wrow = p.gated ? n0 / 2 : n0;
        const int64_t e = p.mode == kByRows ? it.e : 0;
        const StepSrc src0 = {p.a + it.m0 * p.lda + (int64_t)it.k0 * kBK,
                              p.w + e * p.w_group + wrow * p.ldw + (int64_t)it.k0 * kBK,
                              p.as + it.m0 * p.ldas + it.k0 * 4,
                              p.ws + e * p.ws_group + wrow * p.ldws + it.k0 * 4};
        auto src_of = [&](int s) {
            int k = WGK * s + wk;
            k = WGK == 1 || k < it.steps ? k : it.steps - 1;
            return StepSrc{src0.a + (int64_t)k * kBK, src0.b + (int64_t)k * kBK, src0.as + k * 4, src0.bs + k * 4};
        };
        const int nsteps = (it.steps + WGK - 1) / WGK;
        const int valid = (it.steps - wk + WGK - 1) / WGK;
        if constexpr (EXACT)
            exact_mainloop<BM, BN, WGM, WGN, WGK, FA, FB, (WGK > 1)>(stage0, stage1, co, src_of, nsteps, valid, wk,
                                                                     wl, lane, acc);
        else
            native_mainloop<BM, BN, WGM, WGN, WGK, FA, FB>(stage0, stage1, co, src_of, nsteps, valid, wk, wl, lane,
                                                           acc);
    } else {
#pragma unroll
        for (int i = 0; i < GA; ++i)
#pragma unroll
            for (int g = 0; g < GB; ++g)
                acc[i][g] = v16f{};
    }
    __syncthreads();        // every wave has read its last fragments
    if constexpr (WGK == 1) {
        static_assert(NWG % 2 == 0 && NWG / 2 * kSlabBytes <= G::STAGE, "half the waves' slabs per stage");
        uint8_t* buf = (wave < NWG / 2 ? stage0 : stage1) + (wave % (NWG / 2)) * kSlabBytes;
        // one copy of the finishing code: only the accumulators' writes are
        // picked by the slab's number
        constexpr int kSlabs = GA * GB / 2;
#pragma unroll 1
        for (int t = 0; t < kSlabs; ++t) {
#pragma unroll
            for (int k = 0; k < kSlabs; ++k)
                if (t == k)
                    slab_write<GB>(buf, acc[k / (GB / 2)], k % (GB / 2) * 2, lane);
            // LDS operations of one wave complete in order, and the wave
            // reads back only what it wrote itself
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            slab_finish(p, buf, 1, 0, 0, 32, it.m0 + wm * TM + 32 * (t / (GB / 2)), it.end,
                        n0 + wn * TN + 64 * (t % (GB / 2)), it.e, lane);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    } else {
        static_assert(NWG == 1 && GB == 2 && WGK * kSlabBytes <= WGK * G::STAGE, "one slab per group and stage");
#pragma unroll
        for (int i = 0; i < GA; ++i) {
            uint8_t* st = i % 2 ? stage1 : stage0;
            if (i >= 2)
                __syncthreads();
            slab_write<GB>(st + wk * kSlabBytes, acc[i], 0, lane);
            __syncthreads();
            constexpr int kRows = 32 / WGK;
            slab_finish(p, st, WGK, kSlabBytes, wk * kRows, wk * kRows + kRows, it.m0 + 32 * i, it.end, n0, it.e, lane);
        }
    }
}

// ------------------------------------------------- few rows: skinny kernel --

// Up to 16 RT rows: the weights' bytes are the cost, and no row of w is used
// by a second wave, so they go straight from memory to registers in the
// MFMA's operand layout (lane l: row l % 16, K [16 q, +16) and [64 + 16 q,
// +16), q = l / 16), without LDS.  A work-group of NW waves takes NB blocks
// of 16 columns (gated: the first NB / 2 gate, the others up) and splits K
// over its waves in runs of K-steps; U steps' loads are in flight per wave
// before the first is multiplied.  The waves' sums are added in wave order
// through LDS, where the epilogue reads them row-wise.
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
    for (int s0 = lo; s0 < hi; s0 += U) {
        u32x4 wv[U][NB][2], av[U][RT][2];
        uint32_t wsv[U][NB], asv[U][RT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u < hi ? s0 + u : hi - 1;
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
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u >= hi)
                break;
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
                if (((s0 + u - lo) & 1) == 1 || s0 + u == hi - 1) {
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
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            *reinterpret_cast<v4f*>(red + (wave * BM + 16 * r + lr) * LD + 16 * b + 4 * lq) = tot[r][b];
    __syncthreads();
    const int per8 = width / 8;             // eights of outputs per row
    const int total = BM * per8;
    for (int i = tid; i - lane < total; i += NW * 64) {
        const int r = i < total ? i / per8 : BM - 1, c8 = i < total ? i % per8 : 0;
        float z[8], z1[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            z[u] = z1[u] = 0.f;
        for (int k = 0; k < NW; ++k) {
            const float* src = red + (k * BM + r) * LD + 8 * c8;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                z[u] += src[u];
            if (p.gated) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    z1[u] += src[BN / 2 + u];
            }
        }
        const int row = it.m0 + r, c = c0 + 8 * c8;
        finish8(p, it.e, row, c, cols, i < total && row < it.end && c < cols, z, z1, lane);
    }
}

// ------------------------------------------------------------------ launch --

template <int BM, int BN, int WGM, int WGN, int EWM, int EWN, int WGK, int FA, int FB>
static hipError_t launch_lin_tile(bool exact, const LinArgs& a, hipStream_t stream)
{
    if (exact) {
        if constexpr ((BM / EWM) * (BN / EWN) <= 64 * 64) {
            hipLaunchKernelGGL((linear_kernel<BM, BN, EWM, EWN, WGK, true, FA, FB>), dim3(a.total_work),
                               dim3(EWM * EWN * WGK * 64), 0, stream, a);
            return hipGetLastError();
        } else {
            return hipErrorInvalidValue;    // never planned
        }
    }
    hipLaunchKernelGGL((linear_kernel<BM, BN, WGM, WGN, WGK, false, FA, FB>), dim3(a.total_work),
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

// Blocks of 16 columns of a skinny tile (see lin_tile).
template <int FA, int FB>
hipError_t launch_linear_fmt(int cfg, bool exact, const LinArgs& a, hipStream_t stream)
{
    const int nb = lin_tile(cfg, a).tile_n / 16;
    switch (cfg) {
    case kLin256x256: return launch_lin_tile<256, 256, 2, 2, 2, 2, 1, FA, FB>(exact, a, stream);
    case kLin256x128: return launch_lin_tile<256, 128, 2, 2, 4, 2, 1, FA, FB>(exact, a, stream);
    case kLin128x128: return launch_lin_tile<128, 128, 2, 2, 2, 2, 1, FA, FB>(exact, a, stream);
    case kLin64x64: return launch_lin_tile<64, 64, 1, 1, 1, 1, 4, FA, FB>(exact, a, stream);
    case kLinRows64:
        return nb == 4 ? launch_lin_skinny<4, 4, 8, 1, FA, FB>(exact, a, stream)
                       : launch_lin_skinny<4, 2, 8, 2, FA, FB>(exact, a, stream);
    case kLinRows32:
        return nb == 4 ? launch_lin_skinny<2, 4, 8, 2, FA, FB>(exact, a, stream)
                       : launch_lin_skinny<2, 2, 8, 4, FA, FB>(exact, a, stream);
    case kLinRows16:
        return nb == 4 ? launch_lin_skinny<1, 4, 8, 4, FA, FB>(exact, a, stream)
                       : launch_lin_skinny<1, 2, 8, 4, FA, FB>(exact, a, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace mxg
