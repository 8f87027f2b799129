// Tokens sorted by expert and back.
#include "element.h"
#include "quant.h"

namespace mxg {

// ------------------------------------------------------------------ sort --
//
// Stable counting sort of the (token, choice) pairs by expert; a pair whose
// id is outside [0, experts) gets the key `experts` and so follows all
// others.  The row of pair i is
//   #{pairs with a smaller key} + #{earlier pairs with the same key}.
// A wave takes a run of consecutive pairs, 64 at a time: the lanes that hold
// the same key are found with one ballot per key bit, a pair's place among
// them is the number of lower lanes in that mask, and the wave's counter of
// the key moves on by the mask's size.  The counters of the waves before it
// (and, over several work-groups, of the work-groups before) are summed in
// between, so the order never depends on timing.  Bound by latency: one
// launch for few pairs, else two (count, place).  Measured: 32 pairs of 128
// experts 4.2 us, 16K pairs of 256 experts 9.5, 256K pairs 14.9, 8M pairs of
// 64 experts 144.

template <typename ID>
__device__ __forceinline__ uint32_t sort_key(const SortArgs& p, int64_t i)
{
    const ID id = static_cast<const ID*>(p.ids)[i];
    return id >= 0 && id < (ID)p.experts ? (uint32_t)id : (uint32_t)p.experts;
}

__device__ __forceinline__ uint64_t same_key(uint32_t key, bool valid, int bits)
{
    uint64_t m = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const bool one = (key >> b) & 1;
        const uint64_t v = __ballot(one);
        m &= one ? v : ~v;
    }
    return m;
}

enum { kSortAll, kSortCount, kSortPlace };

// A wave's share is p.iters pieces of 64 pairs.  ITERS >= p.iters: their keys
// and places stay in registers between the two passes; 0: any number of
// pieces, read and ranked twice.
template <int MODE, typename ID, int ITERS>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortArgs p)
{
    __shared__ uint32_t cnt[kSortWaves * (kSortMaxExperts + 1)];
    __shared__ uint32_t tot[kSortMaxExperts + 1], ktot[kSortMaxExperts + 1], before[kSortMaxExperts + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E1 = p.experts + 1;
    const int bits = 32 - __builtin_clz((unsigned)p.experts);   // keys 0 .. experts
    const int mine = wave * E1;                                 // the wave's counters
    const int64_t first = ((int64_t)blockIdx.x * kSortWaves + wave) * p.iters * 64;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    uint32_t key[ITERS > 0 ? ITERS : 1], local[ITERS > 0 ? ITERS : 1];
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        const int64_t i = first + it * 64 + lane;
        key[it] = it < p.iters && i < p.pairs ? sort_key<ID>(p, i) : 0;
    }
    for (int i = tid; i < kSortWaves * E1; i += kSortThreads)
        cnt[i] = 0;
    __syncthreads();

    // The place of a lane's key among the wave's so far; its counter moves
    // on.  One wave's LDS operations complete in order; the fences keep the
    // compiler's hands off.
    auto place = [&](uint32_t k, bool valid) __attribute__((always_inline)) {
        const uint64_t m = same_key(k, valid, bits);
        const int rank = __popcll(m & below);
        asm volatile("" ::: "memory");
        const uint32_t base = cnt[mine + k];
        asm volatile("" ::: "memory");
        if (valid && rank == 0)
            cnt[mine + k] = base + __popcll(m);
        asm volatile("" ::: "memory");
        return base + rank;
    };
#pragma unroll
    for (int it = 0; it < ITERS; ++it)
        if (it < p.iters)                           // the same for all lanes
            local[it] = place(key[it], first + it * 64 + lane < p.pairs);
    if (ITERS == 0)
        for (int it = 0; it < p.iters; ++it) {
            const int64_t i = first + (int64_t)it * 64 + lane;
            const bool valid = i < p.pairs;
            place(valid ? sort_key<ID>(p, i) : 0, valid);
        }
    __syncthreads();
    for (int e = tid; e < E1; e += kSortThreads) {
        uint32_t run = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t t = cnt[w * E1 + e];
            cnt[w * E1 + e] = run;
            run += t;
        }
        if (MODE == kSortCount)
            p.ws[(int64_t)blockIdx.x * E1 + e] = run;
        if (MODE == kSortAll) {
            tot[e] = run;
            before[e] = 0;
        }
        if (MODE == kSortPlace)
            tot[e] = before[e] = 0;
    }
    if (MODE == kSortCount)
        return;
    __syncthreads();
    if (MODE == kSortPlace) {
        // Sums over the work-groups of every key, and over those before this
        // one: the threads left over by the keys share the work-groups (sums
        // of counts: their order does not matter).
        const int parts = kSortThreads / E1 > 1 ? kSortThreads / E1 : 1;
        const int share = (p.blocks + parts - 1) / parts;
        for (int i = tid; i < parts * E1; i += kSortThreads) {
            const int e = i % E1;
            const int lo = i / E1 * share, hi = lo + share < p.blocks ? lo + share : p.blocks;
            uint32_t all = 0, pre = 0;
            for (int b0 = lo; b0 < hi; b0 += 16) {
                uint32_t n[16];
#pragma unroll
                for (int u = 0; u < 16; ++u)        // all in flight; past the end, the last again
                    n[u] = p.ws[(int64_t)(b0 + u < hi ? b0 + u : hi - 1) * E1 + e];
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    n[u] = b0 + u < hi ? n[u] : 0;
                    pre += b0 + u < (int)blockIdx.x ? n[u] : 0;
                    all += n[u];
                }
            }
            atomicAdd(&tot[e], all);
            atomicAdd(&before[e], pre);
        }
        __syncthreads();
    }
    if (wave == 0) {
        // exclusive sums over the experts, a run of them per lane
        const int per = (E1 + 63) / 64, lo = lane * per, hi = lo + per < E1 ? lo + per : E1;
        uint32_t s = 0, ks = 0;
        for (int e = lo; e < hi; ++e) {
            s += tot[e];
            ks += (tot[e] + kGroupK - 1) / kGroupK * kGroupK;
        }
        uint32_t inc = s, kinc = ks;
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t a = __shfl_up(inc, d), b = __shfl_up(kinc, d);
            if (lane >= d) {
                inc += a;
                kinc += b;
            }
        }
        s = inc - s;
        ks = kinc - ks;
        for (int e = lo; e < hi; ++e) {
            const uint32_t n = tot[e];
            tot[e] = s;
            ktot[e] = ks;
            s += n;
            ks += (n + kGroupK - 1) / kGroupK * kGroupK;
        }
    }
    __syncthreads();
    for (int e = tid; e < E1; e += kSortThreads) {
        const uint32_t base = tot[e] + before[e];
        for (int w = 0; w < kSortWaves; ++w)
            cnt[w * E1 + e] += base;
        if (blockIdx.x == 0) {
            p.offsets[e] = (int32_t)tot[e];
            p.k_offsets[e] = (int32_t)ktot[e];
        }
    }
    __syncthreads();
    auto put = [&](int64_t i, uint32_t row) __attribute__((always_inline)) {
        p.row_of[i] = (int32_t)row;
        p.pair_of[row] = (int32_t)i;
    };
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        const int64_t i = first + it * 64 + lane;
        if (it < p.iters && i < p.pairs)
            put(i, local[it] + cnt[mine + key[it]]);
    }
    if (ITERS == 0)
        for (int it = 0; it < p.iters; ++it) {
            const int64_t i = first + (int64_t)it * 64 + lane;
            const bool valid = i < p.pairs;
            const uint32_t row = place(valid ? sort_key<ID>(p, i) : 0, valid);
            if (valid)
                put(i, row);
        }
}

template <typename ID, int ITERS>
static void sort_launches(const SortArgs& a, hipStream_t stream)
{
    if (a.blocks == 1) {
        hipLaunchKernelGGL((sort_kernel<kSortAll, ID, ITERS>), dim3(1), dim3(kSortThreads), 0, stream, a);
        return;
    }
    hipLaunchKernelGGL((sort_kernel<kSortCount, ID, ITERS>), dim3(a.blocks), dim3(kSortThreads), 0, stream, a);
    hipLaunchKernelGGL((sort_kernel<kSortPlace, ID, ITERS>), dim3(a.blocks), dim3(kSortThreads), 0, stream, a);
}

template <typename ID>
static void sort_id(const SortArgs& a, hipStream_t stream)
{
    if (a.iters <= 1)
        sort_launches<ID, 1>(a, stream);
    else if (a.iters <= 4)
        sort_launches<ID, 4>(a, stream);
    else if (a.iters <= 16)
        sort_launches<ID, 16>(a, stream);
    else
        sort_launches<ID, 0>(a, stream);
}

hipError_t launch_sort(const SortArgs& a, hipStream_t stream)
{
    if (a.ids64)
        sort_id<int64_t>(a, stream);
    else
        sort_id<int32_t>(a, stream);
    return hipGetLastError();
}

// -------------------------------------------------------------- dispatch --
//
// One thread per piece of V elements of a token: read once, written to the
// rows of the token's k pairs (zero where the pair was dropped).  Bound by
// memory: tokens * cols read, tokens * k * cols written.  Measured: 5001 x 2047
// FP16 to 6 rows each, 42 us (143 MB, 3.4 TB/s: rows of odd length, so most
// 16-byte pieces lie across two lines).

// Kept rows, within the rows there are.
__device__ __forceinline__ int live_rows(const TokenArgs& p)
{
    const int live = *p.live;
    return live < 0 ? 0 : live < p.all_rows ? live : (int)p.all_rows;
}

// Token and piece of the thread (pieces per token); false past the last.
// Launches hold at most 2^31 threads.
__device__ __forceinline__ bool thread_piece(const TokenArgs& p, int pieces, int64_t& t, int& c)
{
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, q = i / (uint32_t)pieces;
    t = q;
    c = (int)(i - q * (uint32_t)pieces);
    return t < p.tokens;
}

template <int TYPE, int V>
__global__ void __launch_bounds__(256) dispatch_kernel(TokenArgs p, int pieces)
{
    typedef typename Element<TYPE>::T T;
    int64_t t;
    int piece;
    if (!thread_piece(p, pieces, t, piece))
        return;
    const int c = piece_start<V>(piece, p.cols);
    Pack<TYPE, V> v, none;
    v.load(static_cast<const T*>(p.x) + t * p.ld_x + c);
    none.zero();
    const int live = live_rows(p);
    const uint32_t rows = (uint32_t)p.all_rows;
    T* out = static_cast<T*>(p.out) + c;
#pragma unroll 4
    for (int j = 0; j < p.k; ++j) {
        const int r = p.row_of[t * p.k + j];
        if (r >= 0 && r < live)
            v.store(out + r * p.ld_out);
        else if ((uint32_t)r < rows)
            none.store(out + r * p.ld_out);
    }
}

// To MXFP8: two threads per block of 32, sixteen elements each; quantised
// once per token, the codes and scale byte written k times.  The rules are
// the quantiser's (a NaN makes the block's scale 0xFF and its codes 0x7F).
// Bound by memory: 8192 x 4096 bfloat16 to 8 rows each, 69 us (344 MB, 5.0
// TB/s; a large copy reaches 4.9).
template <int TYPE, int F>
__global__ void __launch_bounds__(256) dispatch_mx_kernel(TokenArgs p, int pieces)
{
    typedef typename Element<TYPE>::T T;
    int64_t t;
    int piece;
    if (!thread_piece(p, pieces, t, piece))     // pieces is even: both threads of a block leave together
        return;
    const int c = piece * 16;
    Pack<TYPE, 16> v;
    v.load(static_cast<const T*>(p.x) + t * p.ld_x + c);
    float f[16];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        f[u] = v.get(u);
        m = max(m, __float_as_uint(f[u]) & 0x7FFFFFFFu);
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    const MxScale sc = mx_scale<F>(m);
    u32x4 code;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        code[w] = mx_codes<F>(sc, f[4 * w], f[4 * w + 1], f[4 * w + 2], f[4 * w + 3]);
    const int live = live_rows(p);
    const uint32_t rows = (uint32_t)p.all_rows;
    uint8_t* q = p.q + c;
    uint8_t* s = p.s + (c >> 5);
#pragma unroll 4
    for (int j = 0; j < p.k; ++j) {
        const int r = p.row_of[t * p.k + j];
        if ((uint32_t)r >= rows)
            continue;
        const bool kept = r < live;
        *reinterpret_cast<u32x4*>(q + (int64_t)r * p.cols) = kept ? code : u32x4{0, 0, 0, 0};
        if ((piece & 1) == 0)
            s[(int64_t)r * (p.cols >> 5)] = kept ? sc.byte : 0;
    }
}

// --------------------------------------------------------------- combine --
//
// out[t] = residual[t] + sum over j, in order, of w[t, j] rows[row_of[t, j]],
// summed in FP32 and rounded once; dropped pairs add nothing (whatever their
// weight holds).  One thread per piece; eight rows' loads are in flight at a
// time.  Bound by memory.  The gradient of dispatch is the same sum with all
// weights one.  Measured: 8192 x 4096 bfloat16 from 8 rows each and a
// residual, 155 us (671 MB, 4.3 TB/s); one token 3.8 us.
template <int TYPE, int V>
__global__ void __launch_bounds__(256) combine_kernel(TokenArgs p, int pieces)
{
    typedef typename Element<TYPE>::T T;
    int64_t t;
    int piece;
    if (!thread_piece(p, pieces, t, piece))
        return;
    const int c = piece_start<V>(piece, p.cols);
    const int live = live_rows(p);
    const T* rows = static_cast<const T*>(p.rows) + c;
    float acc[V];
#pragma unroll
    for (int u = 0; u < V; ++u)
        acc[u] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        int r[8];
        float w[8];
        Pack<TYPE, V> v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t at = t * p.k + (j0 + j < p.k ? j0 + j : p.k - 1);
            r[j] = p.row_of[at];
            w[j] = p.weights ? p.weights[at] : 1.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < p.k && (uint32_t)r[j] < (uint32_t)live)
                v[j].load(rows + r[j] * p.ld_rows);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < p.k && (uint32_t)r[j] < (uint32_t)live) {
#pragma unroll
                for (int u = 0; u < V; ++u)
                    acc[u] += w[j] * v[j].get(u);
            }
    }
    Pack<TYPE, V> o;
    if (p.x) {
        Pack<TYPE, V> res;
        res.load(static_cast<const T*>(p.x) + t * p.ld_x + c);
#pragma unroll
        for (int u = 0; u < V; ++u)
            acc[u] += res.get(u);
    }
#pragma unroll
    for (int u = 0; u < V; ++u)
        o.put(u, acc[u]);
    o.store(static_cast<T*>(p.out) + t * p.ld_out + c);
}

// Gradients of combine: d_rows[row_of[t, j]] = w[t, j] d_out[t] (zero rows
// for dropped pairs) and d_w[t, j] = <rows[row_of[t, j]], d_out[t]>, summed
// in FP32 (zero for dropped pairs).  A work-group takes one token; a thread
// takes pieces threadIdx.x, + blockDim.x, ... of d_out and, for eight pairs
// at a time, the same pieces of their rows, so d_out is read once and every
// row once.  The partial dots are added over the lanes and then over the
// waves, in a fixed order.  Bound by memory: 8192 x 4096 bfloat16, 8 rows
// each, 274 us (1.14 GB, 4.1 TB/s).  Rows of few columns leave most of the
// threads without a piece: 16384 tokens x 128, one row each, 62 us where 13 MB
// move; x 512, two rows each, 78 us (84 MB).
template <int TYPE, int V>
__global__ void __launch_bounds__(256) combine_backward_kernel(TokenArgs p, int pieces)
{
    typedef typename Element<TYPE>::T T;
    __shared__ float part[4][8];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int live = live_rows(p);
    const uint32_t nrows = (uint32_t)p.all_rows;
    const T* d = static_cast<const T*>(p.x) + t * p.ld_x;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        int r[8];
        float w[8], dot[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t at = t * p.k + (j0 + j < p.k ? j0 + j : p.k - 1);
            r[j] = j0 + j < p.k ? p.row_of[at] : -1;
            w[j] = p.weights ? p.weights[at] : 1.f;
            dot[j] = 0.f;
        }
        for (int piece = threadIdx.x; piece < pieces; piece += blockDim.x) {
            const int c = piece_start<V>(piece, p.cols);
            const int fresh = piece * V - c;        // elements before it belong to the piece before
            Pack<TYPE, V> g, v[8];
            g.load(d + c);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((uint32_t)r[j] < (uint32_t)live)
                    v[j].load(static_cast<const T*>(p.rows) + r[j] * p.ld_rows + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if ((uint32_t)r[j] >= nrows)
                    continue;
                Pack<TYPE, V> o;
                o.zero();
                if (r[j] < live) {
#pragma unroll
                    for (int u = 0; u < V; ++u) {
                        const float gu = g.get(u);
                        if (u >= fresh)
                            dot[j] += v[j].get(u) * gu;
                        o.put(u, w[j] * gu);
                    }
                }
                o.store(static_cast<T*>(p.out) + r[j] * p.ld_out + c);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            for (int s = 32; s > 0; s >>= 1)
                dot[j] += __shfl_xor(dot[j], s);
            if (lane == 0)
                part[wave][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < 8 && j0 + (int)threadIdx.x < p.k) {
            float sum = part[0][threadIdx.x];
            for (int i = 1; i < waves; ++i)
                sum += part[i][threadIdx.x];
            p.d_weights[t * p.k + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- launch --

// launch(p, work-groups) for ranges of tokens with at most 2^31 threads each,
// `per_token` threads a token in work-groups of `group`: the runtime takes a
// grid of 2^32 threads or more modulo 2^32, without an error.  x, d_weights
// and the k-wide arrays are tokens' own; out is where `out_by_token`.
template <class Launch>
static hipError_t by_ranges(const TokenArgs& a, int element, bool out_by_token, int per_token, int group,
                            const Launch& launch)
{
    const int64_t most = (1LL << 31) / per_token;
    for (int64_t t = 0; t < a.tokens; t += most) {
        TokenArgs p = a;
        p.tokens = a.tokens - t < most ? a.tokens - t : most;
        p.row_of += t * a.k;
        p.x = a.x ? static_cast<const char*>(a.x) + t * a.ld_x * element : nullptr;
        p.weights = a.weights ? a.weights + t * a.k : nullptr;
        p.d_weights = a.d_weights ? a.d_weights + t * a.k : nullptr;
        if (out_by_token)
            p.out = static_cast<char*>(a.out) + t * a.ld_out * element;
        launch(p, (unsigned)((p.tokens * per_token + group - 1) / group));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// Threads of 256 per token for pieces of V elements, and the launch of a
// kernel that takes them so.
#define MXG_LAUNCH_PIECES(kernel, V, element, out_by_token)                                               \
    do {                                                                                                  \
        const int pieces = (a.cols + V - 1) / V;                                                          \
        return by_ranges(a, element, out_by_token, pieces, 256, [&](const TokenArgs& p, unsigned groups) { \
            hipLaunchKernelGGL(kernel, dim3(groups), dim3(256), 0, stream, p, pieces);                    \
        });                                                                                               \
    } while (0)

template <int TYPE>
static hipError_t dispatch_type(const TokenArgs& a, hipStream_t stream)
{
    constexpr int element = sizeof(typename Element<TYPE>::T);
    if (a.cols >= 8)
        MXG_LAUNCH_PIECES((dispatch_kernel<TYPE, 8>), 8, element, false);
    MXG_LAUNCH_PIECES((dispatch_kernel<TYPE, 1>), 1, element, false);
}

template <int TYPE>
static hipError_t dispatch_mx_type(const TokenArgs& a, hipStream_t stream)
{
    constexpr int element = sizeof(typename Element<TYPE>::T);
    if (a.fmt == kE5M2)
        MXG_LAUNCH_PIECES((dispatch_mx_kernel<TYPE, kE5M2>), 16, element, false);
    MXG_LAUNCH_PIECES((dispatch_mx_kernel<TYPE, kE4M3>), 16, element, false);
}

template <int TYPE>
static hipError_t combine_type(const TokenArgs& a, hipStream_t stream)
{
    constexpr int element = sizeof(typename Element<TYPE>::T);
    if (a.cols >= 8)
        MXG_LAUNCH_PIECES((combine_kernel<TYPE, 8>), 8, element, true);
    MXG_LAUNCH_PIECES((combine_kernel<TYPE, 1>), 1, element, true);
}

template <int TYPE>
static hipError_t combine_backward_type(const TokenArgs& a, hipStream_t stream)
{
    constexpr int element = sizeof(typename Element<TYPE>::T);
    if (a.cols >= 8)
        return by_ranges(a, element, false, 256, 256, [&](const TokenArgs& p, unsigned groups) {
            hipLaunchKernelGGL((combine_backward_kernel<TYPE, 8>), dim3(groups), dim3(256), 0, stream, p,
                               (a.cols + 7) / 8);
        });
    return by_ranges(a, element, false, 64, 64, [&](const TokenArgs& p, unsigned groups) {
        hipLaunchKernelGGL((combine_backward_kernel<TYPE, 1>), dim3(groups), dim3(64), 0, stream, p, a.cols);
    });
}

#define MXG_BY_TYPE(name)                                                       \
    hipError_t launch_##name(const TokenArgs& a, int type, hipStream_t stream) \
    {                                                                           \
        switch (type) {                                                         \
        case kBF16: return name##_type<kBF16>(a, stream);                       \
        case kFP16: return name##_type<kFP16>(a, stream);                       \
        case kFP32: return name##_type<kFP32>(a, stream);                       \
        default: return hipErrorInvalidValue;                                   \
        }                                                                       \
    }

MXG_BY_TYPE(dispatch)
MXG_BY_TYPE(dispatch_mx)
MXG_BY_TYPE(combine)
MXG_BY_TYPE(combine_backward)

}  // namespace mxg
