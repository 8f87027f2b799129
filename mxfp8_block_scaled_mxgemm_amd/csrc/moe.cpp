// Host side of the expert layer: argument rules, the choice of tiles, and the
// C ABI of include/mxgemm_moe.h.
#include "mxgemm_moe.h"

#include <hip/hip_runtime.h>

#include <math.h>
#include <string.h>

#include <atomic>

#include "host_util.h"
#include "linear.h"
#include "moe.h"
#include "schedule.h"

using mxg::fail;

namespace mxg {

template <int FA, int FB>
hipError_t launch_linear_fmt(int cfg, bool exact, const LinArgs& a, hipStream_t stream);
extern template hipError_t launch_linear_fmt<0, 0>(int, bool, const LinArgs&, hipStream_t);
extern template hipError_t launch_linear_fmt<0, 1>(int, bool, const LinArgs&, hipStream_t);
extern template hipError_t launch_linear_fmt<1, 0>(int, bool, const LinArgs&, hipStream_t);
extern template hipError_t launch_linear_fmt<1, 1>(int, bool, const LinArgs&, hipStream_t);

hipError_t launch_linear(int cfg, bool exact, int fa, int fw, const LinArgs& a, hipStream_t stream)
{
    if (fa == 0)
        return fw == 0 ? launch_linear_fmt<0, 0>(cfg, exact, a, stream) : launch_linear_fmt<0, 1>(cfg, exact, a, stream);
    return fw == 0 ? launch_linear_fmt<1, 0>(cfg, exact, a, stream) : launch_linear_fmt<1, 1>(cfg, exact, a, stream);
}

LinTile lin_tile(int cfg, const LinArgs& a)
{
    const int few = a.skinny == kSkinnyWide ? 64 : a.skinny == kSkinnyNarrow ? 16 : 32;
    const int threads = a.skinny == kSkinnyNarrow ? 1024 : a.skinny == kSkinny8 ? 512 : a.skinny == kSkinny2 ? 128 : 256;
    switch (cfg) {
    case kLin256x256: return {256, 256, 256};
    case kLin128x128: return {128, 128, 256};
    case kLin64x64: return {64, 64, 256};
    case kLinRows32: return {32, few, threads};
    default: return {16, few, threads};
    }
}

}  // namespace mxg

namespace {

constexpr int kMaxDevices = 64;

// Compute units of the current device, which must be a gfx950; looked up
// once per device.
int current_device(int* dev, int* cus)
{
    static std::atomic<int> known[kMaxDevices];     // 0: not looked up, else compute units
    HIP_TRY(hipGetDevice(dev));
    if (*dev < 0 || *dev >= kMaxDevices)
        return fail(MXGEMM_EUNSUPPORTED, "device index %d out of range", *dev);
    *cus = known[*dev].load(std::memory_order_relaxed);
    if (*cus == 0) {
        hipDeviceProp_t prop;
        HIP_TRY(hipGetDeviceProperties(&prop, *dev));
        if (strncmp(prop.gcnArchName, "gfx950", 6) != 0)
            return fail(MXGEMM_EUNSUPPORTED, "device %d is %s; this library is built for gfx950", *dev,
                        prop.gcnArchName);
        *cus = prop.multiProcessorCount;
        known[*dev].store(*cus, std::memory_order_relaxed);
    }
    return MXGEMM_OK;
}

struct Buffer {
    const void* p;
    const char* name;
    int align;
    bool optional;
};

template <size_t N>
int check_buffers(const Buffer (&b)[N], int dev)
{
    for (const Buffer& x : b) {
        if (!x.p) {
            if (x.optional)
                continue;
            return fail(MXGEMM_EINVAL, "%s is NULL", x.name);
        }
        if ((uintptr_t)x.p % x.align != 0)
            return fail(MXGEMM_EINVAL, "%s must be %d-byte aligned", x.name, x.align);
        const int rc = mxg::gpu_accessible(x.p, x.name, dev);
        if (rc != MXGEMM_OK)
            return rc;
    }
    return MXGEMM_OK;
}

int element_size(int type) { return type == MXGEMM_TYPE_FP32 ? 4 : 2; }

// -------------------------------------------------------------- tokens -----

// One work-group sorts up to this many pairs in one launch; more are spread
// over work-groups in two.  Measured with 256 experts: 4096 pairs 8.1 us in
// one, about 9 in two; 8192 pairs 13.6 and 9.5; 16384 pairs 22.5 and 9.5.
constexpr int64_t kSortOneBlock = 4 * 1024;

int sort_blocks(int64_t pairs, int* iters)
{
    const int64_t per_iter = mxg::kSortThreads;
    if (pairs <= kSortOneBlock) {
        *iters = (int)((pairs + per_iter - 1) / per_iter);
        return 1;
    }
    int64_t it = (pairs + per_iter * mxg::kSortMaxBlocks - 1) / (per_iter * mxg::kSortMaxBlocks);
    *iters = (int)it;
    return (int)((pairs + per_iter * it - 1) / (per_iter * it));
}

int check_pairs(int64_t tokens, int32_t k, int32_t experts)
{
    if (tokens < 0 || k < 1 || experts < 1)
        return fail(MXGEMM_EINVAL, "tokens %lld must not be negative, k %d and experts %d must be positive",
                    (long long)tokens, k, experts);
    // a little below 2^31: the sort's last work-group counts past the end
    if (tokens > ((1LL << 31) - (1LL << 20)) / k)
        return fail(MXGEMM_EUNSUPPORTED, "%lld tokens x %d pairs exceed 2^31 - 2^20", (long long)tokens, k);
    if (experts > mxg::kSortMaxExperts)
        return fail(MXGEMM_EUNSUPPORTED, "%d experts exceed %d", experts, mxg::kSortMaxExperts);
    return MXGEMM_OK;
}

int token_args(mxg::TokenArgs* a, int32_t type, int64_t tokens, int32_t k, int64_t cols, const int32_t* offsets,
               int32_t experts, const int32_t* row_of)
{
    int rc = check_pairs(tokens, k, experts);
    if (rc != MXGEMM_OK)
        return rc;
    if (type < MXGEMM_TYPE_BF16 || type > MXGEMM_TYPE_FP32)
        return fail(MXGEMM_EINVAL, "unknown element type %d", type);
    if (cols < 1)
        return fail(MXGEMM_EINVAL, "cols %lld must be positive", (long long)cols);
    // one thread per eight elements, at most 128 launches of 2^31
    if (cols > (1 << 24) || (cols + 7) / 8 * tokens > (1LL << 38))
        return fail(MXGEMM_EUNSUPPORTED, "%lld tokens of %lld columns are too many", (long long)tokens,
                    (long long)cols);
    memset(a, 0, sizeof(*a));
    a->tokens = tokens;
    a->all_rows = tokens * k;
    a->k = k;
    a->cols = (int)cols;
    a->live = offsets + experts;
    a->row_of = row_of;
    return MXGEMM_OK;
}

int check_stride(const char* name, int64_t ld, int64_t cols)
{
    if (ld < cols)
        return fail(MXGEMM_EINVAL, "row stride %lld of %s is less than its %lld columns", (long long)ld, name,
                    (long long)cols);
    return MXGEMM_OK;
}

#define TRY(expr)                 \
    do {                          \
        const int rc_ = (expr);   \
        if (rc_ != MXGEMM_OK)     \
            return rc_;           \
    } while (0)

// -------------------------------------------------------------- product ----

// The tile configuration for a product.  Few rows (of an average expert):
// the weights' bytes are the cost, and the skinny kernel streams them (4 rows
// per expert, 64 tokens x 8 over 128 experts, 2048 x 768: 52 us).  An expert
// with more rows than the tile reads its weights again, so from 8 rows per
// expert on the 128 x 128 tiles stream them better (native, 64 x 8 over 64,
// 4096 x 4096: 250 us against 351; exact, 299 against 356).  Dense, 32 x 2048
// x 7168: 17.8 against 21.9 us with 64 x 64 tiles whose K is not split; 64 rows:
// 31 against 24 us.  (With K split, which needs a workspace and is offered from
// 33 rows on, 33 rows take 16.7 us and 64 rows 17.2, where 32 take 18.5 and 16
// take 14.5: between 17 and 32 rows of a long K the limit is not the best one.)
// Otherwise 128 x 128 tiles, two of whose work-groups share a compute unit (the
// epilogue of one runs beside the K loop of the other), where they occupy more
// than half of the compute units (1024 x 2048 x 4096, 128 tiles: 35 against 31
// us with 64 x 64 ones, exact).  Native dense products of a long K take 256 x
// 256 tiles, which ask the L2 for half the bytes: 8192 x 8192 x 8192, 472
// against 592 us; x 2048, 161 against 169; x 512, 93 against 76.  By expert
// they need rows enough to end few tiles early and four tiles per compute
// unit, since one work-group has it whole: 32 experts of 2048 rows, 4096 x
// 4096, 1224 against 1449 us; of 1024 rows, 644 against 757, and 381 against
// 411 at K 2048; of 512 rows, 393 against 410, 245 against 228 at K 2048; 4
// experts of 2048 rows, 180 against 178.
int choose_tile(const mxg::LinArgs& a, bool exact, int cus)
{
    const bool by = a.mode == mxg::kByRows;
    const int64_t r = by ? (a.rows + a.groups - 1) / a.groups : a.rows;
    if (r <= (by ? 6 : 16))
        return mxg::kLinRows16;
    if (r <= 32 && !by)
        return mxg::kLinRows32;
    auto tiles = [&](int64_t m, int64_t n) {
        return (a.mode == mxg::kDense ? 1 : a.groups) * ((r + m - 1) / m) * ((a.N + n - 1) / n);
    };
    if (!exact && a.K >= 2048 && (a.mode == mxg::kDense ? tiles(256, 256) >= cus
                                                        : by && r >= 1024 && tiles(256, 256) >= 4 * cus))
        return mxg::kLin256x256;
    return tiles(128, 128) > cus / 2 ? mxg::kLin128x128 : mxg::kLin64x64;
}

// K splits of a dense product of 64 x 64 tiles: as many work-groups as
// compute units, each with two K-steps at least for each of its four groups.
// (64 x 2048 x 7168 exact, 32 tiles: 24 us unsplit.)
int choose_split(const mxg::LinArgs& a, int cus)
{
    const int64_t tiles = (int64_t)((a.rows + 63) / 64) * ((a.N + 63) / 64);
    int64_t s = cus / tiles;
    const int64_t most = a.K / mxg::kGroupK / 8;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s);
}

// Sums of all splits; no more than the 64 x 64 tiles of every compute unit.
int64_t split_bytes(const mxg::LinArgs& a, int split) { return (int64_t)split * a.rows * a.N * 4; }

int check_linear(const mxgemm_linear_t* g, mxg::LinArgs* a)
{
    if (g->rows < 0 || g->N < 1 || g->K < 1)
        return fail(MXGEMM_EINVAL, "rows %lld must not be negative, N %lld and K %lld must be positive",
                    (long long)g->rows, (long long)g->N, (long long)g->K);
    if (g->K % 32 != 0)
        return fail(MXGEMM_EINVAL, "K %lld must be a multiple of the MX block 32", (long long)g->K);
    if (g->K % 128 != 0)
        return fail(MXGEMM_EUNSUPPORTED, "K %lld must be a multiple of 128 (one MFMA K-step) in this build",
                    (long long)g->K);
    if (g->K > (1 << 30) || g->N >= (1LL << 31) - 1024 || g->rows >= (1LL << 31) - 1024)
        return fail(MXGEMM_EUNSUPPORTED, "problem too large for 32-bit indexes");
    if (g->mode < MXGEMM_GROUP_NONE || g->mode > MXGEMM_GROUP_INNER)
        return fail(MXGEMM_EINVAL, "unknown group mode %d", g->mode);
    if (g->mode != MXGEMM_GROUP_NONE && (g->experts < 1 || !g->offsets))
        return fail(MXGEMM_EINVAL, "a product by expert needs experts and offsets");
    if (g->mode != MXGEMM_GROUP_NONE && g->experts > (1 << 20))
        return fail(MXGEMM_EUNSUPPORTED, "%d experts exceed 2^20", g->experts);
    if (g->act < MXGEMM_ACT_NONE || g->act > MXGEMM_ACT_SILU)
        return fail(MXGEMM_EINVAL, "unknown activation %d", g->act);
    if (g->out_type < MXGEMM_TYPE_BF16 || g->out_type > MXGEMM_TYPE_MXE5M2)
        return fail(MXGEMM_EINVAL, "unknown output type %d", g->out_type);
    if (g->bias && (g->bias_type < MXGEMM_TYPE_BF16 || g->bias_type > MXGEMM_TYPE_FP32))
        return fail(MXGEMM_EINVAL, "unknown bias type %d", g->bias_type);
    if ((g->a_format | g->w_format) & ~1)
        return fail(MXGEMM_EINVAL, "unknown FP8 format (a %d, w %d)", g->a_format, g->w_format);
    if (g->precision != MXGEMM_PRECISION_EXACT && g->precision != MXGEMM_PRECISION_NATIVE)
        return fail(MXGEMM_EINVAL, "unknown precision mode %d", g->precision);
    if (g->gated && g->N % 2 != 0)
        return fail(MXGEMM_EINVAL, "a gated product needs an even N, not %lld", (long long)g->N);
    const bool mx = g->out_type >= MXGEMM_TYPE_MXE4M3;
    const int64_t cols = g->gated ? g->N / 2 : g->N;
    if (g->mode == MXGEMM_GROUP_INNER && (g->bias || g->act || g->gated || g->residual || g->z || mx))
        return fail(MXGEMM_EINVAL, "GROUP_INNER takes no epilogue and no MXFP8 output");
    if (mx && (cols % 32 != 0 || g->ld_out % 8 != 0))
        return fail(MXGEMM_EINVAL, "MXFP8 output needs columns (%lld) in blocks of 32 and rows 8 bytes apart",
                    (long long)cols);
    if (mx && g->ld_out_scale < cols / 32)
        return fail(MXGEMM_EINVAL, "ld_out_scale %lld is less than %lld", (long long)g->ld_out_scale,
                    (long long)(cols / 32));
    TRY(check_stride("a", g->lda, g->K));
    TRY(check_stride("a_scale", g->ld_a_scale, g->K / 32));
    TRY(check_stride("w", g->ldw, g->K));
    TRY(check_stride("w_scale", g->ld_w_scale, g->K / 32));
    TRY(check_stride("out", g->ld_out, cols));
    if (g->residual)
        TRY(check_stride("residual", g->ld_residual, cols));
    if (g->z)
        TRY(check_stride("z", g->ld_z, g->N));
    if (g->lda % 16 || g->ldw % 16 || g->w_group % 16)
        return fail(MXGEMM_EINVAL, "strides of a and w must be multiples of 16 bytes");
    if (g->ld_a_scale % 4 || g->ld_w_scale % 4 || g->w_scale_group % 4)
        return fail(MXGEMM_EINVAL, "strides of a_scale and w_scale must be multiples of 4 bytes");
    if (g->lda > (1 << 30) / 256 * 2 || g->ldw > (1 << 30) / 256 * 2 || g->ld_a_scale > (1 << 22) ||
        g->ld_w_scale > (1 << 22))
        return fail(MXGEMM_EUNSUPPORTED, "row strides of the operands are limited to 8 MiB (scales 4 MiB)");
    if (g->gated && ((g->N / 2 + 256) * g->ldw >= (1LL << 32) || (g->N / 2 + 256) * g->ld_w_scale >= (1LL << 32)))
        return fail(MXGEMM_EUNSUPPORTED, "gated weights (or their scales) of 4 GiB or more per expert");
    memset(a, 0, sizeof(*a));
    a->a = (const uint8_t*)g->a;
    a->as = (const uint8_t*)g->a_scale;
    a->w = (const uint8_t*)g->w;
    a->ws = (const uint8_t*)g->w_scale;
    a->lda = g->lda;
    a->ldas = g->ld_a_scale;
    a->ldw = g->ldw;
    a->ldws = g->ld_w_scale;
    a->w_group = g->w_group;
    a->ws_group = g->w_scale_group;
    a->offsets = g->offsets;
    a->mode = g->mode;
    a->groups = g->mode == MXGEMM_GROUP_NONE ? 0 : g->experts;
    a->rows = (int)g->rows;
    a->N = (int)g->N;
    a->K = (int)g->K;
    a->bias = g->bias;
    a->bias_type = g->bias_type;
    a->act = g->act;
    a->gated = g->gated ? 1 : 0;
    a->residual = g->residual;
    a->ld_res = g->ld_residual;
    a->out = g->out;
    a->ld_out = g->ld_out;
    a->out_group = g->out_group;
    a->out_type = g->out_type;
    a->out_s = (uint8_t*)g->out_scale;
    a->ld_out_s = g->ld_out_scale;
    a->z = (uint16_t*)g->z;
    a->ld_z = g->ld_z;
    return MXGEMM_OK;
}

// Tiles of configuration cfg and their order.
int plan_linear(mxg::LinArgs* a, int cfg, int cus, int64_t workspace_bytes)
{
    a->split = 1;
    if (cfg == mxg::kLin64x64 && a->mode == mxg::kDense) {
        const int split = choose_split(*a, cus);
        if (split_bytes(*a, split) <= workspace_bytes)
            a->split = split;
    }
    // Skinny tiles (measurements at their launch): few tiles of a long K take
    // many waves each; many short ones are better as small work-groups
    a->skinny = mxg::kSkinny8;
    if (a->gated && a->out_type >= mxg::kMxE4M3)
        a->skinny = mxg::kSkinnyWide;
    else if (a->mode == mxg::kDense && !a->gated && a->out_type < mxg::kMxE4M3 && (a->N + 31) / 32 < cus)
        a->skinny = mxg::kSkinnyNarrow;
    else if (a->mode != mxg::kDense)
        a->skinny = a->K <= 8 * mxg::kGroupK ? mxg::kSkinny2 : mxg::kSkinny4;
    const mxg::LinTile t = mxg::lin_tile(cfg, *a);
    int64_t tiles_m = ((int64_t)a->rows + t.tile_m - 1) / t.tile_m;
    if (a->mode == mxg::kByRows)    // every expert, and the rows of none, may end inside a tile
        tiles_m = a->rows / t.tile_m + (a->groups + 1 < a->rows ? a->groups + 1 : a->rows);
    const int64_t tiles_n = ((int64_t)a->N + t.tile_n - 1) / t.tile_n;
    int64_t work = tiles_m * tiles_n * a->split;
    if (a->mode == mxg::kByInner)   // equal shares of the tiles for the XCDs, of every expert
        work = (work + mxg::kNumXcd - 1) / mxg::kNumXcd * mxg::kNumXcd * a->groups;
    else if (a->mode == mxg::kByRows)
        work = (work + mxg::kNumXcd - 1) / mxg::kNumXcd * mxg::kNumXcd;
    // (the runtime would take a larger grid modulo 2^32 threads, without an error)
    if (work >= (1LL << 32) / t.threads)
        return fail(MXGEMM_EUNSUPPORTED, "%lld work-groups of %d threads are too many for one launch", (long long)work,
                    t.threads);
    a->tiles_m = (int)tiles_m;
    a->tiles_n = (int)tiles_n;
    a->total_work = (int)work;
    // group width: about a square patch of tiles per XCD per round of
    // resident work-groups; skinny tiles share no rows of w, so theirs run
    // along N
    const int64_t per_xcd = ((work < cus ? work : cus) + mxg::kNumXcd - 1) / mxg::kNumXcd / a->split;
    int64_t g = (int64_t)floor(sqrt((double)(per_xcd > 1 ? per_xcd : 1)));
    if (cfg >= mxg::kLinRows32)
        g = tiles_n;
    a->group_n = (int)(g < 1 ? 1 : g > tiles_n ? tiles_n : g);
    return MXGEMM_OK;
}

}  // namespace

extern "C" {

int64_t mxgemm_sort_tokens_workspace(int64_t tokens, int32_t k, int32_t experts)
{
    if (check_pairs(tokens, k, experts) != MXGEMM_OK)
        return 0;
    int iters;
    const int blocks = sort_blocks(tokens * k, &iters);
    return blocks > 1 ? (int64_t)blocks * (experts + 1) * 4 : 0;
}

int mxgemm_sort_tokens(const void* ids, int32_t id_bytes, int64_t tokens, int32_t k, int32_t experts,
                       int32_t* offsets, int32_t* k_offsets, int32_t* row_of, int32_t* pair_of, void* workspace,
                       int64_t workspace_bytes, void* stream)
{
    TRY(check_pairs(tokens, k, experts));
    if (id_bytes != 4 && id_bytes != 8)
        return fail(MXGEMM_EINVAL, "id_bytes %d must be 4 or 8", id_bytes);
    int dev, cus;
    TRY(current_device(&dev, &cus));
    mxg::SortArgs a;
    a.blocks = sort_blocks(tokens * k, &a.iters);
    const int64_t need = a.blocks > 1 ? (int64_t)a.blocks * (experts + 1) * 4 : 0;
    if (workspace_bytes < need)
        return fail(MXGEMM_EINVAL, "workspace of %lld bytes is less than %lld", (long long)workspace_bytes,
                    (long long)need);
    const bool none = tokens == 0;
    const Buffer bufs[] = {{ids, "ids", id_bytes, none},       {offsets, "offsets", 4, false},
                           {k_offsets, "k_offsets", 4, false}, {row_of, "row_of", 4, none},
                           {pair_of, "pair_of", 4, none},      {need ? workspace : nullptr, "workspace", 4, need == 0}};
    TRY(check_buffers(bufs, dev));
    a.ids = ids;
    a.pairs = tokens * k;
    a.experts = experts;
    a.ids64 = id_bytes == 8;
    a.offsets = offsets;
    a.k_offsets = k_offsets;
    a.row_of = row_of;
    a.pair_of = pair_of;
    a.ws = (uint32_t*)workspace;
    HIP_TRY(mxg::launch_sort(a, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_dispatch_tokens(const void* x, int64_t ld_x, int32_t type, int64_t tokens, int32_t k, int64_t cols,
                           const int32_t* offsets, int32_t experts, const int32_t* row_of, void* rows,
                           int64_t ld_rows, void* stream)
{
    mxg::TokenArgs a;
    TRY(token_args(&a, type, tokens, k, cols, offsets, experts, row_of));
    TRY(check_stride("x", ld_x, cols));
    TRY(check_stride("rows", ld_rows, cols));
    if (tokens == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const int size = element_size(type);
    const Buffer bufs[] = {{x, "x", size, false}, {offsets, "offsets", 4, false}, {row_of, "row_of", 4, false},
                           {rows, "rows", size, false}};
    TRY(check_buffers(bufs, dev));
    a.x = x;
    a.ld_x = ld_x;
    a.out = rows;
    a.ld_out = ld_rows;
    HIP_TRY(mxg::launch_dispatch(a, type, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_dispatch_tokens_mx(const void* x, int64_t ld_x, int32_t type, int64_t tokens, int32_t k, int64_t cols,
                              const int32_t* offsets, int32_t experts, const int32_t* row_of, uint8_t* q, uint8_t* s,
                              int32_t format, void* stream)
{
    mxg::TokenArgs a;
    TRY(token_args(&a, type, tokens, k, cols, offsets, experts, row_of));
    TRY(check_stride("x", ld_x, cols));
    if (cols % 32 != 0)
        return fail(MXGEMM_EINVAL, "cols %lld must be a multiple of the MX block 32", (long long)cols);
    if (format != MXGEMM_FMT_E4M3 && format != MXGEMM_FMT_E5M2)
        return fail(MXGEMM_EINVAL, "unknown FP8 format %d", format);
    if (tokens == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const Buffer bufs[] = {{x, "x", element_size(type), false}, {offsets, "offsets", 4, false},
                           {row_of, "row_of", 4, false}, {q, "q", 16, false}, {s, "s", 1, false}};
    TRY(check_buffers(bufs, dev));
    a.x = x;
    a.ld_x = ld_x;
    a.q = q;
    a.s = s;
    a.fmt = format;
    HIP_TRY(mxg::launch_dispatch_mx(a, type, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_combine_tokens(const void* rows, int64_t ld_rows, int32_t type, int64_t tokens, int32_t k, int64_t cols,
                          const int32_t* offsets, int32_t experts, const int32_t* row_of, const float* weights,
                          const void* residual, int64_t ld_residual, void* out, int64_t ld_out, void* stream)
{
    mxg::TokenArgs a;
    TRY(token_args(&a, type, tokens, k, cols, offsets, experts, row_of));
    TRY(check_stride("rows", ld_rows, cols));
    TRY(check_stride("out", ld_out, cols));
    if (residual)
        TRY(check_stride("residual", ld_residual, cols));
    if (tokens == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const int size = element_size(type);
    const Buffer bufs[] = {{rows, "rows", size, false},         {offsets, "offsets", 4, false},
                           {row_of, "row_of", 4, false},        {weights, "weights", 4, true},
                           {residual, "residual", size, true},  {out, "out", size, false}};
    TRY(check_buffers(bufs, dev));
    a.rows = rows;
    a.ld_rows = ld_rows;
    a.weights = weights;
    a.x = residual;
    a.ld_x = ld_residual;
    a.out = out;
    a.ld_out = ld_out;
    HIP_TRY(mxg::launch_combine(a, type, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_combine_tokens_backward(const void* d_out, int64_t ld_d_out, const void* rows, int64_t ld_rows,
                                   int32_t type, int64_t tokens, int32_t k, int64_t cols, const int32_t* offsets,
                                   int32_t experts, const int32_t* row_of, const float* weights, void* d_rows,
                                   int64_t ld_d_rows, float* d_weights, void* stream)
{
    mxg::TokenArgs a;
    TRY(token_args(&a, type, tokens, k, cols, offsets, experts, row_of));
    TRY(check_stride("d_out", ld_d_out, cols));
    TRY(check_stride("rows", ld_rows, cols));
    TRY(check_stride("d_rows", ld_d_rows, cols));
    if (tokens == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const int size = element_size(type);
    const Buffer bufs[] = {{d_out, "d_out", size, false}, {rows, "rows", size, false},
                           {offsets, "offsets", 4, false}, {row_of, "row_of", 4, false},
                           {weights, "weights", 4, true}, {d_rows, "d_rows", size, false},
                           {d_weights, "d_weights", 4, false}};
    TRY(check_buffers(bufs, dev));
    a.x = d_out;
    a.ld_x = ld_d_out;
    a.rows = rows;
    a.ld_rows = ld_rows;
    a.weights = weights;
    a.out = d_rows;
    a.ld_out = ld_d_rows;
    a.d_weights = d_weights;
    HIP_TRY(mxg::launch_combine_backward(a, type, (hipStream_t)stream));
    return MXGEMM_OK;
}

int64_t mxgemm_linear_workspace(int64_t rows, int64_t N, int64_t K)
{
    // sums of at most one 64 x 64 tile per compute unit
    if (rows < 1 || N < 1 || K < 2048 || (rows + 63) / 64 * ((N + 63) / 64) > 128 || rows <= 32)
        return 0;
    return 256LL * 64 * 64 * 4;
}

int mxgemm_linear(const mxgemm_linear_t* args, void* stream)
{
    if (!args)
        return fail(MXGEMM_EINVAL, "args is NULL");
    mxg::LinArgs a;
    TRY(check_linear(args, &a));
    const bool exact = args->precision == MXGEMM_PRECISION_EXACT;
    const bool mx = args->out_type >= MXGEMM_TYPE_MXE4M3;
    if (args->tile_cfg >= mxg::kLinCfgs || (exact && args->tile_cfg == mxg::kLin256x256))
        return fail(MXGEMM_EINVAL, "tile_cfg %d has no kernel for this precision mode", args->tile_cfg);
    if (args->rows == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const int size = mx ? 8 : element_size(args->out_type);
    const Buffer bufs[] = {{args->a, "a", 16, false},
                           {args->a_scale, "a_scale", 4, false},
                           {args->w, "w", 16, false},
                           {args->w_scale, "w_scale", 4, false},
                           {args->bias, "bias", element_size(args->bias_type), true},
                           {args->residual, "residual", mx ? 2 : size, true},
                           {args->out, "out", size, false},
                           {mx ? args->out_scale : nullptr, "out_scale", 1, !mx},
                           {args->z, "z", 2, true},
                           {args->workspace, "workspace", 16, true},
                           {a.groups ? args->offsets : nullptr, "offsets", 4, true}};
    TRY(check_buffers(bufs, dev));
    const int cfg = args->tile_cfg >= 0 ? args->tile_cfg : choose_tile(a, exact, cus);
    TRY(plan_linear(&a, cfg, cus, args->workspace ? args->workspace_bytes : 0));
    a.part = (float*)args->workspace;
    HIP_TRY(mxg::launch_linear(cfg, exact, args->a_format, args->w_format, a, (hipStream_t)stream));
    if (a.split > 1)
        HIP_TRY(mxg::launch_linear_finish(a, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_epilogue_backward(const void* d_out, int32_t d_type, int64_t ld_d_out, const void* z, int64_t ld_z,
                             int64_t rows, int64_t N, int32_t act, int32_t gated, const int32_t* offsets,
                             const int32_t* k_offsets, int32_t experts, int32_t format, uint8_t* q, uint8_t* s,
                             uint8_t* qt, uint8_t* st, int64_t ld_qt, float* d_bias, void* workspace,
                             int64_t workspace_bytes, void* stream)
{
    if (rows < 0 || N < 1 || experts < 0)
        return fail(MXGEMM_EINVAL, "rows %lld and experts %d must not be negative, N %lld must be positive",
                    (long long)rows, experts, (long long)N);
    // 65534 chunks of 128 tokens; four threads per column of N, below 2^32
    if (rows > 65534LL * 128 || N > (1LL << 30) - 1024)
        return fail(MXGEMM_EUNSUPPORTED, "%lld rows or N %lld are too many", (long long)rows, (long long)N);
    if (d_type < MXGEMM_TYPE_BF16 || d_type > MXGEMM_TYPE_FP32)
        return fail(MXGEMM_EINVAL, "unknown element type %d", d_type);
    if (act < MXGEMM_ACT_NONE || act > MXGEMM_ACT_SILU)
        return fail(MXGEMM_EINVAL, "unknown activation %d", act);
    if (format != MXGEMM_FMT_E4M3 && format != MXGEMM_FMT_E5M2)
        return fail(MXGEMM_EINVAL, "unknown FP8 format %d", format);
    if (gated && N % 2 != 0)
        return fail(MXGEMM_EINVAL, "a gated product needs an even N, not %lld", (long long)N);
    if (rows > 0 && !z && (gated || act != MXGEMM_ACT_NONE))     // an array of no rows may be NULL
        return fail(MXGEMM_EINVAL, "an activation's gradient needs z");
    if ((q == nullptr) != (s == nullptr) || (qt == nullptr) != (st == nullptr))
        return fail(MXGEMM_EINVAL, "codes and scales come together (q with s, qt with st)");
    if (experts && (!offsets || !k_offsets))
        return fail(MXGEMM_EINVAL, "by expert, offsets and k_offsets are needed");
    const int64_t padded = (rows + 127) / 128 * 128;
    if (ld_qt % 128 != 0 || (!experts && ld_qt != padded))
        return fail(MXGEMM_EINVAL, "ld_qt %lld must be a multiple of 128 (%lld where not by expert)",
                    (long long)ld_qt, (long long)padded);
    const int64_t chunks = ld_qt / 128;
    if (chunks > 65534 || experts > 65535)      // of the grid's second dimension, one for what is past the last
        return fail(MXGEMM_EUNSUPPORTED, "%lld chunks of 128 tokens or %d experts exceed 65534", (long long)chunks,
                    experts);
    TRY(check_stride("d_out", ld_d_out, gated ? N / 2 : N));
    if (z)
        TRY(check_stride("z", ld_z, N));
    const int64_t need = d_bias ? chunks * N * 4 : 0;
    if (workspace_bytes < need)
        return fail(MXGEMM_EINVAL, "workspace of %lld bytes is less than %lld", (long long)workspace_bytes,
                    (long long)need);
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const bool none = rows == 0;
    const Buffer bufs[] = {{d_out, "d_out", element_size(d_type), none},
                           {z, "z", 2, true},
                           {experts ? offsets : nullptr, "offsets", 4, true},
                           {experts ? k_offsets : nullptr, "k_offsets", 4, true},
                           {q, "q", 16, true},
                           {s, "s", 1, true},
                           {qt, "qt", 16, true},
                           {st, "st", 1, true},
                           {d_bias, "d_bias", 4, true},
                           {need ? workspace : nullptr, "workspace", 4, need == 0}};
    TRY(check_buffers(bufs, dev));
    mxg::GradArgs a;
    memset(&a, 0, sizeof(a));
    a.d = d_out;
    a.d_type = d_type;
    a.ld_d = ld_d_out;
    a.z = (const uint16_t*)z;
    a.ld_z = ld_z;
    a.rows = (int)rows;
    a.N = (int)N;
    a.act = act;
    a.gated = gated ? 1 : 0;
    a.offsets = experts ? offsets : nullptr;
    a.k_offsets = experts ? k_offsets : nullptr;
    a.groups = experts;
    a.fmt = format;
    a.q = q;
    a.s = s;
    a.ld_q = (N + 127) / 128 * 128;
    a.qt = qt;
    a.st = st;
    a.ld_qt = ld_qt;
    a.part = d_bias ? (float*)workspace : nullptr;
    a.d_bias = d_bias;
    a.chunks = (int)chunks;
    HIP_TRY(mxg::launch_grad(a, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_transpose_bytes(const void* src, int64_t ld_src, int64_t src_batch, int64_t rows, int64_t cols,
                           int64_t batch, void* dst, void* stream)
{
    if (rows < 0 || cols < 0 || batch < 0)
        return fail(MXGEMM_EINVAL, "sizes must not be negative");
    TRY(check_stride("src", ld_src, cols));
    if (batch > 65535 || rows > 65535LL * 128 || cols > (1LL << 31) - 128)
        return fail(MXGEMM_EUNSUPPORTED, "%lld matrices of %lld x %lld bytes are too many", (long long)batch,
                    (long long)rows, (long long)cols);
    if (rows == 0 || cols == 0 || batch == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const Buffer bufs[] = {{src, "src", 1, false}, {dst, "dst", 1, false}};
    TRY(check_buffers(bufs, dev));
    const mxg::TransposeArgs a = {(const uint8_t*)src, src_batch, ld_src, (uint8_t*)dst, rows, cols, batch};
    HIP_TRY(mxg::launch_transpose(a, (hipStream_t)stream));
    return MXGEMM_OK;
}

}  // extern "C"
