// Host side of the operators with scales of 128 and of those around them:
// argument rules, the choice of tiles, and the C ABI of
// include/mxgemm_block.h.
#include "mxgemm_block.h"

#include <hip/hip_runtime.h>

#include <math.h>
#include <string.h>

#include "block.h"
#include "host_util.h"
#include "moe.h"
#include "schedule.h"

using mxg::Buffer;
using mxg::check_buffers;
using mxg::check_stride;
using mxg::current_device;
using mxg::fail;

namespace mxg {

template <int FA, int FB>
hipError_t launch_block_fmt(int cfg, bool exact, const BlockLinArgs& a, hipStream_t stream);
extern template hipError_t launch_block_fmt<0, 0>(int, bool, const BlockLinArgs&, hipStream_t);
extern template hipError_t launch_block_fmt<0, 1>(int, bool, const BlockLinArgs&, hipStream_t);
extern template hipError_t launch_block_fmt<1, 0>(int, bool, const BlockLinArgs&, hipStream_t);
extern template hipError_t launch_block_fmt<1, 1>(int, bool, const BlockLinArgs&, hipStream_t);

hipError_t launch_block_linear(int cfg, bool exact, int fa, int fw, const BlockLinArgs& a, hipStream_t stream)
{
    if (fa == 0)
        return fw == 0 ? launch_block_fmt<0, 0>(cfg, exact, a, stream) : launch_block_fmt<0, 1>(cfg, exact, a, stream);
    return fw == 0 ? launch_block_fmt<1, 0>(cfg, exact, a, stream) : launch_block_fmt<1, 1>(cfg, exact, a, stream);
}

LinTile block_tile(int cfg, const BlockLinArgs& a)
{
    const int few = a.skinny == kSkinnyNarrow ? 16 : 32;
    const int threads = a.skinny == kSkinnyNarrow ? 1024 : a.skinny == kSkinny8 ? 512 : a.skinny == kSkinny2 ? 128 : 256;
    switch (cfg) {
    case kBlock256x256: return {256, 256, 512};
    case kBlock128x128: return {128, 128, 256};
    case kBlock64x64: return {64, 64, 256};
    case kBlockRows32: return {32, few, threads};
    default: return {16, few, threads};
    }
}

}  // namespace mxg

namespace {

bool bad_type(int type) { return type < MXGEMM_TYPE_BF16 || type > MXGEMM_TYPE_FP32; }
int element_size(int type) { return type == MXGEMM_TYPE_FP32 ? 4 : 2; }

#define REQUIRE(cond, ...)                          \
    do {                                            \
        if (!(cond))                                \
            return fail(MXGEMM_EINVAL, __VA_ARGS__); \
    } while (0)

// ------------------------------------------------------------------ route --

int route_args(mxg::RouteArgs* a, const void* logits, int64_t ld, int32_t type, int64_t tokens, int32_t experts,
               int32_t k, int32_t score, int32_t normalize, float scale)
{
    REQUIRE(!bad_type(type), "unknown element type %d", type);
    REQUIRE(score == MXGEMM_SCORE_SOFTMAX || score == MXGEMM_SCORE_SIGMOID, "unknown score %d", score);
    REQUIRE(tokens >= 0 && experts >= 1 && k >= 1 && k <= experts,
            "tokens %lld must not be negative, and k %d positive and at most the %d experts", (long long)tokens, k,
            experts);
    if (experts > mxg::kRouteMaxExperts || k > mxg::kRouteMaxChoices || tokens > (1LL << 40))
        return fail(MXGEMM_EUNSUPPORTED, "%lld tokens, %d experts or %d choices are too many", (long long)tokens,
                    experts, k);
    TRY(check_stride("logits", ld, experts));
    memset(a, 0, sizeof(*a));
    a->logits = logits;
    a->ld = ld;
    a->type = type;
    a->tokens = tokens;
    a->experts = experts;
    a->k = k;
    a->sigmoid = score == MXGEMM_SCORE_SIGMOID;
    a->normalize = normalize ? 1 : 0;
    a->scale = scale;
    return MXGEMM_OK;
}

// ---------------------------------------------------------------- product --

// The tile configuration for a product.  Few rows (of an average expert): the
// weights' bytes are the cost, and the skinny kernels stream them.  By expert,
// exact, 4096 x 4096 weights, 16-row / 32-row / 128 x 128 tiles: 8 rows per
// expert of 64, 195 / 204 / 274 us; 16 of 32, 141 / 116 / 144; 32 of 32, 223 /
// 172 / 146.  Dense, 32-row tiles against 64 x 64 ones with split K: 32 x 2048 x
// 7168, 13.4 and 21.9 us; 64 x 2048 x 7168 13.9 and 16.1; 64 x 8192 x 8192, where
// two row tiles no longer fit on the compute units at once, 36 and 22.
// Then 128 x 128 tiles, two of whose work-groups share a compute unit, where
// they occupy more than half of the compute units (512 x 4096 x 4096 exact, 128
// tiles: 37 us against 29 with 64 x 64 ones).  Native products of squares may
// take 256 x 256 tiles: a round of those on all compute units takes 5 / 3 of the
// time of a round of 128 x 128 ones (8192 x 8192 x 8192: 464 us in 4 rounds and
// 562 in 8), so the rule compares rounds; the experts' last tiles count half.
// 2048 x 4096 x 4096: 55 and 44 us; 2048 x 8192 x 2048: 40 and 45; 3000 x 4096 x
// 2048: 35 and 37; 4096 x 4096 x 512: 20 and 21; by expert, 4096 x 4096 weights:
// 32 of 128 rows 219 and 180, 64 of 256 423 and 484, 32 of 512 430 and 430.
int choose_tile(const mxg::BlockLinArgs& a, bool exact, int cus)
{
    const bool by = a.mode == mxg::kByRows;
    const int64_t r = by ? (a.rows + a.groups - 1) / a.groups : a.rows;
    if (a.squares && r <= (by ? 10 : 16))
        return mxg::kBlockRows16;
    if (a.squares && (r <= (by ? 24 : 32) || (!by && r <= 64 && (r + 31) / 32 * ((a.N + 15) / 16) <= cus)))
        return mxg::kBlockRows32;
    // tiles of m x n, twice (an expert ends inside its last one)
    auto tiles2 = [&](int64_t m, int64_t n) {
        const int64_t rows = by ? (2 * r + m) / m * a.groups : 2 * ((r + m - 1) / m);
        return (a.mode == mxg::kByInner ? a.groups : 1) * rows * ((a.N + n - 1) / n);
    };
    const int64_t big = tiles2(256, 256), mid = tiles2(128, 128);
    if (!exact && a.squares) {
        const int64_t cost_big = 5 * ((big + 2 * cus - 1) / (2 * cus)), cost_mid = 3 * ((mid + 4 * cus - 1) / (4 * cus));
        if (cost_big < cost_mid || (cost_big == cost_mid && a.K >= 2048))
            return mxg::kBlock256x256;
    }
    return mid > cus ? mxg::kBlock128x128 : mxg::kBlock64x64;
}

// K splits of a dense product of 64 x 64 tiles: as many work-groups as
// compute units, each with two K-steps at least for each of its four groups.
int choose_split(const mxg::BlockLinArgs& a, int cus)
{
    const int64_t tiles = (int64_t)((a.rows + 63) / 64) * ((a.N + 63) / 64);
    int64_t s = cus / tiles;
    const int64_t most = a.K / mxg::kGroupK / 8;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s);
}

int check_linear(const mxgemm_block_linear_t* g, mxg::BlockLinArgs* a)
{
    REQUIRE(g->rows >= 0 && g->N >= 1 && g->K >= 1, "rows %lld must not be negative, N %lld and K %lld must be positive",
            (long long)g->rows, (long long)g->N, (long long)g->K);
    REQUIRE(g->K % 128 == 0, "K %lld must be a multiple of the block 128", (long long)g->K);
    if (g->K > (1 << 30) || g->N >= (1LL << 31) - 1024 || g->rows >= (1LL << 31) - 1024)
        return fail(MXGEMM_EUNSUPPORTED, "problem too large for 32-bit indexes");
    REQUIRE(g->mode >= MXGEMM_GROUP_NONE && g->mode <= MXGEMM_GROUP_INNER, "unknown group mode %d", g->mode);
    REQUIRE(g->mode == MXGEMM_GROUP_NONE || (g->experts >= 1 && g->offsets),
            "a product by expert needs experts and offsets");
    if (g->mode != MXGEMM_GROUP_NONE && g->experts > (1 << 20))
        return fail(MXGEMM_EUNSUPPORTED, "%d experts exceed 2^20", g->experts);
    REQUIRE(!(g->mode == MXGEMM_GROUP_INNER && g->squares), "GROUP_INNER takes a scale for each row of w, no squares");
    REQUIRE(!bad_type(g->out_type), "unknown output type %d", g->out_type);
    REQUIRE(!((g->a_format | g->w_format) & ~1), "unknown FP8 format (a %d, w %d)", g->a_format, g->w_format);
    REQUIRE(g->precision == MXGEMM_PRECISION_EXACT || g->precision == MXGEMM_PRECISION_NATIVE,
            "unknown precision mode %d", g->precision);
    TRY(check_stride("a", g->lda, g->K));
    TRY(check_stride("w", g->ldw, g->K));
    TRY(check_stride("out", g->ld_out, g->N));
    REQUIRE(g->lda % 16 == 0 && g->ldw % 16 == 0 && g->w_group % 16 == 0,
            "strides of a and w must be multiples of 16 bytes");
    REQUIRE(g->a_scale_row >= 0 && g->a_scale_k >= 0 && g->w_scale_row >= 0 && g->w_scale_k >= 0 && g->w_group >= 0 &&
                g->w_scale_group >= 0,
            "strides must not be negative");
    if (g->lda > (1 << 23) || g->ldw > (1 << 23) || g->a_scale_row > (1 << 21) || g->w_scale_row > (1 << 21))
        return fail(MXGEMM_EUNSUPPORTED, "row strides of the operands are limited to 8 MiB (scales 2^21 elements)");
    memset(a, 0, sizeof(*a));
    a->a = (const uint8_t*)g->a;
    a->w = (const uint8_t*)g->w;
    a->a_scale = g->a_scale;
    a->w_scale = g->w_scale;
    a->lda = g->lda;
    a->ldw = g->ldw;
    a->w_group = g->w_group;
    a->as_row = g->a_scale_row;
    a->as_k = g->a_scale_k;
    a->ws_row = g->w_scale_row;
    a->ws_k = g->w_scale_k;
    a->w_scale_group = g->w_scale_group;
    a->squares = g->squares ? 1 : 0;
    a->offsets = g->offsets;
    a->mode = g->mode;
    a->groups = g->mode == MXGEMM_GROUP_NONE ? 0 : g->experts;
    a->rows = (int)g->rows;
    a->N = (int)g->N;
    a->K = (int)g->K;
    a->out = g->out;
    a->ld_out = g->ld_out;
    a->out_group = g->out_group;
    a->out_type = g->out_type;
    return MXGEMM_OK;
}

// Tiles of configuration cfg and their order.
int plan_linear(mxg::BlockLinArgs* a, int cfg, int cus, int64_t workspace_bytes)
{
    a->split = 1;
    if (cfg == mxg::kBlock64x64 && a->mode == mxg::kDense) {
        const int split = choose_split(*a, cus);
        if ((int64_t)split * a->rows * a->N * 4 <= workspace_bytes)
            a->split = split;
    }
    a->skinny = mxg::kSkinny8;
    if (a->mode == mxg::kDense && (a->N + 31) / 32 < cus)
        a->skinny = mxg::kSkinnyNarrow;
    else if (a->mode != mxg::kDense)
        a->skinny = a->K <= 8 * mxg::kGroupK ? mxg::kSkinny2 : mxg::kSkinny4;
    const mxg::LinTile t = mxg::block_tile(cfg, *a);
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
    // resident work-groups; skinny tiles of one row tile share no rows of w, so
    // theirs run along N (with two, a column's land on different XCDs, each of
    // which then reads its rows of w)
    const int64_t per_xcd = ((work < cus ? work : cus) + mxg::kNumXcd - 1) / mxg::kNumXcd / a->split;
    int64_t g = (int64_t)floor(sqrt((double)(per_xcd > 1 ? per_xcd : 1)));
    if (cfg >= mxg::kBlockRows32)
        g = tiles_n;
    a->group_n = (int)(g < 1 ? 1 : g > tiles_n ? tiles_n : g);
    return MXGEMM_OK;
}

// ------------------------------------------------------------------- norm --

// Rows of the gradient in units, each within one gate row's, and workers: at
// most as many as 16 waves on each of 256 compute units (their registers allow
// no more; where a wave takes a row, up to 512 columns, they allow 12, and the
// last workers start as others end).  The workers' partial rows are the workspace.
void plan_norm(mxg::NormArgs* a, int64_t gate_rows)
{
    const int64_t most = 256 * 16 * 64 / mxg::norm_threads(a->cols);
    a->gates = gate_rows;
    a->per_gate = a->rows / gate_rows;
    a->units = 1;
    if (a->rows == 0) {             // sums over nothing
        a->units = a->per_unit = a->workers = 0;
        return;
    }
    if (gate_rows < most) {
        a->units = most / gate_rows;
        a->units = a->units < a->per_gate ? a->units : a->per_gate;
    }
    a->per_unit = (a->per_gate + a->units - 1) / a->units;
    a->units = (a->per_gate + a->per_unit - 1) / a->per_unit;
    const int64_t all = gate_rows * a->units;
    a->workers = (int)(all < most ? all : most);
}

int norm_args(const mxgemm_norm_t* g, mxg::NormArgs* a, bool backward)
{
    REQUIRE(g->rows >= 0 && g->cols >= 1, "rows %lld must not be negative, cols %lld must be positive",
            (long long)g->rows, (long long)g->cols);
    if (g->cols > mxg::kNormMaxCols || g->rows > (1LL << 40))
        return fail(MXGEMM_EUNSUPPORTED, "%lld rows of %lld columns are too many (columns: at most %d)",
                    (long long)g->rows, (long long)g->cols, mxg::kNormMaxCols);
    REQUIRE(!bad_type(g->type), "unknown element type %d", g->type);
    REQUIRE(g->kind == MXGEMM_NORM_RMS || g->kind == MXGEMM_NORM_LAYER, "unknown norm %d", g->kind);
    REQUIRE(!(g->gate && bad_type(g->gate_type)) && !(g->post_weight && bad_type(g->post_type)) &&
                !(g->pre_weight && bad_type(g->pre_type)),
            "unknown element type of the gate %d or a weight %d, %d", g->gate_type, g->post_type, g->pre_type);
    const int64_t gates = g->gate ? g->gate_rows : 1;
    REQUIRE(gates >= 1 && g->rows % gates == 0, "%lld gate rows do not divide %lld rows", (long long)gates,
            (long long)g->rows);
    if (g->rows == 0 && gates > 65533)
        return fail(MXGEMM_EUNSUPPORTED, "%lld gate rows without rows are too many", (long long)gates);
    TRY(check_stride("x", g->ld_x, g->cols));
    TRY(check_stride("r", g->ld_r, g->cols));
    REQUIRE(!g->gate || g->ld_gate >= 0, "the gate's row stride must not be negative");
    if (!backward) {
        if (g->residual)
            TRY(check_stride("residual", g->ld_residual, g->cols));
        if (g->pre_weight)
            TRY(check_stride("y", g->ld_y, g->cols));
    } else {
        if (g->d_y)
            TRY(check_stride("d_y", g->ld_d_y, g->cols));
        if (g->d_r)
            TRY(check_stride("d_r", g->ld_d_r, g->cols));
        TRY(check_stride("d_x", g->ld_d_x, g->cols));
        if (g->d_residual)
            TRY(check_stride("d_residual", g->ld_d_residual, g->cols));
        REQUIRE(!(g->d_y && !g->pre_weight), "d_y comes with pre_weight");
    }
    memset(a, 0, sizeof(*a));
    a->x = g->x;
    a->residual = g->residual;
    a->gate = g->gate;
    a->post = g->post_weight;
    a->pre = g->pre_weight;
    a->r = g->r;
    a->y = g->y;
    a->d_y = g->d_y;
    a->d_r = g->d_r;
    a->d_x = g->d_x;
    a->d_residual = g->d_residual;
    a->d_gate = g->d_gate;
    a->d_post = g->d_post_weight;
    a->d_pre = g->d_pre_weight;
    a->ld_x = g->ld_x;
    a->ld_res = g->ld_residual;
    a->ld_gate = g->ld_gate;
    a->ld_r = g->ld_r;
    a->ld_y = g->ld_y;
    a->ld_dy = g->ld_d_y;
    a->ld_dr = g->ld_d_r;
    a->ld_dx = g->ld_d_x;
    a->ld_dres = g->ld_d_residual;
    a->rows = g->rows;
    a->cols = (int)g->cols;
    a->layer = g->kind == MXGEMM_NORM_LAYER;
    a->gate_type = g->gate_type;
    a->post_type = g->post_type;
    a->pre_type = g->pre_type;
    a->scale = g->scale;
    a->eps = g->eps;
    a->part = (float*)g->workspace;
    plan_norm(a, gates);
    return MXGEMM_OK;
}

}  // namespace

extern "C" {

int mxgemm_route_tokens(const void* logits, int64_t ld, int32_t type, int64_t tokens, int32_t experts, int32_t k,
                        int32_t score, const float* bias, int32_t groups, int32_t top_groups, int32_t normalize,
                        float scale, int32_t* ids, float* weights, void* stream)
{
    mxg::RouteArgs a;
    TRY(route_args(&a, logits, ld, type, tokens, experts, k, score, normalize, scale));
    REQUIRE(groups >= 1 && top_groups >= 1 && top_groups <= groups && experts % groups == 0,
            "%d groups (%d taken) do not divide %d experts", groups, top_groups, experts);
    if (groups > mxg::kRouteMaxGroups)
        return fail(MXGEMM_EUNSUPPORTED, "%d groups exceed %d", groups, mxg::kRouteMaxGroups);
    REQUIRE(k <= experts / groups * top_groups, "k %d exceeds the %d experts of %d groups", k,
            experts / groups * top_groups, top_groups);
    if (tokens == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const Buffer bufs[] = {{logits, "logits", element_size(type), false}, {bias, "bias", 4, true},
                           {ids, "ids", 4, false}, {weights, "weights", 4, false}};
    TRY(check_buffers(bufs, dev));
    a.bias = bias;
    a.groups = groups;
    a.top_groups = top_groups;
    a.ids = ids;
    a.weights = weights;
    HIP_TRY(mxg::launch_route(a, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_route_tokens_backward(const float* d_weights, const void* logits, int64_t ld, int32_t type, int64_t tokens,
                                 int32_t experts, int32_t k, int32_t score, int32_t normalize, float scale,
                                 const int32_t* ids, void* d_logits, int64_t ld_d, void* stream)
{
    mxg::RouteArgs a;
    TRY(route_args(&a, logits, ld, type, tokens, experts, k, score, normalize, scale));
    TRY(check_stride("d_logits", ld_d, experts));
    if (tokens == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const int size = element_size(type);
    const Buffer bufs[] = {{d_weights, "d_weights", 4, false}, {logits, "logits", size, false}, {ids, "ids", 4, false},
                           {d_logits, "d_logits", size, false}};
    TRY(check_buffers(bufs, dev));
    a.d_weights = d_weights;
    a.ids = const_cast<int32_t*>(ids);
    a.d_logits = d_logits;
    a.ld_d = ld_d;
    HIP_TRY(mxg::launch_route_backward(a, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_block_quantize(const void* x, int32_t type, int64_t ld_x, const void* z, int64_t ld_z, int64_t rows,
                          int64_t C, int32_t act, int32_t gated, const int32_t* offsets, const int32_t* k_offsets,
                          int32_t experts, int32_t format, uint8_t* q, float* s, uint8_t* qt, float* st, int64_t ld_qt,
                          void* stream)
{
    REQUIRE(rows >= 0 && C >= 1 && experts >= 0, "rows %lld and experts %d must not be negative, C %lld must be positive",
            (long long)rows, experts, (long long)C);
    if (rows > 65534LL * 128 || C > (1LL << 30))
        return fail(MXGEMM_EUNSUPPORTED, "%lld rows or %lld columns are too many", (long long)rows, (long long)C);
    REQUIRE(!bad_type(type), "unknown element type %d", type);
    REQUIRE(act >= MXGEMM_ACT_NONE && act <= MXGEMM_ACT_SILU, "unknown activation %d", act);
    REQUIRE(format == MXGEMM_FMT_E4M3 || format == MXGEMM_FMT_E5M2, "unknown FP8 format %d", format);
    REQUIRE(!(z && gated && C % 2 != 0), "a gated gradient needs even columns, not %lld", (long long)C);
    REQUIRE((q == nullptr) == (s == nullptr) && (qt == nullptr) == (st == nullptr),
            "codes and scales come together (q with s, qt with st)");
    REQUIRE(!experts || (offsets && k_offsets), "by expert, offsets and k_offsets are needed");
    const int64_t padded = (rows + 127) / 128 * 128;
    int64_t chunks = padded / 128;
    if (qt) {
        REQUIRE(ld_qt % 128 == 0 && ld_qt >= 0 && (experts || ld_qt == padded),
                "ld_qt %lld must be a multiple of 128 (%lld where not by expert)", (long long)ld_qt, (long long)padded);
        chunks = ld_qt / 128;
    }
    if (chunks > 65534 || experts > 65535)
        return fail(MXGEMM_EUNSUPPORTED, "%lld chunks of 128 rows or %d experts exceed 65534", (long long)chunks, experts);
    const int64_t held = z ? (gated ? C / 2 : C) : (gated ? 2 * C : C);
    TRY(check_stride("x", ld_x, held));
    if (z)
        TRY(check_stride("z", ld_z, C));
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const Buffer bufs[] = {{x, "x", element_size(type), rows == 0},
                           {z, "z", 2, true},
                           {experts ? offsets : nullptr, "offsets", 4, true},
                           {experts ? k_offsets : nullptr, "k_offsets", 4, true},
                           {q, "q", 16, true},
                           {s, "s", 4, true},
                           {qt, "qt", 16, true},
                           {st, "st", 4, true}};
    TRY(check_buffers(bufs, dev));
    // (no rows: qt's columns past the last segment still become zero)
    if (!q && !qt)
        return MXGEMM_OK;
    if (chunks == 0 && !(qt && experts && rows > 0))
        return MXGEMM_OK;
    mxg::BlockQuantArgs a;
    memset(&a, 0, sizeof(a));
    a.x = x;
    a.type = type;
    a.ld_x = ld_x;
    a.z = (const uint16_t*)z;
    a.ld_z = ld_z;
    a.rows = (int)rows;
    a.C = (int)C;
    a.half = !gated ? 0 : z ? (int)(C / 2) : (int)C;
    a.act = act;
    a.offsets = experts ? offsets : nullptr;
    a.k_offsets = experts ? k_offsets : nullptr;
    a.groups = experts;
    a.chunks = (int)chunks;
    a.fmt = format;
    a.q = q;
    a.s = s;
    a.qt = qt;
    a.st = st;
    a.ld_qt = ld_qt;
    HIP_TRY(mxg::launch_block_quant(a, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_block_quantize_weight(const void* w, int32_t type, int64_t ld, int64_t group, int64_t batch, int64_t N,
                                 int64_t K, int32_t format, uint8_t* q, float* s, uint8_t* qt, float* st, void* stream)
{
    REQUIRE(batch >= 0 && N >= 1 && K >= 1, "sizes must be positive");
    REQUIRE(!bad_type(type), "unknown element type %d", type);
    REQUIRE(format == MXGEMM_FMT_E4M3 || format == MXGEMM_FMT_E5M2, "unknown FP8 format %d", format);
    REQUIRE((qt == nullptr) == (st == nullptr), "codes and scales come together (qt with st)");
    TRY(check_stride("w", ld, K));
    REQUIRE(group >= 0, "the matrix stride must not be negative");
    if (batch > 65535 || N > 65535LL * 128 || K > (1LL << 30))
        return fail(MXGEMM_EUNSUPPORTED, "%lld matrices of %lld x %lld are too many", (long long)batch, (long long)N,
                    (long long)K);
    if (batch == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const Buffer bufs[] = {{w, "w", element_size(type), false}, {q, "q", 16, false}, {s, "s", 4, false},
                           {qt, "qt", 16, true}, {st, "st", 4, true}};
    TRY(check_buffers(bufs, dev));
    const mxg::SquareQuantArgs a = {w, type, ld, group, (int)batch, (int)N, (int)K, format, q, s, qt, st};
    HIP_TRY(mxg::launch_square_quant(a, (hipStream_t)stream));
    return MXGEMM_OK;
}

int64_t mxgemm_block_linear_workspace(int64_t rows, int64_t N, int64_t K) { return mxgemm_linear_workspace(rows, N, K); }

int mxgemm_block_linear(const mxgemm_block_linear_t* args, void* stream)
{
    if (!args)
        return fail(MXGEMM_EINVAL, "args is NULL");
    mxg::BlockLinArgs a;
    TRY(check_linear(args, &a));
    const bool exact = args->precision == MXGEMM_PRECISION_EXACT;
    const int forced = args->tile_cfg;
    if (forced >= mxg::kBlockCfgs || (forced == mxg::kBlock256x256 && (exact || !a.squares)) ||
        (forced >= mxg::kBlockRows32 && !a.squares))
        return fail(MXGEMM_EINVAL, "tile_cfg %d has no kernel for this precision mode or these scales", forced);
    if (args->rows == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const Buffer bufs[] = {{args->a, "a", 16, false},
                           {args->a_scale, "a_scale", 4, false},
                           {args->w, "w", 16, false},
                           {args->w_scale, "w_scale", 4, false},
                           {args->out, "out", element_size(args->out_type), false},
                           {args->workspace, "workspace", 16, true},
                           {a.groups ? args->offsets : nullptr, "offsets", 4, true}};
    TRY(check_buffers(bufs, dev));
    const int cfg = forced >= 0 ? forced : choose_tile(a, exact, cus);
    TRY(plan_linear(&a, cfg, cus, args->workspace ? args->workspace_bytes : 0));
    a.part = (float*)args->workspace;
    HIP_TRY(mxg::launch_block_linear(cfg, exact, args->a_format, args->w_format, a, (hipStream_t)stream));
    if (a.split > 1)
        HIP_TRY(mxg::launch_linear_finish(a, (hipStream_t)stream));
    return MXGEMM_OK;
}

int64_t mxgemm_add_norm_workspace(int64_t rows, int64_t cols, int64_t gate_rows)
{
    if (rows < 1 || cols < 1 || cols > mxg::kNormMaxCols || gate_rows < 1 || rows % gate_rows != 0)
        return 0;
    mxg::NormArgs a;
    memset(&a, 0, sizeof(a));
    a.rows = rows;
    a.cols = (int)cols;
    plan_norm(&a, gate_rows);
    return 3LL * a.workers * cols * 4;
}

int mxgemm_add_norm(const mxgemm_norm_t* args, void* stream)
{
    if (!args)
        return fail(MXGEMM_EINVAL, "args is NULL");
    mxg::NormArgs a;
    TRY(norm_args(args, &a, false));
    if (args->rows == 0)
        return MXGEMM_OK;
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const int size = element_size(args->type);
    const Buffer bufs[] = {{a.x, "x", size, false},
                           {a.residual, "residual", size, true},
                           {a.gate, "gate", element_size(args->gate_type), true},
                           {a.post, "post_weight", element_size(args->post_type), true},
                           {a.pre, "pre_weight", element_size(args->pre_type), true},
                           {a.r, "r", size, false},
                           {a.pre ? a.y : nullptr, "y", size, !a.pre}};
    TRY(check_buffers(bufs, dev));
    HIP_TRY(mxg::launch_norm(a, args->type, cus, (hipStream_t)stream));
    return MXGEMM_OK;
}

int mxgemm_add_norm_backward(const mxgemm_norm_t* args, void* stream)
{
    if (!args)
        return fail(MXGEMM_EINVAL, "args is NULL");
    mxg::NormArgs a;
    TRY(norm_args(args, &a, true));
    const int64_t need = mxgemm_add_norm_workspace(args->rows, args->cols, args->gate ? args->gate_rows : 1);
    REQUIRE(args->workspace_bytes >= need, "workspace of %lld bytes is less than %lld", (long long)args->workspace_bytes,
            (long long)need);
    int dev, cus;
    TRY(current_device(&dev, &cus));
    const int size = element_size(args->type);
    const bool none = args->rows == 0, reads_x = a.post || a.gate;
    const Buffer bufs[] = {{reads_x ? a.x : nullptr, "x", size, none || !reads_x},
                           {a.d_y ? a.r : nullptr, "r", size, none || !a.d_y},
                           {a.gate, "gate", element_size(args->gate_type), true},
                           {a.post, "post_weight", element_size(args->post_type), true},
                           {a.pre, "pre_weight", element_size(args->pre_type), true},
                           {a.d_y, "d_y", size, true},
                           {a.d_r, "d_r", size, true},
                           {a.d_x, "d_x", size, none},
                           {a.d_residual, "d_residual", size, true},
                           {a.gate ? a.d_gate : nullptr, "d_gate", element_size(args->gate_type), !a.gate},
                           {a.post ? a.d_post : nullptr, "d_post_weight", 4, !a.post},
                           {a.pre ? a.d_pre : nullptr, "d_pre_weight", 4, !a.pre},
                           {need ? args->workspace : nullptr, "workspace", 4, need == 0}};
    TRY(check_buffers(bufs, dev));
    if (!a.post)
        a.d_post = nullptr;
    if (!a.pre)
        a.d_pre = nullptr;
    HIP_TRY(mxg::launch_norm_backward(a, args->type, (hipStream_t)stream));
    return MXGEMM_OK;
}

}  // extern "C"
