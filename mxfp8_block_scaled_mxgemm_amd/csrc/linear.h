// Internal interface of the MXFP8 product with a fused epilogue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxg {

// Activations (the values of MXGEMM_ACT_*)
constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;
// Output types beyond the element types: MXFP8 codes (the values of MXGEMM_TYPE_*)
constexpr int kMxE4M3 = 3, kMxE5M2 = 4;

// How the experts share a product.
//   kDense    out = a w^T
//   kByRows   rows [offsets[e], offsets[e + 1]) of a times w[e]^T; the rows
//             past offsets[groups] of out are zero
//   kByInner  out[e] = a w^T over inner range [offsets[e], offsets[e + 1]),
//             whose ends are multiples of 128
enum { kDense = 0, kByRows = 1, kByInner = 2 };

struct LinArgs {
    const uint8_t* a;             // codes [rows][K], row stride lda bytes
    const uint8_t* as;            // scales [rows][K / 32]
    const uint8_t* w;             // codes [N][K] (per expert)
    const uint8_t* ws;
    int64_t lda, ldas, ldw, ldws;
    int64_t w_group, ws_group;    // bytes between experts
    const int32_t* offsets;
    int mode, groups;
    int rows, N, K;               // N: columns of the product (both halves when gated)
    // epilogue: out = act(z) + residual with z = a w^T + bias, or, gated,
    // act(z[:N/2]) * z[N/2:] + residual
    const void* bias;             // [groups][N] or null
    int bias_type, act, gated;
    const void* residual;         // [rows][cols] of the output's type (bfloat16 for MXFP8) or null
    int64_t ld_res;
    void* out;                    // [rows][cols], cols = N or N / 2; kByInner: [groups][rows][cols]
    int64_t ld_out, out_group;    // elements
    int out_type;
    uint8_t* out_s;               // MXFP8: scale bytes [rows][cols / 32]
    int64_t ld_out_s;
    uint16_t* z;                  // bfloat16 [rows][N] or null: z, before the activation
    int64_t ld_z;
    // plan
    int skinny;                   // kSkinny*, for the skinny tiles
    int split;                    // K splits (kLin64x64, kDense), their sums in `part`
    float* part;                  // [split][rows][N]
    int tiles_m, tiles_n, group_n, total_work;
};

// Tile configurations of the product
enum {
    kLin256x256 = 0,              // native only: four waves of 128 x 128
    kLin128x128 = 1,              // four waves of 64 x 64, two work-groups per compute unit
    kLin64x64 = 2,                // four K groups
    kLinRows32 = 3,               // 32 or 16 rows, weights straight to registers
    kLinRows16 = 4,
    kLinCfgs = 5
};

// Skinny tiles: 16 columns and sixteen waves; 32 columns and 2, 4 or 8 waves;
// 64 columns of a gated product with MXFP8 output (32 outputs: its block)
enum { kSkinnyNarrow, kSkinny2, kSkinny4, kSkinny8, kSkinnyWide };

struct LinTile {
    int tile_m, tile_n;           // tile_n: columns of the product
    int threads;                  // of a work-group
};

hipError_t launch_linear(int cfg, bool exact, int fa, int fw, const LinArgs& a, hipStream_t stream);
// Sums of a product with split > 1 through its epilogue.
hipError_t launch_linear_finish(const LinArgs& a, hipStream_t stream);
// Tile of configuration cfg.
LinTile lin_tile(int cfg, const LinArgs& a);

// Gradient of the epilogue, in tiles of 128 tokens x 64 columns of the
// product: dz = d_out act'(z) (gated: [d_out u act'(g), d_out act(g)]).
struct GradArgs {
    const void* d;                // [rows][cols] (also the plain input when z is null)
    int d_type;
    int64_t ld_d;
    const uint16_t* z;            // bfloat16 [rows][N] or null (act none)
    int64_t ld_z;
    int rows, N, act, gated;
    const int32_t* offsets;       // by expert, or null
    const int32_t* k_offsets;
    int groups;
    int fmt;
    uint8_t* q;                   // codes [rows][ld_q] along the columns, or null
    uint8_t* s;                   // [rows][ld_q / 32]
    int64_t ld_q;                 // columns rounded up to 128
    uint8_t* qt;                  // codes [N][ld_qt] along the tokens, or null
    uint8_t* st;                  // [N][ld_qt / 32]
    int64_t ld_qt;                // tokens of all segments, a multiple of 128
    float* part;                  // [ld_qt / 128][N] column sums per tile, or null
    float* d_bias;                // [groups or 1][N]
    int chunks;                   // 128-token chunks
};
hipError_t launch_grad(const GradArgs& a, hipStream_t stream);

// dst[batch][cols][rows] = src[batch][rows][cols] transposed, bytes.
struct TransposeArgs {
    const uint8_t* src;
    int64_t src_batch, ld_src;
    uint8_t* dst;
    int64_t rows, cols, batch;
};
hipError_t launch_transpose(const TransposeArgs& a, hipStream_t stream);

}  // namespace mxg
