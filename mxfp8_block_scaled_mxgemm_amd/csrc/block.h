// Internal interface of the operators with scales of 128 and of those around
// them: routing, norms, quantisation, products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear.h"

namespace mxg {

// ------------------------------------------------------------------- norm --

// Rows of H <= kNormMaxCols elements; strides in elements.
constexpr int kNormMaxCols = 8192;

struct NormArgs {
    const void* x;                // the block's output
    const void* residual;         // or null
    const void* gate;             // [gate_rows][cols] or null
    const void* post;             // weights of the norm of x, or null: x as it is
    const void* pre;              // weights of the norm of r, or null: no y
    void* r;                      // forward: written; backward: read
    void* y;
    const void* d_y;              // null: zero
    const void* d_r;              // null: zero
    void* d_x;
    void* d_residual;             // or null
    void* d_gate;                 // [gate_rows][cols] of the gate's type
    float* d_post;                // [cols]
    float* d_pre;
    int64_t ld_x, ld_res, ld_gate, ld_r, ld_y, ld_dy, ld_dr, ld_dx, ld_dres;
    int64_t rows, gates, per_gate;        // rows of one gate row
    int cols, layer;
    int gate_type, post_type, pre_type;
    float scale, eps;
    // backward: rows in units, each within one gate row's; units per worker
    int64_t units, per_unit;      // units of a gate row; rows of a unit
    int workers;
    float* part;                  // [3][workers][cols]: post, pre, gate
};

int norm_threads(int cols);       // of a row: eight elements each
hipError_t launch_norm(const NormArgs& a, int type, int cus, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs& a, int type, hipStream_t stream);

// ------------------------------------------------------------------ route --

constexpr int kRouteMaxExperts = 1024, kRouteMaxChoices = 64, kRouteMaxGroups = 64;

struct RouteArgs {
    const void* logits;           // [tokens][experts]
    int64_t ld;                   // elements
    int type;
    int64_t tokens;
    int experts, k;
    int sigmoid, normalize;
    const float* bias;            // [experts] or null
    int groups, top_groups;
    float scale;
    int32_t* ids;                 // [tokens][k]; backward: read
    float* weights;               // [tokens][k]
    const float* d_weights;       // [tokens][k]
    void* d_logits;               // [tokens][experts] of `type`
    int64_t ld_d;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t stream);

// --------------------------------------------------------------- quantise --

constexpr int kScaleBlock = 128;

// y = act(x) (gated: act(x[:, :half]) x[:, half:]), or with z the gradient
// dz = x act'(z) (gated: [x u act'(g), x act(g)]), quantised in blocks of 128
// along its columns (q, s) and, transposed, along its rows (qt, st).
struct BlockQuantArgs {
    const void* x;                // [rows][..]
    int type;
    int64_t ld_x;
    const uint16_t* z;            // bfloat16 [rows][N], or null
    int64_t ld_z;
    int rows, C;                  // C: columns of y
    int half;                     // gated: the columns of one half of x (y = C) or of z (C = 2 half); else 0
    int act;
    const int32_t* offsets;       // by expert, or null
    const int32_t* k_offsets;
    int groups, chunks;           // chunks of 128 rows in ld_qt (cols) or in rows
    int fmt;
    uint8_t* q;                   // [rows][Cp], Cp = C rounded up to 128, or null
    float* s;                     // [Cp / 128][rows]
    uint8_t* qt;                  // [C][ld_qt], or null
    float* st;                    // [ld_qt / 128][C]
    int64_t ld_qt;
};
hipError_t launch_block_quant(const BlockQuantArgs& a, hipStream_t stream);

// Weights in squares of 128 x 128.
struct SquareQuantArgs {
    const void* w;                // [batch][N][K]
    int type;
    int64_t ld, group;
    int batch, N, K, fmt;
    uint8_t* q;                   // [batch][N][Kp]
    float* s;                     // [batch][Np / 128][Kp / 128]
    uint8_t* qt;                  // [batch][K][Np], or null
    float* st;                    // [batch][Kp / 128][Np / 128]
};
hipError_t launch_square_quant(const SquareQuantArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- product --

// As LinArgs (without an epilogue), the operands' scales float32 with any
// strides, in elements: a's [rows][K / 128]; w's [N / 128][K / 128] (squares)
// or [N][K / 128].
struct BlockLinArgs : LinArgs {
    const float* a_scale;
    const float* w_scale;
    int64_t as_row, as_k, ws_row, ws_k, w_scale_group;
    int squares;
};

// Tile configurations of the product
enum {
    kBlock256x256 = 0,            // native only: eight waves of 128 x 64
    kBlock128x128 = 1,            // four waves of 64 x 64, two work-groups per compute unit
    kBlock64x64 = 2,              // four K groups of one wave
    kBlockRows32 = 3,             // 32 or 16 rows, weights straight to registers; squares only
    kBlockRows16 = 4,
    kBlockCfgs = 5
};
LinTile block_tile(int cfg, const BlockLinArgs& a);
hipError_t launch_block_linear(int cfg, bool exact, int fa, int fw, const BlockLinArgs& a, hipStream_t stream);

}  // namespace mxg
