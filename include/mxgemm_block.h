/*
 * mxgemm_block -- the operators of an expert layer with scales of 128, for
 * AMD Instinct MI355X (gfx950): routing of tokens to experts, quantisation to
 * FP8 with a float32 scale for each block of 128, the product of such
 * operands (dense and by expert), and the norms before and after a block with
 * its gate and residual scale; each with its gradient.
 *
 * C ABI of the same library as mxgemm_seg.h, with the same error codes and
 * mxgemm_seg_last_error(), and of mxgemm_moe.h's manner: every call is
 * asynchronous on `stream`, allocates nothing, keeps nothing between calls,
 * can be captured into a HIP graph and may run concurrently with any other
 * (each with a workspace of its own).  All pointers are device memory (or
 * memory the GPU can access; anything else is refused with MXGEMM_EINVAL) and
 * must stay valid until the work completes; buffer sizes are the caller's
 * contract, and so is that no output overlaps another operand.  No
 * floating-point sum is formed by atomics: results repeat bit for bit.
 */
#ifndef MXGEMM_BLOCK_H
#define MXGEMM_BLOCK_H

#include <stdint.h>

#include "mxgemm_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ route --
 * Experts of each token.  With logits l [tokens][experts] of `type` (BF16,
 * FP16, FP32; row stride ld elements) and scores s = softmax(l) over the
 * token's experts, or sigmoid(l):
 *   key[e] = s[e] + bias[e]                (bias float32 [experts], or NULL)
 *   with groups > 1: the experts are `groups` equal runs; a run's rank is the
 *     sum of its two largest keys (of one, its key); only the top_groups runs
 *     of the largest rank take part
 *   ids [tokens][k]      the k experts of the largest keys, in that order
 *   weights [tokens][k]  scale s[id], or, normalised, scale s[id] / sum over
 *                        the token's chosen experts
 * Equal keys and ranks go to the lowest index.  Keys are compared in 64 bits
 * (without bias and groups the logits themselves are).  An expert whose logit
 * or key is -infinity or NaN is never chosen; where fewer than k experts are
 * left the last ids are -1, with weight 0: pairs that mxgemm_sort_tokens drops.
 * A logit of +infinity counts as the largest finite number; sigmoids of logits
 * below -700 are 0.
 * 1 <= experts <= 1024, 1 <= k <= min(experts, 64), groups <= 64 divides
 * experts, 1 <= top_groups <= groups, k <= top_groups * experts / groups.
 * Errors: EINVAL, EUNSUPPORTED, EHIP.
 */
enum { MXGEMM_SCORE_SOFTMAX = 0, MXGEMM_SCORE_SIGMOID = 1 };

int mxgemm_route_tokens(const void* logits, int64_t ld, int32_t type, int64_t tokens, int32_t experts, int32_t k,
                        int32_t score, const float* bias, int32_t groups, int32_t top_groups, int32_t normalize,
                        float scale, int32_t* ids, float* weights, void* stream);

/* Gradient of the weights to the logits (the choice itself has none): d_logits
 * [tokens][experts] of `type`, row stride ld_d.  Ids outside [0, experts)
 * contribute nothing. */
int mxgemm_route_tokens_backward(const float* d_weights, const void* logits, int64_t ld, int32_t type, int64_t tokens,
                                 int32_t experts, int32_t k, int32_t score, int32_t normalize, float scale,
                                 const int32_t* ids, void* d_logits, int64_t ld_d, void* stream);

/* --------------------------------------------------------------- quantise --
 * FP8 codes (MXGEMM_FMT_*) with a float32 scale for each block of 128:
 *   s = max(amax / fmax, 2^-126),  q = y / s rounded to nearest even
 * (fmax 448 or 57344; q from the quotient with s before its rounding, itself
 * rounded to float32).  A block that holds a NaN or an infinity has scale NaN
 * and codes 0x7F, those past the matrix's edge too.  Quantised is, in FP32,
 *   z NULL: y = act(x), or, gated, act(x[:, :C]) * x[:, C:] with x [rows][2 C]
 *   else:   y = x act'(z), or, gated, [x u act'(g), x act(g)] with [g, u] = z
 *           (z bfloat16 [rows][C]; x [rows][C], gated [rows][C / 2])
 * C: the columns of y.
 *   q, s    along the columns: codes [rows][Cp], Cp = C rounded up to 128
 *           (zeros past C), scales [Cp / 128][rows] (a block's of all rows side
 *           by side); by expert (offsets), rows from offsets[experts] on are
 *           not read, and zero, codes and scales
 *   qt, st  transposed, along the rows: codes [C][ld_qt], scales [ld_qt / 128]
 *           [C]; by expert, expert e's rows take columns [k_offsets[e],
 *           k_offsets[e + 1]) (zeros past its last row, and codes and scales
 *           zero past the last segment), else ld_qt is rows rounded up to 128
 * Either pair may be NULL.  By expert: offsets, k_offsets int32 [experts + 1]
 * as mxgemm_sort_tokens makes them, ld_qt >= k_offsets[experts] and a multiple
 * of 128; experts = 0 and NULL otherwise.  q, qt 16-byte aligned.
 * Errors: EINVAL, EUNSUPPORTED (more than 65534 chunks of 128 rows in rows or
 * ld_qt, C above 2^30), EHIP.
 */
int mxgemm_block_quantize(const void* x, int32_t type, int64_t ld_x, const void* z, int64_t ld_z, int64_t rows,
                          int64_t C, int32_t act, int32_t gated, const int32_t* offsets, const int32_t* k_offsets,
                          int32_t experts, int32_t format, uint8_t* q, float* s, uint8_t* qt, float* st, int64_t ld_qt,
                          void* stream);

/* Weights w [batch][N][K] (row stride ld, matrix stride group, elements) with
 * one scale for each square of 128 x 128: codes q [batch][N][Kp], scales s
 * [batch][Np / 128][Kp / 128], Np and Kp rounded up to 128 (zeros past K; a square
 * that holds a NaN or an infinity as a block that does); and of the transposed
 * weights (the same squares) qt [batch][K][Np], st [batch][Kp / 128][Np / 128], or
 * NULL.
 * Errors: EINVAL, EUNSUPPORTED (more than 65535 matrices or rows of squares). */
int mxgemm_block_quantize_weight(const void* w, int32_t type, int64_t ld, int64_t group, int64_t batch, int64_t N,
                                 int64_t K, int32_t format, uint8_t* q, float* s, uint8_t* qt, float* st, void* stream);

/* ---------------------------------------------------------------- product --
 * out = a w^T:  out[m][n] = sum over blocks b of K of
 *                a_scale[m][b] w_scale[n][b] (sum over k in b of a[m][k] w[n][k])
 * Each block's inner sum is formed by itself and added in FP32, times the FP32
 * product of its scales (which must be finite); one rounding to the output's
 * type.  Precision EXACT forms the inner sums of exactly converted codes on
 * the BF16 matrix unit (FP32 roundings), NATIVE on the FP8 one, which drops
 * products 2^13 times smaller than another of the same eight.
 *   a [rows][K], w [experts][N][K]  codes, 16-byte aligned, row strides lda,
 *       ldw and expert stride w_group in bytes (multiples of 16)
 *   a_scale [rows][K / 128]  any strides (elements; rows side by side are
 *       fastest, as mxgemm_block_quantize writes them)
 *   w_scale  squares: [experts][N / 128, rounded up][K / 128], as
 *       mxgemm_block_quantize_weight writes them; else [experts][N][K / 128]
 *   out [rows][N] of out_type (BF16, FP16, FP32), row stride ld_out elements
 *       (GROUP_INNER: [experts][rows][N], expert stride out_group)
 *   offsets, mode, experts  as for mxgemm_linear (mxgemm_moe.h)
 * K % 128 == 0.  GROUP_INNER takes no squares.
 * Errors: EINVAL, EUNSUPPORTED (row strides of a or w over 8 MiB, of scales
 * over 2^21 elements; a grid of 2^32 threads or more), EHIP.
 */
typedef struct mxgemm_block_linear {
    const void* a;
    const float* a_scale;
    const void* w;
    const float* w_scale;
    void* out;
    const int32_t* offsets;
    int64_t rows, N, K;
    int64_t lda, a_scale_row, a_scale_k, ldw, w_group, w_scale_row, w_scale_k, w_scale_group;
    int64_t ld_out, out_group;
    int32_t squares, mode, experts;
    int32_t a_format, w_format;   /* MXGEMM_FMT_*       */
    int32_t precision;            /* MXGEMM_PRECISION_* */
    int32_t out_type;
    int32_t tile_cfg;             /* -1: chosen by the sizes (tests force one, 0 .. 4) */
    void* workspace;              /* 16-byte aligned, or NULL                          */
    int64_t workspace_bytes;
} mxgemm_block_linear_t;

/* As mxgemm_linear_workspace: bytes with which a product that is not by expert
 * may split K over work-groups; without them it is formed unsplit. */
int64_t mxgemm_block_linear_workspace(int64_t rows, int64_t N, int64_t K);

int mxgemm_block_linear(const mxgemm_block_linear_t* args, void* stream);

/* ------------------------------------------------------------------- norm --
 * The end of one block and the start of the next, row by row:
 *   n = norm(x) post_weight         (post_weight NULL: n = x)
 *   r = residual + scale gate n     (residual, gate may be NULL: 0 and 1)
 *   y = norm(r) pre_weight          (pre_weight NULL: no y)
 *   norm(v) = (v - m) / sqrt(mean((v - m)^2) + eps), m = 0 (RMS) or v's mean
 *             (LAYER)
 * in FP32 (a row whose squares leave its range is normalised to 0); r is rounded
 * to its type first, and y is of the rounded r.  x, residual, r, y [rows][cols]
 * of `type`, row strides in elements, any alignment of the element type.  gate
 * [gate_rows][cols] of gate_type: row i for rows [i, i + 1) rows / gate_rows;
 * gate_rows divides rows; its row stride may be 0.  Weights [cols] of their types.
 * 1 <= cols <= 8192.
 *
 * Gradient, from d_y and d_r (either may be NULL: zero), x, and r as it was
 * written: d_x and d_residual (or NULL) of `type`, d_gate [gate_rows][cols] of
 * gate_type, d_post_weight and d_pre_weight float32 [cols]; each in FP32,
 * rounded once, sums over rows in an order of their own.  workspace:
 * mxgemm_add_norm_workspace() bytes, 4-byte aligned.
 * Errors: EINVAL, EUNSUPPORTED, EHIP.
 */
enum { MXGEMM_NORM_RMS = 0, MXGEMM_NORM_LAYER = 1 };

typedef struct mxgemm_norm {
    const void* x;
    const void* residual;
    const void* gate;
    const void* post_weight;
    const void* pre_weight;
    void* r;                      /* backward: read */
    void* y;
    const void* d_y;
    const void* d_r;
    void* d_x;
    void* d_residual;
    void* d_gate;
    float* d_post_weight;
    float* d_pre_weight;
    void* workspace;
    int64_t workspace_bytes;
    int64_t rows, cols, gate_rows;
    int64_t ld_x, ld_residual, ld_gate, ld_r, ld_y, ld_d_y, ld_d_r, ld_d_x, ld_d_residual;
    int32_t type, gate_type, post_type, pre_type, kind;
    float scale, eps;
    int32_t reserved;
} mxgemm_norm_t;

int mxgemm_add_norm(const mxgemm_norm_t* args, void* stream);
int mxgemm_add_norm_backward(const mxgemm_norm_t* args, void* stream);
int64_t mxgemm_add_norm_workspace(int64_t rows, int64_t cols, int64_t gate_rows);

#ifdef __cplusplus
}
#endif

#endif /* MXGEMM_BLOCK_H */
