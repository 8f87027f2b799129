/*
 * mxgemm_moe -- the expert layer around the MXFP8 product, for AMD Instinct
 * MI355X (gfx950): tokens sorted by expert and back with their weights, and
 * the MXFP8 product with bias, activation and residual in its epilogue, dense
 * and by expert, each with its gradient.
 *
 * C ABI of the same library as mxgemm_seg.h, with the same error codes and
 * mxgemm_seg_last_error().  Every call is asynchronous on `stream` (a
 * hipStream_t passed as void*, NULL = the default stream), allocates nothing,
 * keeps nothing between calls, can be captured into a HIP graph and may run
 * concurrently with any other.  All pointers are device memory (or memory the
 * GPU can access; anything else is refused with MXGEMM_EINVAL) and must stay
 * valid until the work completes; buffer sizes are the caller's contract, and
 * so is that no output overlaps another operand.
 * Results do not depend on timing: no floating-point sum is formed by atomics
 * (the sort adds whole numbers with them).
 *
 * MXFP8 here is as in mxgemm_seg.h: FP8 codes (E4M3 or E5M2) in blocks of 32
 * along the inner axis with one E8M0 scale byte each, value = fp8(q) *
 * 2^(s - 127), a scale byte 0xFF making its block NaN.
 */
#ifndef MXGEMM_MOE_H
#define MXGEMM_MOE_H

#include <stdint.h>

#include "mxgemm_seg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types.  MXE4M3 / MXE5M2 (outputs only): MXFP8 codes with scales. */
enum { MXGEMM_TYPE_BF16 = 0, MXGEMM_TYPE_FP16 = 1, MXGEMM_TYPE_FP32 = 2, MXGEMM_TYPE_MXE4M3 = 3,
       MXGEMM_TYPE_MXE5M2 = 4 };

/* Activations, computed in FP32: max(z, 0); 0.5 z (1 + erf(z / sqrt 2));
 * 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))); z / (1 + exp(-z)).  Exponentials
 * and reciprocals are the hardware's (a unit in the last place; an exponential
 * also carries the rounding of its argument). */
enum { MXGEMM_ACT_NONE = 0, MXGEMM_ACT_RELU = 1, MXGEMM_ACT_GELU = 2, MXGEMM_ACT_GELU_TANH = 3,
       MXGEMM_ACT_SILU = 4 };

/*
 * Tokens sorted by expert.  ids [tokens][k] (int32, or int64 with id_bytes =
 * 8) names the experts of each token; a pair (token, choice) whose id is
 * outside [0, experts) is dropped.  The pairs are put in stable order by
 * expert, dropped pairs after the last expert:
 *   offsets   [experts + 1]  expert e holds rows [offsets[e], offsets[e+1]);
 *                            rows from offsets[experts] on are dropped pairs
 *   k_offsets [experts + 1]  the same with every expert's count rounded up to
 *                            128: the experts' segments of arrays blocked
 *                            along the tokens (mxgemm_epilogue_backward)
 *   row_of    [tokens][k]    row of each pair
 *   pair_of   [tokens * k]   pair (token * k + choice) of each row
 * workspace: mxgemm_sort_tokens_workspace() bytes, 4-byte aligned (may be
 * NULL where that is 0).  tokens >= 0, k >= 1, tokens * k < 2^31 - 2^20,
 * 1 <= experts <= 1024.  Errors: EINVAL, EUNSUPPORTED, EHIP.
 */
int mxgemm_sort_tokens(const void* ids, int32_t id_bytes, int64_t tokens, int32_t k, int32_t experts,
                       int32_t* offsets, int32_t* k_offsets, int32_t* row_of, int32_t* pair_of,
                       void* workspace, int64_t workspace_bytes, void* stream);
int64_t mxgemm_sort_tokens_workspace(int64_t tokens, int32_t k, int32_t experts);

/*
 * Rows of the sorted order from tokens: rows[row_of[t, j]] = x[t], zero for
 * dropped pairs (row_of >= offsets[experts], read on the device).  x
 * [tokens][cols] and rows [tokens * k][cols] of `type` (BF16, FP16, FP32)
 * with row strides ld_x, ld_rows in elements; any alignment of the element
 * type.  Errors: EINVAL, EUNSUPPORTED, EHIP.
 */
int mxgemm_dispatch_tokens(const void* x, int64_t ld_x, int32_t type, int64_t tokens, int32_t k, int64_t cols,
                           const int32_t* offsets, int32_t experts, const int32_t* row_of, void* rows,
                           int64_t ld_rows, void* stream);

/* The same into MXFP8 of `format` (MXGEMM_FMT_*): codes q [tokens * k][cols]
 * (16-byte aligned) and scale bytes s [tokens * k][cols / 32], quantised by
 * mxgemm_quantize_mx's rule (dropped pairs: code and scale bytes 0).
 * cols % 32 == 0. */
int mxgemm_dispatch_tokens_mx(const void* x, int64_t ld_x, int32_t type, int64_t tokens, int32_t k, int64_t cols,
                              const int32_t* offsets, int32_t experts, const int32_t* row_of, uint8_t* q,
                              uint8_t* s, int32_t format, void* stream);

/*
 * Tokens back from their rows: out[t] = residual[t] + sum over j of
 * weights[t, j] rows[row_of[t, j]], in FP32 in the order of j and rounded
 * once; dropped pairs add nothing whatever their weight or row holds.
 * weights: float32 [tokens][k], or NULL for ones (the gradient of
 * mxgemm_dispatch_tokens); residual may be NULL.  Errors as dispatch.
 */
int mxgemm_combine_tokens(const void* rows, int64_t ld_rows, int32_t type, int64_t tokens, int32_t k, int64_t cols,
                          const int32_t* offsets, int32_t experts, const int32_t* row_of, const float* weights,
                          const void* residual, int64_t ld_residual, void* out, int64_t ld_out, void* stream);

/*
 * Gradients of mxgemm_combine_tokens (the residual's is d_out itself):
 *   d_rows[row_of[t, j]] = weights[t, j] d_out[t]         (dropped: zero)
 *   d_weights[t, j] = <rows[row_of[t, j]], d_out[t]>      (dropped: zero)
 * d_rows of `type`, d_weights float32 [tokens][k], the sums in FP32.
 */
int mxgemm_combine_tokens_backward(const void* d_out, int64_t ld_d_out, const void* rows, int64_t ld_rows,
                                   int32_t type, int64_t tokens, int32_t k, int64_t cols, const int32_t* offsets,
                                   int32_t experts, const int32_t* row_of, const float* weights, void* d_rows,
                                   int64_t ld_d_rows, float* d_weights, void* stream);

/* How experts share a product (mxgemm_linear_t.mode). */
enum { MXGEMM_GROUP_NONE = 0,   /* one product                                                   */
       MXGEMM_GROUP_ROWS = 1,   /* rows [offsets[e], offsets[e+1]) of a times w[e]^T; rows from
                                   offsets[experts] on are zero in out and z                     */
       MXGEMM_GROUP_INNER = 2   /* out[e] = a w^T over inner range [offsets[e], offsets[e+1])
                                   (multiples of 128; an empty range gives zeros): the weights'
                                   gradient by expert                                            */ };

/*
 * out = act(z) + residual with z = a w^T + bias, or, gated, with N even,
 *       act(z[:, :N/2]) * z[:, N/2:] + residual.
 * The product is formed as mxgemm_seg_run does in the given precision mode
 * (FP32 sums); bias, activation, gate and residual are applied in FP32 and
 * rounded once.
 *   a [rows][K], w [experts][N][K]  codes, 16-byte aligned, row strides lda,
 *       ldw and expert stride w_group in bytes (multiples of 16)
 *   a_scale [rows][K/32], w_scale [experts][N][K/32]  4-byte aligned, strides
 *       multiples of 4 bytes
 *   bias [experts][N] of bias_type (BF16, FP16, FP32), or NULL
 *   residual [rows][cols], row stride ld_residual elements, of the output's
 *       type (BF16 where that is MXFP8), or NULL; cols = N, or N/2 if gated
 *   out [rows][cols], row stride ld_out elements (GROUP_INNER:
 *       [experts][rows][cols], expert stride out_group elements); MXFP8:
 *       codes with ld_out bytes (cols % 32 == 0, 8-byte aligned rows) and
 *       out_scale [rows][cols/32], row stride ld_out_scale
 *   z  bfloat16 [rows][N], row stride ld_z, or NULL: z kept for the gradient
 *   offsets  int32 [experts + 1] in device memory (modes ROWS and INNER),
 *       clamped to the rows (or K) there are
 * K % 128 == 0 (one MFMA K-step), as everywhere in this library.  GROUP_INNER
 * takes no bias, activation, gate, residual or z.
 * Errors: EINVAL, EUNSUPPORTED (K not a multiple of 128; row strides of a or w
 * over 8 MiB, of their scales over 4 MiB; a grid of 2^32 threads or more; gated
 * weights, or their scales, that span 4 GiB or more per expert), EHIP.
 */
typedef struct mxgemm_linear {
    const void* a;
    const void* a_scale;
    const void* w;
    const void* w_scale;
    const void* bias;
    const void* residual;
    void* out;
    void* out_scale;
    void* z;
    const int32_t* offsets;
    int64_t rows, N, K;
    int64_t lda, ld_a_scale, ldw, ld_w_scale, w_group, w_scale_group;
    int64_t ld_residual, ld_out, out_group, ld_out_scale, ld_z;
    int32_t mode, experts;
    int32_t a_format, w_format;   /* MXGEMM_FMT_*       */
    int32_t precision;            /* MXGEMM_PRECISION_* */
    int32_t bias_type, act, gated, out_type;
    int32_t tile_cfg;             /* -1: chosen by the sizes (tests force one, 0 .. 4) */
    void* workspace;              /* 16-byte aligned, or NULL                          */
    int64_t workspace_bytes;
} mxgemm_linear_t;

/* Bytes of workspace with which a product of these sizes that is not by
 * expert may split K over work-groups (their FP32 sums are added in order by
 * a second launch); 0 where it would not.  Without a workspace, or with a
 * smaller one, the product is formed unsplit. */
int64_t mxgemm_linear_workspace(int64_t rows, int64_t N, int64_t K);

int mxgemm_linear(const mxgemm_linear_t* args, void* stream);

/*
 * Gradient of mxgemm_linear's epilogue, held in MXFP8 of `format` both ways,
 * ready for the two products that finish the gradient:
 *   dz = d_out act'(z), or, gated, [d_out u act'(g), d_out act(g)] with
 *        [g, u] = z; in FP32 (relu: derivative 0 at 0)
 *   q, s    dz quantised along its columns: codes [rows][Np], scales
 *           [rows][Np/32], Np = N rounded up to 128 (zeros past N); d_a = dz w
 *           is mxgemm_linear of them with w transposed ([K][Np]); by expert, rows
 *           of dropped pairs are zero
 *   qt, st  dz transposed and quantised along the tokens: codes [N][ld_qt],
 *           scales [N][ld_qt/32]; by expert, expert e's tokens take columns
 *           [k_offsets[e], k_offsets[e+1]) (zeros past its last token, and past
 *           the last segment), else ld_qt is rows rounded up to 128; d_w = dz^T a is mxgemm_linear of
 *           them with a transposed ([K][ld_qt]), by expert in GROUP_INNER mode
 *           with k_offsets
 *   d_bias  float32 [experts][N] ([N] where not by expert): sums of dz over
 *           the tokens
 * Any of (q, s), (qt, st) and d_bias may be NULL.  d_out [rows][cols] of
 * d_type; z bfloat16 [rows][N], NULL only for act NONE and not gated (then
 * this quantises d_out itself, both ways, which is how a and w are laid out
 * transposed) or for no rows.  By expert: offsets, k_offsets int32
 * [experts + 1], ld_qt >= k_offsets[experts] and a multiple of 128; experts = 0
 * and NULL otherwise.
 * workspace: ld_qt/128 * N floats, needed for d_bias.
 * Errors: EINVAL, EUNSUPPORTED (more than 65534 chunks of 128 tokens in rows or
 * ld_qt, more than 65535 experts, N above 2^30 - 1024), EHIP.
 */
int mxgemm_epilogue_backward(const void* d_out, int32_t d_type, int64_t ld_d_out, const void* z, int64_t ld_z,
                             int64_t rows, int64_t N, int32_t act, int32_t gated, const int32_t* offsets,
                             const int32_t* k_offsets, int32_t experts, int32_t format, uint8_t* q, uint8_t* s,
                             uint8_t* qt, uint8_t* st, int64_t ld_qt, float* d_bias, void* workspace,
                             int64_t workspace_bytes, void* stream);

/*
 * Bytes transposed: dst [batch][cols][rows] from src [batch][rows][cols], row
 * stride ld_src, matrix stride src_batch (bytes): codes or scales held with
 * their inner axis strided, laid out for mxgemm_linear.  Any alignment.
 * Errors: EINVAL, EUNSUPPORTED (more than 65535 matrices or tiles of 128
 * rows, more than 2^31 - 128 columns), EHIP.
 */
int mxgemm_transpose_bytes(const void* src, int64_t ld_src, int64_t src_batch, int64_t rows, int64_t cols,
                           int64_t batch, void* dst, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXGEMM_MOE_H */
