/*
 * zc_moe.h -- C ABI of the mixture-of-experts operators around the compressed
 * all-to-all, MI355X (gfx950).
 *
 * zc.h codes the payload of an all-to-all; the calls here make that payload
 * and use it:
 *   routing    zc_route, zc_route_backward: expert scores -> experts and
 *              weights of every token
 *   exchange   zc_dispatch_plan, zc_dispatch: the token copies in expert order,
 *              which is the order of the per-destination segments that
 *              zc_compress_batch takes; zc_combine, zc_combine_backward: the
 *              weighted sum of a token's copies and its gradients (the gradient
 *              of zc_dispatch is zc_combine without weights)
 *   product    zc_fp8_quantize, zc_fp8_quantize_t, zc_fp8_transpose,
 *              zc_fp8_matmul, zc_fp8_matmul_wgrad: the experts' products in
 *              8-bit floating point with a scale for each block of 128; the
 *              8-bit input is the checkpoint that the weight gradient reads
 *   activation zc_swiglu, zc_swiglu_backward: the gated activation between two
 *              products, its input kept in 8 bits for the backward pass
 * and what stands between them in a whole block, from residual to residual:
 *   norm       zc_norm, zc_norm_backward: the norm of a block's output, its gate
 *              and scale, the residual sum, and the norm before the next block
 *   product    zc_matmul, zc_activation_backward, zc_matmul_dgrad,
 *              zc_matmul_wgrad: BF16 products with bias, activation and residual
 *              in their epilogue (the router's logits, a shared expert, dense
 *              projections)
 *   balance    zc_balance, zc_balance_backward: copies of every expert, the
 *              balance loss and the z loss of every sequence
 *
 * Conventions: those of zc.h (caller-owned buffers, no allocation, no
 * synchronization, no state between calls, device work is kernel launches
 * only, so every call may be captured into a HIP graph; host-detectable errors
 * return before anything is enqueued).  Beyond that:
 *   - strides are counted in elements of the array they belong to, and are at
 *     least the row's length; buffers of an 8-bit type or scales have the fixed
 *     layout below;
 *   - token counts, row counts and tokens * top_k are at most 2^31 - 1 -
 *     ZC_MOE_ROW_SLACK; addresses are computed in 64 bits;
 *   - a count of zero (tokens, rows, groups) is valid and enqueues nothing
 *     unless the description says that something is written;
 *   - every output is a pure function of the inputs: sums have an order fixed
 *     by the sizes, no atomic adds floating-point numbers;
 *   - indices that the device reads (expert ids, positions, offsets) are
 *     checked there: one out of range is treated as the description of the call
 *     says, and never read or written through.
 * Alignment: 2-byte elements need 2-byte, 4-byte elements 4-byte aligned
 * buffers, as do scales; 8-bit arrays and workspaces 16-byte.  BF16 arrays
 * that start on 16 bytes with row lengths and strides that are multiples of 8
 * take the wide path.
 *
 * 8-bit blocks.  128 consecutive values of a row (or a square of 128 x 128)
 * share one scale 2^(b - 127), kept as the byte b (0..247): the smallest power
 * of two at which the largest finite magnitude of the block is at most the
 * type's largest value (448 for e4m3, 57344 for e5m2; b = 0 for a block of
 * zeros).  A value is stored as v / scale rounded to the type, to nearest with
 * ties to even; since the scale is a power of two this is its only rounding.
 * NaN and infinities keep their kind (e4m3 has no infinity: NaN), and do not
 * enter the scale.  A magnitude from 1.9375 * 2^127 (e4m3) or 1.875 * 2^127 (e5m2)
 * up rounds to 2^128, which BF16 and floats cannot hold: full sums,
 * zc_fp8_quantize_t from 8 bits and zc_swiglu_backward take it as an infinity.
 * Power-of-two scales are what the scaled matrix instructions of gfx950 apply by
 * themselves.
 *   values  rows of zc_fp8_stride(cols) bytes: cols rounded up to 128, the
 *           bytes past cols are zero
 *   scales  rows of zc_fp8_scale_stride(cols) bytes: ceil(cols / 128) of them
 *           used, the rest zero; one row of scales per row of values, or per
 *           128 rows for squares
 */
#ifndef ZC_MOE_H
#define ZC_MOE_H

#include <stdint.h>

#include "zc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define ZC_F32 0u
#define ZC_BF16 1u
#define ZC_FP8_E4M3 2u
#define ZC_FP8_E5M2 3u

/* How a product of 8-bit matrices is summed.  FAST: the 8-bit matrix
 * instructions.  They align the products of a few neighbouring values of a row
 * to the largest of them and drop what lies about 12 binary digits below it;
 * the sums of those are kept in 32 bits.  Measured against exact products:
 * 1.4e-5 of the result on Gaussian values, a hundredth of what rounding it to BF16 costs.
 * FULL: the values, with their scales, as BF16 (exact) through the BF16 matrix
 * instructions, whose products are exact and whose sums have 32 bits; half the
 * matrix rate. */
#define ZC_FP8_SUM_FAST 0u
#define ZC_FP8_SUM_FULL 1u

#define ZC_SCORE_SOFTMAX 0u
#define ZC_SCORE_SIGMOID 1u

#define ZC_NORM_NONE 0u
#define ZC_NORM_RMS 1u
#define ZC_NORM_LAYER 2u

#define ZC_ACT_NONE 0u
#define ZC_ACT_RELU 1u
#define ZC_ACT_SILU 2u
#define ZC_ACT_GELU 3u
#define ZC_ACT_GELU_TANH 4u
#define ZC_ACT_SIGMOID 5u

#define ZC_NORM_MAX_COLS 16384u
#define ZC_MAX_SEQUENCES 1024u
/* neither zc_matmul_workspace_bytes nor zc_balance_workspace_bytes is ever more than this */
#define ZC_MATMUL_WORKSPACE_MAX (64ull << 20)
#define ZC_BALANCE_WORKSPACE_MAX (64ull << 20)

#define ZC_MAX_EXPERTS 1024u
#define ZC_MAX_TOP_K 32u
#define ZC_MAX_EXPERT_GROUPS 64u
#define ZC_FP8_BLOCK 128u
#define ZC_MOE_ROW_SLACK 262144u
/* zc_fp8_matmul never asks for more workspace than this */
#define ZC_FP8_MATMUL_WORKSPACE_MAX (64ull << 20)

/* How a token's experts are chosen.
 *   s = softmax or sigmoid of the token's logits; c = s + bias (the bias, for
 *   balance, enters the choice only); with groups > 1, a group (experts /
 *   groups consecutive experts) scores the sum of its `group_score` largest c,
 *   and the `group_top` best groups stay; the top_k largest c of the experts
 *   that stay are chosen, in descending order.  Every tie goes to the lower
 *   index.  Weight of a chosen expert: scale * s, or scale * s / (sum of the
 *   chosen s + 1e-20) with renormalise.
 * The choice is made on 64-bit scores, so that it does not depend on how a
 * 32-bit exponential rounds; weights are 32-bit. */
typedef struct zc_route_config {
    uint32_t experts;     /* 1..ZC_MAX_EXPERTS */
    uint32_t top_k;       /* 1..ZC_MAX_TOP_K, at most group_top * experts / groups */
    uint32_t score;       /* ZC_SCORE_SOFTMAX or ZC_SCORE_SIGMOID */
    uint32_t groups;      /* 1..ZC_MAX_EXPERT_GROUPS, divides experts */
    uint32_t group_top;   /* 1..groups */
    uint32_t group_score; /* 1 or 2 (2 on groups of one expert acts as 1) */
    uint32_t renormalise; /* 0 or 1 */
    float scale;          /* finite */
} zc_route_config;

/* Experts and weights of every token.
 *   d_logits    device, tokens rows of cfg->experts values of logits_type
 *               (ZC_F32 or ZC_BF16), stride logits_stride
 *   d_bias      device, cfg->experts floats, or NULL
 *   d_ids       device, tokens x top_k int32
 *   d_weights   device, tokens x top_k floats
 * Special values: a logit of -inf scores 0 (a row of nothing else has weights
 * 0 and, with no finite bias to tell them apart, the lowest ids); c = NaN or
 * -inf ranks below every other c, ties to the lower index; a NaN score shows
 * in the weights it enters (a softmax row with NaN or +inf is all NaN).
 * Errors: ZC_ERR_INVALID_ARG, ZC_ERR_MISALIGNED, ZC_ERR_HIP. */
zc_status zc_route(const void *d_logits, uint32_t logits_type, uint64_t tokens, uint64_t logits_stride,
                   const float *d_bias, const zc_route_config *cfg, int32_t *d_ids, float *d_weights, void *stream);

/* Gradient of the logits from the gradient of the weights (d_dweights, tokens x
 * top_k) for the experts d_ids that zc_route chose.  The choice itself has no
 * gradient; an id outside 0..experts-1 takes no part.  d_dlogits (logits_type,
 * stride dlogits_stride) receives all cfg->experts values of every row.  A row
 * of -inf logits gets zeros. */
zc_status zc_route_backward(const void *d_logits, uint32_t logits_type, uint64_t tokens, uint64_t logits_stride,
                            const zc_route_config *cfg, const int32_t *d_ids, const float *d_dweights,
                            void *d_dlogits, uint64_t dlogits_stride, void *stream);

/* Workspace of zc_dispatch_plan (a multiple of 256; 0 for invalid sizes). */
uint64_t zc_dispatch_workspace_bytes(uint64_t tokens, uint32_t top_k, uint32_t experts);

/* The order of the token copies by expert: a copy is a pair (token, k) with the
 * expert d_ids[token * top_k + k]; copies of one expert keep their order.  An
 * id outside 0..experts-1 drops its copy.
 *   d_offsets   device, experts + 1 int32: the copies of expert e take the rows
 *               [d_offsets[e], d_offsets[e + 1])
 *   d_position  device, tokens x top_k int32: a copy's row, or -1 if dropped
 *   d_source    device, tokens * top_k int32, or NULL: the copy (token * top_k
 *               + k) of a row, -1 past the last row
 * With tokens = 0 the offsets are written (zeros). */
zc_status zc_dispatch_plan(const int32_t *d_ids, uint64_t tokens, uint32_t top_k, uint32_t experts,
                           void *d_workspace, uint64_t workspace_bytes, int32_t *d_offsets, int32_t *d_position,
                           int32_t *d_source, void *stream);

/* The payload: d_out[d_position[t, k], :] = d_x[t, :] for every copy that is
 * not dropped (position outside 0..rows-1: dropped).  BF16, hidden values a
 * row.  Rows that no copy names are left as they are. */
zc_status zc_dispatch(const void *d_x, uint64_t tokens, uint64_t hidden, uint64_t x_stride,
                      const int32_t *d_position, uint32_t top_k, void *d_out, uint64_t rows, uint64_t out_stride,
                      void *stream);

/* d_y[t, :] = sum over k, ascending, of d_weights[t, k] * d_z[d_position[t, k], :],
 * in 32 bits, rounded to BF16 once; dropped copies take no part (a token
 * without copies gets zeros).  d_weights NULL: all 1, which is the gradient of
 * zc_dispatch. */
zc_status zc_combine(const void *d_z, uint64_t rows, uint64_t hidden, uint64_t z_stride, const int32_t *d_position,
                     const float *d_weights, uint64_t tokens, uint32_t top_k, void *d_y, uint64_t y_stride,
                     void *stream);

/* Gradients of zc_combine from d_dy (tokens rows): d_dz[d_position[t, k], :] =
 * d_weights[t, k] * d_dy[t, :] (rows that no copy names are left as they are)
 * and d_dweights[t, k] = sum over h of d_dy[t, h] * d_z[position, h] in 32 bits
 * (0 for a dropped copy).  Either output may be NULL; d_z is needed for
 * d_dweights only, d_weights (NULL: all 1) for d_dz only. */
zc_status zc_combine_backward(const void *d_dy, uint64_t dy_stride, const void *d_z, uint64_t rows, uint64_t hidden,
                              uint64_t z_stride, const int32_t *d_position, const float *d_weights,
                              uint64_t tokens, uint32_t top_k, void *d_dz, uint64_t dz_stride, float *d_dweights,
                              void *stream);

/* Row strides of 8-bit arrays: cols rounded up to 128 bytes, and
 * ceil(cols / 128) rounded up to 4 bytes. */
uint64_t zc_fp8_stride(uint64_t cols);
uint64_t zc_fp8_scale_stride(uint64_t cols);

/* BF16 rows to 8-bit blocks along the rows (block_rows 1: inputs, gradients),
 * or to 128 x 128 squares (block_rows 128: weights).
 *   type  ZC_FP8_E4M3 or ZC_FP8_E5M2
 *   d_q       rows x zc_fp8_stride(cols) bytes
 *   d_scales  rows (or ceil(rows / 128)) x zc_fp8_scale_stride(cols) bytes */
zc_status zc_fp8_quantize(const void *d_x, uint64_t rows, uint64_t cols, uint64_t x_stride, uint32_t type,
                          uint32_t block_rows, void *d_q, uint8_t *d_scales, void *stream);

/* Columns that hold every group's rows when each group starts on a block of
 * 128: an upper bound for any split of `rows` into `groups`. */
uint64_t zc_fp8_padded_rows(uint64_t rows, uint32_t groups);

/* The transposed 8-bit form, blocks of 128 along the rows (tokens) of d_x: the
 * operands of zc_fp8_matmul_wgrad.
 *   d_x       x_type ZC_BF16: rows x cols, stride x_stride; an 8-bit x_type: the
 *             checkpoint that zc_fp8_quantize made with block_rows 1 (x_stride
 *             = zc_fp8_stride(cols)), with its d_x_scales
 *   groups, d_offsets  rows [d_offsets[g], d_offsets[g + 1]) are group g
 *             (groups + 1 int32, ascending; values are clamped to 0..rows and
 *             to ascending order); NULL with groups 1: all rows
 *   type      of the result
 *   d_q       cols rows of padded_rows bytes.  Group g's rows start at the
 *             column 128 * (sum over the groups before it of ceil(their rows /
 *             128)), its columns past its last row are zero; columns past the
 *             last group's are left as they are
 *   d_scales  cols rows of zc_fp8_scale_stride(padded_rows) bytes
 *   padded_rows  a multiple of 128, at least zc_fp8_padded_rows(rows, groups) */
zc_status zc_fp8_quantize_t(const void *d_x, const uint8_t *d_x_scales, uint32_t x_type, uint64_t rows,
                            uint64_t cols, uint64_t x_stride, uint32_t groups, const int32_t *d_offsets,
                            uint32_t type, void *d_q, uint8_t *d_scales, uint64_t padded_rows, void *stream);

/* Transposes `batch` matrices of 128 x 128 squares (weights): rows x cols to
 * cols x rows, values and scales unchanged; the weights of the gradient of a
 * product's input.  Row strides as zc_fp8_stride; consecutive matrices follow
 * each other without a gap (rows x zc_fp8_stride(cols) bytes, ceil(rows / 128)
 * x zc_fp8_scale_stride(cols) scales, and the same of the result). */
zc_status zc_fp8_transpose(const void *d_q, const uint8_t *d_scales, uint64_t batch, uint64_t rows, uint64_t cols,
                           void *d_qt, uint8_t *d_scales_t, void *stream);

/* Workspace with which zc_fp8_matmul may split the contraction of a product
 * with few rows (0: it does not; at most ZC_FP8_MATMUL_WORKSPACE_MAX). */
uint64_t zc_fp8_matmul_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, uint32_t groups);

/* Grouped product: d_out[r, c] = sum over k of A[r, k] * B_g[c, k] for the rows
 * r of group g, rounded to out_type (ZC_BF16 or ZC_F32) once.
 *   A  m rows of k values, blocks of 128 along the rows (zc_fp8_quantize,
 *      block_rows 1)
 *   B  groups matrices of n rows of k values in 128 x 128 squares, one after
 *      another (n x zc_fp8_stride(k) bytes, ceil(n / 128) x
 *      zc_fp8_scale_stride(k) scales each)
 *   groups, d_offsets  as in zc_fp8_quantize_t; rows of no group are left as
 *      they are
 *   d_workspace, workspace_bytes  16-byte aligned, or NULL: no split.  A
 *      workspace smaller than zc_fp8_matmul_workspace_bytes is not used.
 *   sum_mode  ZC_FP8_SUM_FAST or ZC_FP8_SUM_FULL (products bound by reading the
 *      weights are summed in full in either mode)
 * a_type and b_type are each e4m3 or e5m2; k = 0 gives zeros; k is at most
 * 2^24. */
zc_status zc_fp8_matmul(const void *d_a, const uint8_t *d_a_scales, uint32_t a_type, uint64_t m, const void *d_b,
                        const uint8_t *d_b_scales, uint32_t b_type, uint64_t n, uint64_t k, uint32_t groups,
                        const int32_t *d_offsets, void *d_out, uint32_t out_type, uint64_t out_stride,
                        uint32_t sum_mode, void *d_workspace, uint64_t workspace_bytes, void *stream);

/* Weight gradients, one n x k matrix per group, contracted over the group's
 * rows: d_out[g, i, j] = sum over the rows r of group g of A[i, r] * B[j, r].
 *   A, B  n and k rows of padded_rows bytes from zc_fp8_quantize_t with the
 *         same rows, groups and d_offsets (padded_rows at most 2^24)
 *   d_out groups x n x k values of out_type, contiguous; zeros for a group
 *         without rows */
zc_status zc_fp8_matmul_wgrad(const void *d_a, const uint8_t *d_a_scales, uint32_t a_type, uint64_t n,
                              const void *d_b, const uint8_t *d_b_scales, uint32_t b_type, uint64_t k,
                              uint64_t padded_rows, uint64_t rows, uint32_t groups, const int32_t *d_offsets,
                              void *d_out, uint32_t out_type, uint32_t sum_mode, void *stream);

/* Gated activation of rows (gate_0..gate_{cols-1}, up_0..up_{cols-1}), BF16:
 *   h = gate * sigmoid(gate) * up, in 32 bits, rounded to BF16.
 * Any of the three results may be NULL:
 *   d_h                 BF16, stride h_stride
 *   d_hq, d_hq_scales   the 8-bit e4m3 blocks that zc_fp8_quantize makes of h:
 *                       the input of the next product
 *   d_kept, d_kept_scales  the checkpoint: e4m3 blocks of the gates, then of
 *                       the ups, each half cols rounded up to 128 (a row of
 *                       2 * zc_fp8_stride(cols) bytes, and
 *                       zc_fp8_scale_stride(2 * zc_fp8_stride(cols)) scales) */
zc_status zc_swiglu(const void *d_gate_up, uint64_t rows, uint64_t cols, uint64_t gu_stride, void *d_h,
                    uint64_t h_stride, void *d_hq, uint8_t *d_hq_scales, void *d_kept, uint8_t *d_kept_scales,
                    void *stream);

/* Gradient of zc_swiglu's input from d_dh (BF16, rows x cols), evaluated at the
 * kept values: dgate = dh * up * s * (1 + gate * (1 - s)), dup = dh * gate * s
 * with s = sigmoid(gate); written as BF16 rows of 2 * cols values. */
zc_status zc_swiglu_backward(const void *d_kept, const uint8_t *d_kept_scales, uint64_t rows, uint64_t cols,
                             const void *d_dh, uint64_t dh_stride, void *d_dgate_up, uint64_t gu_stride,
                             void *stream);

/* One norm: kind NONE (N(v) = v; nothing else of it is read), RMS: N(v)[c] =
 * w[c] * v[c] / sqrt(mean(v^2) + eps) + b[c], or LAYER: the same of v - mean(v).
 * eps is a finite normal number above 0. */
typedef struct zc_norm_params {
    const void *d_weight; /* cols values of `type`, or NULL: all 1 */
    const void *d_bias;   /* cols values of `type`, or NULL: all 0 */
    uint32_t kind;        /* ZC_NORM_ */
    uint32_t type;        /* ZC_F32 or ZC_BF16 */
    float eps;
} zc_norm_params;

/* What stands between two blocks of a residual stream:
 *   h = after(z);  r[t, c] = x[t, c] + scale * row_gate[t] * gate[c] * h[t, c];  y = before(r) */
typedef struct zc_norm_config {
    zc_norm_params after;  /* the norm of the block's output z */
    zc_norm_params before; /* the norm of the sum r, before the next block */
    const void *d_gate;    /* cols values of gate_type, or NULL: all 1 */
    const float *d_row_gate; /* rows floats, or NULL: all 1 */
    uint32_t gate_type;    /* ZC_F32 or ZC_BF16 */
    float scale;           /* finite */
} zc_norm_config;

/* Norms, gate and residual sum in one pass over the rows; statistics and sums
 * in 32 bits, each result rounded once (y comes from r before r is rounded).
 *   d_x     the residual stream, stream_type ZC_BF16 or ZC_F32
 *   d_z     BF16, or NULL: no block output, r = x (cfg->after, the gates and the
 *           scale are not read)
 *   d_r     stream_type, or NULL; may be d_x with the same stride
 *   d_y     BF16, or NULL
 *   d_yq, d_yq_scales  the 8-bit e4m3 blocks that zc_fp8_quantize makes of y: the
 *           input of the next product; or NULL
 * cols is at most ZC_NORM_MAX_COLS.  A finite row has finite statistics also
 * where its squares leave the range of a float.  A row that holds NaN or an infinity:
 * what the formula gives, NaN where it has no value. */
zc_status zc_norm(const void *d_x, uint32_t stream_type, uint64_t rows, uint64_t cols, uint64_t x_stride,
                  const void *d_z, uint64_t z_stride, const zc_norm_config *cfg, void *d_r, uint64_t r_stride,
                  void *d_y, uint64_t y_stride, void *d_yq, uint8_t *d_yq_scales, void *stream);

/* Gradients of the parameters, sums over the rows in 32 bits; any may be NULL.
 * Those of a norm of kind NONE, or without d_z those of the whole first half, are zeros. */
typedef struct zc_norm_grads {
    float *d_weight_after, *d_bias_after, *d_gate; /* cols floats each */
    float *d_weight_before, *d_bias_before;        /* cols floats each */
    float *d_row_gate;                             /* rows floats */
} zc_norm_grads;

/* Workspace of zc_norm_backward: the parts of the sums over the rows (a
 * multiple of 256; 0 for invalid sizes). */
uint64_t zc_norm_backward_workspace_bytes(uint64_t rows, uint64_t cols);

/* Gradients of zc_norm, evaluated at the stored sum d_r (stream_type).
 *   d_dr   gradient that arrives at r beside y's, stream_type, or NULL: 0
 *   d_dy   BF16, or NULL: 0
 *   d_dx   stream_type, or NULL: the whole gradient of r, which is that of x; may
 *          be d_dr with the same stride
 *   d_dz   BF16, or NULL
 * d_workspace is needed where a parameter's gradient over the rows is asked for. */
zc_status zc_norm_backward(const void *d_r, uint32_t stream_type, uint64_t rows, uint64_t cols, uint64_t r_stride,
                           const void *d_z, uint64_t z_stride, const zc_norm_config *cfg, const void *d_dr,
                           uint64_t dr_stride, const void *d_dy, uint64_t dy_stride, void *d_dx, uint64_t dx_stride,
                           void *d_dz, uint64_t dz_stride, const zc_norm_grads *grads, void *d_workspace,
                           uint64_t workspace_bytes, void *stream);

/* What zc_matmul does with a sum v before it leaves:
 *   pre = v + bias;  out = residual + scale * activation(pre)
 * activation: NONE, RELU, SILU v * sigmoid(v), GELU v * Phi(v) (the normal
 * distribution), GELU_TANH v * (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2,
 * SIGMOID.  At infinities all but NONE have their limits, and so have their slopes: 0 and
 * 0 at -inf, +inf and 1 at +inf (SIGMOID: 1 and 0); NaN stays NaN. */
typedef struct zc_epilogue {
    const void *d_bias;       /* cols values of bias_type, or NULL: 0 */
    const void *d_residual;   /* rows of residual_type, or NULL: 0; may be the output, with its type and stride */
    void *d_pre;              /* BF16, or NULL: pre, kept for zc_activation_backward */
    uint64_t residual_stride;
    uint64_t pre_stride;
    uint32_t bias_type;       /* ZC_F32 or ZC_BF16 */
    uint32_t residual_type;   /* ZC_F32 or ZC_BF16 */
    uint32_t activation;      /* ZC_ACT_ */
    float scale;              /* finite */
} zc_epilogue;

/* Workspace with which a product of rows x cols results over `contraction`
 * values may be split (0: it is not; at most ZC_MATMUL_WORKSPACE_MAX): (m, n, k) for zc_matmul, (m,
 * k, n) for zc_matmul_dgrad, (n, k, m) for zc_matmul_wgrad. */
uint64_t zc_matmul_workspace_bytes(uint64_t rows, uint64_t cols, uint64_t contraction);

/* d_out[r, c] = epilogue(sum over k of A[r, k] * W[c, k]), A (m x k) and W (n x
 * k) BF16; products are exact, sums in 32 bits, d_out (out_type ZC_BF16 or
 * ZC_F32) and pre rounded once.  epilogue NULL: the sum itself.  k = 0: a sum of nothing
 * is 0, and the epilogue is applied.  A workspace smaller than
 * zc_matmul_workspace_bytes is not used; NULL: no split.  n and k are at most 2^28, and results of
 * more than 2^24 tiles of 128 x 128 (256 x 256 on 16-byte aligned rows) are refused. */
zc_status zc_matmul(const void *d_a, uint64_t m, uint64_t a_stride, const void *d_w, uint64_t n, uint64_t k,
                    uint64_t w_stride, const zc_epilogue *epilogue, void *d_out, uint32_t out_type,
                    uint64_t out_stride, void *d_workspace, uint64_t workspace_bytes, void *stream);

/* Workspace of zc_activation_backward for d_dbias (a multiple of 256; 0 for invalid sizes). */
uint64_t zc_activation_backward_workspace_bytes(uint64_t rows, uint64_t cols);

/* From the gradient of zc_matmul's output (dout_type ZC_BF16 or ZC_F32) to that
 * of its pre-activation: dpre = scale * dout * activation'(pre) at the kept pre
 * (BF16; not read for NONE), rounded to BF16; d_dbias[c] = sum over the rows of
 * dpre before that rounding, in 32 bits.  The slope of RELU at 0 is 0.  Either
 * result may be NULL; d_dpre may be d_dout where that is BF16, or d_pre, with the
 * same stride.  d_workspace is needed for d_dbias. */
zc_status zc_activation_backward(const void *d_dout, uint32_t dout_type, uint64_t rows, uint64_t cols,
                                 uint64_t dout_stride, const void *d_pre, uint64_t pre_stride, uint32_t activation,
                                 float scale, void *d_dpre, uint64_t dpre_stride, float *d_dbias, void *d_workspace,
                                 uint64_t workspace_bytes, void *stream);

/* Gradient of zc_matmul's A: d_dx[r, j] = add[r, j] + sum over c of dpre[r, c] *
 * W[c, j] (m x k; dpre m x n BF16).  d_add: add_type, NULL: 0; may be d_dx with
 * its type and stride.  Sums, results and workspace as in zc_matmul. */
zc_status zc_matmul_dgrad(const void *d_dpre, uint64_t m, uint64_t n, uint64_t dpre_stride, const void *d_w,
                          uint64_t k, uint64_t w_stride, const void *d_add, uint32_t add_type, uint64_t add_stride,
                          void *d_dx, uint32_t dx_type, uint64_t dx_stride, void *d_workspace,
                          uint64_t workspace_bytes, void *stream);

/* Gradient of zc_matmul's W: d_dw[c, j] = add[c, j] + sum over r of dpre[r, c] *
 * A[r, j] (n x k).  d_add, for gradients that add up over calls, as above. */
zc_status zc_matmul_wgrad(const void *d_dpre, uint64_t m, uint64_t n, uint64_t dpre_stride, const void *d_a,
                          uint64_t k, uint64_t a_stride, const void *d_add, uint32_t add_type, uint64_t add_stride,
                          void *d_dw, uint32_t dw_type, uint64_t dw_stride, void *d_workspace,
                          uint64_t workspace_bytes, void *stream);

/* Workspace of zc_balance (a multiple of 256; 0 for invalid sizes). */
uint64_t zc_balance_workspace_bytes(uint64_t tokens, uint32_t experts, uint32_t sequences);

/* Copies of every expert, balance loss and z loss of every sequence.  Of cfg,
 * only experts, top_k and score are read.  Sequence s: the tokens [d_offsets[s],
 * d_offsets[s + 1]) (sequences + 1 int32, ascending; values are clamped to
 * 0..tokens and to ascending order; NULL with sequences 1: all tokens) whose
 * d_mask is not 0 (tokens bytes; NULL: all).  With p = the softmax of a token's
 * logits, or sigmoid / (sum of its sigmoids + 1e-20):
 *   d_used[s]       its tokens, n
 *   d_counts[s, e]  its copies with d_ids = e (tokens x top_k int32; an id outside
 *                   0..experts-1 counts nowhere)
 *   d_loss[s]       experts / (top_k n^2) * sum over e of counts[s, e] * sum over its tokens of p[t, e]
 *   d_zloss[s]      1 / n * sum over its tokens of (log of the sum over e of exp(logits[t, e]))^2
 * Without tokens the losses are 0.  The losses may be NULL, and then d_logits
 * too.  A token whose logits are all -inf has p = 0 and no part in the z loss; +inf makes its
 * sequence's z loss infinite, and the softmax of its token NaN, NaN all of its sequence's.
 * sequences is at most ZC_MAX_SEQUENCES; with tokens = 0 everything is written (zeros). */
zc_status zc_balance(const void *d_logits, uint32_t logits_type, uint64_t tokens, uint64_t logits_stride,
                     const zc_route_config *cfg, const int32_t *d_ids, const uint8_t *d_mask, uint32_t sequences,
                     const int32_t *d_offsets, void *d_workspace, uint64_t workspace_bytes, int32_t *d_counts,
                     int32_t *d_used, float *d_loss, float *d_zloss, void *stream);

/* Gradient of the logits from the gradients of the losses (sequences floats
 * each; NULL: 0), for the counts and used that zc_balance wrote (the counts have no
 * gradient): d_dlogits[t, :] = add[t, :] + that of token t's sequence; a token of no sequence, or
 * masked, has add alone.  d_add: logits_type, NULL: 0 (the gradient of
 * zc_route_backward); may be d_dlogits with the same stride. */
zc_status zc_balance_backward(const void *d_logits, uint32_t logits_type, uint64_t tokens, uint64_t logits_stride,
                              const zc_route_config *cfg, const uint8_t *d_mask, uint32_t sequences,
                              const int32_t *d_offsets, const int32_t *d_counts, const int32_t *d_used,
                              const float *d_dloss, const float *d_dzloss, const void *d_add, uint64_t add_stride,
                              void *d_dlogits, uint64_t dlogits_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZC_MOE_H */
