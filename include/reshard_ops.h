/*
 * reshard_ops.h -- the expert layer over resharded weights (libreshard.so): routing to experts and its gradient,
 * quantization to 8-bit floating point in blocks of 128, the matrix product over such blocks, and the routed expert
 * feed-forward that uses them.
 *
 * A refit (reshard.h) leaves a generation rank with FP8 expert weights and their fp32 block scales
 * (reshard_plan_blockwise_fp8, 128 x 128 blocks) or with BF16 weights (reshard_quantize_blocks gives them that form);
 * these calls compute with them.
 *
 * Conventions
 *  - Sizes and strides are in elements. Rows are contiguous (innermost stride 1); a row stride may exceed the row.
 *  - 8-bit values are E4M3 (1 byte; +-448, no infinity). A block's value is code * scale.
 *      rows    (activations [rows, cols]):    scale [rows, ceil(cols / 128)], any two strides
 *      blocks  (weights [batch, rows, cols]): scale [batch, ceil(rows / 128), ceil(cols / 128)], dense
 *  - Types: RESHARD_BF16, RESHARD_F16, RESHARD_F32 (reshard.h). Sums, softmax statistics and scales are fp32.
 *  - Buffers are device memory of the current device, managed memory or page-locked host memory, caller-owned and valid
 *    until the stream reaches the end of the work; pageable host memory and another device's memory are refused. Outputs
 *    must not overlap inputs. Calls are asynchronous on `stream`, allocate no device memory, keep nothing
 *    between calls and may be captured into a CUDA graph.
 *  - Errors: RESHARD_OK or a RESHARD_ERR_* code (reshard.h); reshard_last_error() lists every violation. Nothing is
 *    enqueued on an error found in the arguments.
 *  - Results do not depend on the run: no floating-point atomics, every sum in a fixed order.
 */
#ifndef RESHARD_OPS_H
#define RESHARD_OPS_H

#include "reshard.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RESHARD_SCORE_SOFTMAX 0
#define RESHARD_SCORE_SIGMOID 1

#define RESHARD_ROUTE_MAX_EXPERTS 1024
#define RESHARD_ROUTE_MAX_K 32
#define RESHARD_MAX_GROUPS 512              /* experts on one rank */
#define RESHARD_MAX_SLOTS (1 << 30)         /* tokens * k */
#define RESHARD_MAX_EXTENT (1 << 30)        /* rows or columns of a matrix */

/*
 * reshard_route -- choose k experts per token.
 * logits [tokens, experts] (row_stride), bias [experts] fp32 or NULL. score s: softmax over the row or sigmoid.
 * Experts are ordered by s + bias (without a bias by the logit, which orders them as s does), the lowest index first
 * among equals. groups > 1 (dividing experts, at most 32): only the groups_kept groups whose group_top (1 or 2) best
 * experts have the largest sum of s + bias take part; equal sums go to the lowest group.
 * weights [tokens, k] fp32 = scale * s of the chosen (without the bias), divided by their sum where renormalize is
 * set (0 where that sum is 0); ids [tokens, k] int32, in order. A logit of -inf or NaN is never chosen and has score 0;
 * neither is an expert whose bias makes its key one of these; where fewer than k experts are left the id is -1 and the
 * weight 0. Scores are fp32: those that round or underflow to the same number are equal. A logit of +inf makes a softmax row's weights NaN.
 */
int reshard_route(const void *logits, int dtype, int64_t tokens, int experts, int64_t row_stride, const float *bias,
                  int score, int groups, int groups_kept, int group_top, int k, int renormalize, float scale,
                  float *weights, int32_t *ids, reshard_stream_t stream);

/*
 * reshard_route_backward -- the gradient to the logits of reshard_route's weights, the choice held fixed.
 * grad_weights [tokens, k] fp32, ids as reshard_route gave them (-1, or an id that is no expert: no gradient).
 * grad_logits [tokens, experts] in the logits' type is written whole. The bias has no gradient.
 */
int reshard_route_backward(const float *grad_weights, const void *logits, int dtype, int64_t tokens, int experts,
                           int64_t row_stride, const int32_t *ids, int k, int score, int renormalize, float scale,
                           void *grad_logits, int64_t grad_stride, reshard_stream_t stream);

/*
 * reshard_dispatch -- the slots (token * k + choice) sorted by expert, for experts first_expert .. first_expert + experts - 1.
 * offsets [experts + 1]: expert e's places are offsets[e] .. offsets[e + 1] - 1, its slots in ascending order.
 * order [slots]: the slot at each place (only the first offsets[experts] are written). position [slots]: each slot's
 * place, -1 for an id outside the range.
 */
int reshard_dispatch(const int32_t *ids, int64_t slots, int first_expert, int experts, int32_t *offsets,
                     int32_t *order, int32_t *position, reshard_stream_t stream);

/*
 * reshard_quantize_rows -- x [rows, cols] to E4M3 in blocks of 1 x 128; reshard_quantize_blocks -- w [batch, rows, cols]
 * in blocks of 128 x 128. With a the block's largest magnitude (at least 2^-100): scale = a * (1 / 448), value =
 * E4M3(x * ((1 / a) * 448)), each step rounded to fp32, the last to nearest even. A block that holds an infinity or NaN has scale and values NaN.
 */
int reshard_quantize_rows(const void *x, int dtype, int64_t rows, int64_t cols, int64_t row_stride, void *q,
                          int64_t q_stride, float *scale, int64_t scale_row_stride, int64_t scale_block_stride,
                          reshard_stream_t stream);
int reshard_quantize_blocks(const void *w, int dtype, int64_t batch, int64_t rows, int64_t cols, int64_t batch_stride,
                            int64_t row_stride, void *q, int64_t q_batch_stride, int64_t q_row_stride, float *scale,
                            reshard_stream_t stream);

/*
 * reshard_matmul_fp8 -- out[m, n] = sum over blocks b of a_scale[m, b] w_scale[n / 128, b] (sum over k in b of
 * a[m, k] w[n, k]): a [m, k] quantized by rows, w [groups, n, k] by blocks.
 * offsets NULL: groups must be 1. Otherwise offsets [groups + 1] int32 on the device, ascending from 0 to at most m (one that is not
 * counts as the nearest that is: within 0 .. m and not below those before it): rows
 * offsets[g] .. offsets[g + 1] - 1 meet w[g]; rows from offsets[groups] on are not written.
 * a_scale's strides are 0 where it is broadcast (one scale a row, or one in all).
 * a, w: 16-byte aligned, row strides (and w's batch stride) multiples of 16, w's matrices one after another. out [m, n] BF16, F16 or F32.
 * Each 128-block's products are summed by the tensor cores in fp32 and scaled and added in fp32 registers.
 * A gradient to the rows is the same product with w transposed (its blocks transpose with it).
 */
int reshard_matmul_fp8(const void *a, int64_t a_stride, const float *a_scale, int64_t a_scale_row, int64_t a_scale_block,
                       const void *w, int64_t w_batch_stride, int64_t w_stride, const float *w_scale,
                       const int32_t *offsets, int groups, int64_t m, int64_t n, int64_t k, void *out, int out_dtype,
                       int64_t out_stride, reshard_stream_t stream);

/*
 * reshard_linear_fp8 -- out = Q(x) w^T: x [m, k] quantized by rows, then the product with one weight matrix w [n, k].
 * workspace: reshard_linear_fp8_workspace(m, k) bytes, 256-byte aligned; 0 bytes (NULL will do) for the few rows that the
 * product quantizes on its way. out has x's type.
 */
int64_t reshard_linear_fp8_workspace(int64_t m, int64_t k);
int reshard_linear_fp8(const void *x, int dtype, int64_t m, int64_t k, int64_t row_stride, const void *w, int64_t w_stride,
                       const float *w_scale, int64_t n, void *out, int64_t out_stride, void *workspace,
                       int64_t workspace_bytes, reshard_stream_t stream);

/*
 * reshard_experts_fp8 -- the routed expert feed-forward of one rank:
 *   out[t] = sum over j of weights[t, j] * W2[e] Q(silu(g) * u),  [g; u] = W13[e] Q(x[t]),  e = ids[t, j] - first_expert,
 * over the choices with 0 <= e < experts (other ids, -1 among them, add nothing: another rank's, or no choice).
 * x, out [tokens, hidden] in dtype; ids, weights [tokens, k]; w13 [experts, 2 ffn, hidden] (gate rows, then up rows)
 * and w2 [experts, hidden, ffn] E4M3 with block scales, 16-byte aligned, row and batch strides multiples of 16.
 * ffn must be a multiple of 128, so that no block holds gate and up rows. silu(g) * u stays in fp32 until it is quantized,
 * each expert's output until the weighted sum, which is rounded to dtype once.
 * workspace: reshard_experts_fp8_workspace(...) bytes, 256-byte aligned; it has room for all tokens * k choices, since how
 * many are of this rank's experts is known on the device only.
 */
int64_t reshard_experts_fp8_workspace(int64_t tokens, int k, int experts, int64_t hidden, int64_t ffn, int dtype);
int reshard_experts_fp8(const void *x, int dtype, int64_t tokens, int64_t hidden, int64_t row_stride, const int32_t *ids,
                        const float *weights, int k, int first_expert, int experts, int64_t ffn, const void *w13,
                        int64_t w13_batch_stride, int64_t w13_stride, const float *w13_scale, const void *w2,
                        int64_t w2_batch_stride, int64_t w2_stride, const float *w2_scale, void *out, int64_t out_stride,
                        void *workspace, int64_t workspace_bytes, reshard_stream_t stream);

/*
 * reshard_ops_call -- one of the calls above with its arguments, in order, as 64-bit words (integers and pointers in `i`,
 * floats in `f`): for bindings in which marshalling each argument costs more than the call. op is a RESHARD_OP_* number;
 * another one is INVALID_ARG.
 */
#define RESHARD_OP_ROUTE 0
#define RESHARD_OP_ROUTE_BACKWARD 1
#define RESHARD_OP_DISPATCH 2
#define RESHARD_OP_QUANTIZE_ROWS 3
#define RESHARD_OP_QUANTIZE_BLOCKS 4
#define RESHARD_OP_MATMUL_FP8 5
#define RESHARD_OP_LINEAR_FP8 6
#define RESHARD_OP_EXPERTS_FP8 7
typedef union {
  int64_t i;
  double f;
} reshard_word_t;
int reshard_ops_call(int op, const reshard_word_t *args);

/*
 * reshard_ops_status -- the product kernels' status word on the current device (0 = fine; bit 0: a wait inside a
 * kernel gave up after its time limit and that launch's output is incomplete). Synchronizes the device, then reads
 * the word; reset != 0 clears it.
 */
int reshard_ops_status(int32_t *status, int reset);

#ifdef __cplusplus
}
#endif
#endif /* RESHARD_OPS_H */
