/*
 * moe_experts.h -- C ABI of a block's own operators: the gated feed-forward of experts on rows sorted by
 * expert (or of a dense block: one expert), rows kept in 8 bits for the backward pass, and the norms
 * around a block with its gate and residual scale, each with its gradient
 * (library: expert_offload_lru_amd/libmoe_offload.so).
 *
 * moe_layer_forward (moe_offload.h) runs frozen 4-bit experts; these entry points are for experts that a
 * caller trains, or serves in its own types, on the rows of moe_tokens_dispatch (moe_tokens.h).  A training
 * step is: moe_block_norm, moe_tokens_dispatch, moe_experts_hidden, moe_experts_product,
 * moe_tokens_combine, and back through the same.  Adapters (moe_adapters_forward with the product as its base)
 * go beside moe_experts_product; moe_experts_hidden takes none beside its projections, which it joins before
 * anything is written.
 *
 * Conventions: those of moe_tokens.h (streams, captured graphs, strides, overlaps, errors, indexes checked
 * on the device, the same bits from the same inputs), and
 *  - dtype (MOE_T_*) is the type of every tensor without a type of its own.  Sums are held in fp32, a
 *    result is rounded once; inf and NaN take part in sums and products as they do in fp32.
 *  - offsets [n_experts + 1] as written by moe_tokens_dispatch: rows offsets[e] .. offsets[e+1] are
 *    expert e's.  An offset counts as at least the ones before it, and as between 0 and n_rows.  Rows
 *    before offsets[0] and from offsets[n_experts] on are not read, and left as they were in an output.
 *  - Weights are contiguous [n_experts x outer x inner], of dtype.
 *  - Rows kept in 8 bits: codes int8 [rows x cols], scales uint8 [rows x ceil(cols / 32)], with ld of their
 *    own.  Column c of a row has the value codes[c] * 2^(scales[c / 32] - 133): an int8 block of 32 with a
 *    shared power of two.  The scale is the least (of 0 .. 254) for which the block's largest size becomes 127 or
 *    less when rounded (254 where that takes more), so a value is off by at most 1/127 of that size, or by 2^-134 where
 *    that size is under 2^-127.  Scale 255 marks a block that held an infinity or NaN: its codes are 0 and all its
 *    values are read as NaN.  Reading rounds nothing in fp32 and bf16; fp16 has its own range and subnormal steps.
 *  - Limits: n_experts <= 1024; n_rows and every width (2 * inter too) below 2^24; and what the workgroups of one
 *    launch can be.  With a and b a call's two widths (inner, outer, inter) and w the larger one, quotients by n_rows
 *    rounded down and the others up:
 *      (n_rows / 128 + min(n_rows, n_experts)) * (w / 64)  below 2^24 - 16,
 *      or, if a or b is under 8, (n_rows / 64 + min(n_rows, n_experts)) * (w / 32)  below 2^25 - 32;
 *      n_experts * (a / 128) * (b / 128)  below 2^24 - 16.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include <stddef.h>
#include <stdint.h>

#include "moe_tokens.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- activations of the gate
 * Evaluated in fp32, with their slopes: 0 where the exponential leaves fp32 (silu from about g = -87 down), infinity or NaN
 * as the formulas give it at an infinite g (its slope: NaN). */
#define MOE_ACT_SILU  0   /* g / (1 + exp(-g)) */
#define MOE_ACT_GELU  1   /* g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */

/* ---------------------------------------------------------------- rows kept in 8 bits */

/* codes and scales of x [n_rows x cols]. */
int moe_rows_encode(const void *x, int64_t ld_x, int dtype, int n_rows, int cols, int8_t *codes, int64_t ld_codes,
                    uint8_t *scales, int64_t ld_scales, void *stream);

/* Their values, rounded to dtype; a value beyond the type's largest finite one is read as that. */
int moe_rows_decode(const int8_t *codes, int64_t ld_codes, const uint8_t *scales, int64_t ld_scales, int dtype,
                    int n_rows, int cols, void *x, int64_t ld_x, void *stream);

/* ---------------------------------------------------------------- gated feed-forward */

/* hidden[i] = act(g) * u with g = Wg_e x[i], u = Wu_e x[i]; w [n_experts x 2*inter x inner] holds each
 * expert's gate rows, then its up rows; x [n_rows x inner], hidden [n_rows x inter].
 * For the backward pass g and u (before their rounding) can be kept: pre [n_rows x 2*inter] of dtype, g
 * before u; or codes [n_rows x 2*inter] and scales [n_rows x 2*ceil(inter/32)], g's before u's (each half
 * is blocked by itself).  NULL: not kept; pre and codes do not go together. */
int moe_experts_hidden(const void *x, int64_t ld_x, int dtype, int n_rows, int inner, int inter, const int32_t *offsets,
                       int n_experts, const void *w, int activation, void *hidden, int64_t ld_hidden, void *pre,
                       int64_t ld_pre, int8_t *codes, int64_t ld_codes, uint8_t *scales, int64_t ld_scales,
                       void *stream);

/* Back through the down projection and the activation in one step.  d_out [n_rows x outer] is the gradient
 * of moe_experts_product(hidden, w [n_experts x outer x inter]); g and u as kept, in one of the two forms:
 *   d_h = W_e^T d_out[i];  d_pre[i] = [d_h u act'(g), d_h act(g)]  [n_rows x 2*inter];
 *   hidden[i] = act(g) u again (for the gradient of w; NULL: not wanted).
 * d_pre is then the d_out of moe_experts_product_backward with moe_experts_hidden's w. */
int moe_experts_hidden_backward(const void *d_out, int64_t ld_d_out, int dtype, int n_rows, int outer, int inter,
                                const int32_t *offsets, int n_experts, const void *w, int activation, const void *pre,
                                int64_t ld_pre, const int8_t *codes, int64_t ld_codes, const uint8_t *scales,
                                int64_t ld_scales, void *d_pre, int64_t ld_d_pre, void *hidden, int64_t ld_hidden,
                                void *stream);

/* out[i] = W_e x[i]; w [n_experts x outer x inner], x [n_rows x inner], out [n_rows x outer]. */
int moe_experts_product(const void *x, int64_t ld_x, int dtype, int n_rows, int inner, int outer, const int32_t *offsets,
                        int n_experts, const void *w, void *out, int64_t ld_out, void *stream);

/* Its gradients: d_x[i] = W_e^T d_out[i] [n_rows x inner], and d_w[e] = sum over e's rows of d_out[i] x[i]^T,
 * fp32 [n_experts x outer x inner], overwritten (zeros for an expert without rows).  Either may be NULL.
 * For d_w, x is given in dtype or as kept in 8 bits (x NULL; the values rounded to dtype as by
 * moe_rows_decode); without d_w neither is read, without d_x w is not.  workspace:
 * moe_experts_product_workspace bytes (NULL if that is 0, as it is without d_w), 16-byte aligned. */
size_t moe_experts_product_workspace(int n_rows, int inner, int outer, int n_experts);
int moe_experts_product_backward(const void *d_out, int64_t ld_d_out, int dtype, int n_rows, int inner, int outer,
                                 const int32_t *offsets, int n_experts, const void *w, const void *x, int64_t ld_x,
                                 const int8_t *codes, int64_t ld_codes, const uint8_t *scales, int64_t ld_scales,
                                 void *d_x, int64_t ld_d_x, float *d_w, void *workspace, size_t workspace_bytes,
                                 void *stream);

/* ---------------------------------------------------------------- norms around a block */

/* One pass over the rows between two blocks: y [n_rows x hidden] is a block's output, x the residual stream.
 *   r_y = (mean(y^2) + eps)^-1/2,  out = alpha * x + gate * (w_post * (y r_y)),
 *   r_out = (mean(out^2) + eps)^-1/2 (of out before its rounding),  normed = w_pre * (out r_out)
 * w_post, alpha, w_pre [hidden] and gate are fp32.  rows_per_gate rows share a row of gate: gate has
 * ceil(n_rows / rows_per_gate) rows (n_rows or more a gate: one row for all; 1: a row each), contiguous.
 * NULL: w_post no norm of y (out = alpha x + gate y); gate, alpha 1; w_pre and normed (together) no second
 * norm.  y NULL: the first norm alone, normed = w_pre * (x r_out) (then w_post, gate, alpha and out are NULL).
 * Mean squares may leave fp32's range, above or below: r_y and r_out are right wherever they are fp32 numbers
 * themselves and out is finite in fp32.
 * out may be NULL with y too.  stats [n_rows x 2] gets r_y and r_out (0 for a norm that is not there);
 * NULL: not wanted.  out and normed may each be x or y (the same pointer and ld), but not both the same.
 * Limits: hidden <= 16384; n_rows below 2^23 where hidden > 8192. */
int moe_block_norm(const void *x, int64_t ld_x, const void *y, int64_t ld_y, int dtype, int n_rows, int hidden,
                   const float *w_post, const float *gate, int rows_per_gate, const float *alpha, const float *w_pre,
                   float eps, void *out, int64_t ld_out, void *normed, int64_t ld_normed, float *stats, void *stream);

/* Its gradients from those of out and normed (either may be NULL: zeros), with x, y and the parameters as
 * given forward and stats as written:
 *   D = d_out + r_out (t - out r_out^2 mean(t * out)), t = w_pre * d_normed;   d_x = alpha * D,
 *   c = gate * w_post * D;  d_y = r_y (c - y r_y^2 mean(c * y)),  or c without w_post,
 * and, each fp32, overwritten and NULL where not wanted: d_w_post, d_alpha, d_w_pre [hidden], sums over all
 * rows of gate * D * y r_y, D * x and d_normed * out r_out; d_gate, as gate, sums over a gate's rows of
 * w_post * D * y r_y.  d_x or d_y may be NULL too; each may be one of d_out, d_normed, x and y (the same
 * pointer and ld).  stats may be NULL where there is no norm.  workspace: moe_block_norm_workspace bytes, 16-byte aligned (NULL where no
 * parameter's gradient is wanted). */
size_t moe_block_norm_workspace(int n_rows, int hidden, int rows_per_gate);
int moe_block_norm_backward(const void *d_out, int64_t ld_d_out, const void *d_normed, int64_t ld_d_normed,
                            const void *x, int64_t ld_x, const void *y, int64_t ld_y, int dtype, int n_rows, int hidden,
                            const float *w_post, const float *gate, int rows_per_gate, const float *alpha,
                            const float *w_pre, const float *stats, void *d_x, int64_t ld_d_x, void *d_y,
                            int64_t ld_d_y, float *d_w_post, float *d_gate, float *d_alpha, float *d_w_pre,
                            void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_EXPERTS_H */
