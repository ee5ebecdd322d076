/*
 * bsq_block.h -- what a transformer block computes around the quantized
 * linears of bsq.h: rotary positions with several axes, the gated residual
 * with the norms before and after it (and its gradient), and linears with
 * bias, activation, gate and residual in their epilogue.
 *
 * The conventions of bsq.h and bsq_serve.h hold: device pointers owned by the
 * caller, work enqueued on `stream`, nothing allocated, freed or synchronized,
 * arguments validated on the host before any HIP call, no exception across the
 * ABI, the same inputs give the same bits (no atomics). Structs are host memory,
 * read during the call only.
 *
 * Row groups. A call's rows may fall into groups (the images of a batch) that
 * have vectors of their own: row g of a [groups][dim] tensor belongs to group g.
 *   group_starts  int32 [groups + 1] device, 4-byte aligned: group g has rows
 *     group_starts[g] to group_starts[g + 1] - 1 (none, if they are equal). It
 *     starts at 0 and does not decrease. Rows from group_starts[groups] on belong to
 *     no group: not written, and without effect, as the vectors of a group without rows.
 *     Where it decreases or leaves [0, rows], which vectors a row takes, and what is
 *     written for it, is not defined; nothing outside the call's tensors is read or written.
 *   group_starts NULL: each group has rows / groups consecutive rows
 *     (rows % groups == 0, BSQ_ERR_SHAPE otherwise).
 * 1 <= groups <= 2^24 (1 where a call has no such vectors).
 */
#ifndef BSQ_BLOCK_H
#define BSQ_BLOCK_H

#include "bsq_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rotary positions with several axes (rows and columns of an image; time, rows
 * and columns of a video): bsq_rope, where pair i turns by the position of its
 * own axis, angle a_i = positions[t][axis(i)] * inv_freq[i]. There are
 * r = 2 (sections[0] + .. + sections[axes - 1]) rotated elements, and
 *   BSQ_AXES_BLOCKS  the first sections[0] pairs have axis 0, the next
 *                    sections[1] axis 1, and so on;
 *   BSQ_AXES_CYCLED  pair i has axis i % axes if i / axes < sections[i % axes],
 *                    and axis 0 otherwise: the axes in turn, and axis 0 where
 *                    another one has had its pairs. Axis c > 0 has to find its
 *                    sections[c] pairs: axes (sections[c] - 1) + c < r / 2.
 * The frequencies are the caller's: of bsq_rope_inv_freq(2 sections[c], ..) for each
 * axis, one after the other, or of bsq_rope_inv_freq(r, ..) for all pairs.
 * Everything else (dtype, layout, backward, exactness, strides, in place, limits of T, H
 * and D, errors) is as in bsq_rope.
 *   sections  int64 [axes], HOST memory, 1 <= axes <= 4, each >= 0
 *   positions int64: that of token t on axis c at
 *     positions[t * pos_stride_t + c * pos_stride_a], strides in elements >= 0
 * BSQ_ERR_SHAPE: axes or sections out of range, r < 2 or r > D. BSQ_ERR_ARG: an
 * unknown order. BSQ_ERR_NULL: no sections.
 */
typedef enum { BSQ_AXES_BLOCKS = 1, BSQ_AXES_CYCLED = 2 } bsq_axes_order;
bsq_status bsq_rope_axes(bsq_dtype dtype, const void* x, int64_t x_stride_t, int64_t x_stride_h,
                         const int64_t* positions, int64_t pos_stride_t, int64_t pos_stride_a, const int64_t* sections,
                         int64_t axes, bsq_axes_order order, const float* inv_freq, bsq_rope_layout layout,
                         float attn_factor, uint32_t flags, void* y, int64_t y_stride_t, int64_t y_stride_h, int64_t T,
                         int64_t H, int64_t D, hipStream_t stream);

/*
 * What happens between two blocks of a transformer, in one pass over its rows:
 * the branch h that a block computed is normed (if `post` asks for it) and
 * added to the stream x, gated, and the sum is normed, scaled and shifted for the next block:
 *   h'    = post_weight * N_post(h),  or h with BSQ_NORM_NONE
 *   x_out = x + gate[g] * h',         or x without a branch
 *   y     = (N_norm(x_out) * weight + bias) * (1 + scale[g]) + shift[g]
 * for a row of group g, element by element, where a row's norm is
 *   BSQ_NORM_RMS    N(v) = v / sqrt(mean v^2 + eps)
 *   BSQ_NORM_LAYER  N(v) = (v - mean v) / sqrt(mean (v - mean v)^2 + eps)
 * Vectors that are NULL are left out (weight, gate, post_weight count as 1, scale, shift, bias as 0).
 * norm == BSQ_NORM_NONE: there is no y (no weight, bias, scale, shift), x_out alone.
 * Rows are held in fp32 from their load to their store: y is formed from x_out as it is before its
 * rounding, statistics are sums of squares in fp32: they overflow where |x| reaches 2^57, and with eps 0 they lose what is
 * below 2^-56 (a row whose largest |x|, or |x - mean|, is less; one of zeros is 0 / 0, NaN).
 *   dtype     of all tensors (any of the three)
 *   weight, bias, post_weight [dim]; scale, shift, gate [groups] rows of dim,
 *     their strides apart (>= dim where groups > 1; multiples of 8)
 * 8 <= dim <= 16384, dim % 8 == 0, 0 <= rows <= 2^30; strides of rows in elements,
 * multiples of 8, >= dim and < 2^40 (x and branch: also 0, one row for all; rows == 1: any multiple of 8);
 * pointers 16-byte aligned. bsq_block_norm has a workgroup for each row or four of them: rows times the waves of a row,
 * ceil(dim / 512) up to dim 2048 and ceil(dim / 1024) above, stay below 2^25 - 4 there (BSQ_ERR_SHAPE otherwise; longer
 * tensors are several calls, since rows are independent). bsq_block_norm_backward takes all 2^30.
 * eps, post_eps >= 0 and finite. post_weight needs a post norm. (BSQ_ERR_ARG for an unknown dtype, norm or format,
 * eps out of range, vectors of a norm that is not there.)
 */
typedef enum { BSQ_NORM_NONE = 0, BSQ_NORM_LAYER = 1, BSQ_NORM_RMS = 2 } bsq_norm;
typedef struct {
  bsq_dtype dtype;
  bsq_norm norm, post;
  float eps, post_eps;
  int64_t rows, dim, groups;
  const int32_t* group_starts;
  const void *weight, *bias, *post_weight;
  const void *scale, *shift, *gate;
  int64_t scale_stride, shift_stride, gate_stride;
} bsq_block;

/*
 * Forward. out_format 0: y of dtype. BSQ_FMT_FP8R, BSQ_FMT_NVFP4 (dim % 32 == 0): y is written as the activation of
 * the next quantized linear instead, by the arithmetic of bsq_quantize_act_fp8r / bsq_quantize_act_nvfp4 on the
 * fp32 y (which is not rounded to 16 bits first). A row of NaN gives NaN scales.
 *   x [rows], branch [rows] (or NULL; then gate and x_out are NULL too and post is BSQ_NORM_NONE)
 *   x_out [rows] or NULL (not written); may be x with the same stride
 *   y [rows] of dtype | fp8r uint8 [rows][dim] dense | nvfp4 uint8 [rows][dim/2] dense; y_stride is read for
 *     out_format 0 only
 *   y_scale  fp8r fp32 [rows] | nvfp4 uint8 [rows][dim/16] | otherwise NULL
 *   y_global nvfp4 fp32 [1], the next linear's input_scale | otherwise NULL
 * Outputs must not overlap one another or inputs otherwise.
 */
bsq_status bsq_block_norm(const bsq_block* block, const void* x, int64_t x_stride, const void* branch,
                          int64_t branch_stride, void* x_out, int64_t x_out_stride, int out_format,
                          const float* y_global, void* y, int64_t y_stride, void* y_scale, hipStream_t stream);

/*
 * Gradient, from the saved x_out (x where there is no branch) and branch, for the gradients dy of y and dx_out of
 * x_out (NULL counts as 0; what the stream passes on to later blocks). With c = the gradient of x_out in all:
 *   n = N_norm(x_out), dn = dy * (1 + scale[g]) * weight,
 *   c = dx_out + (dn - [mean dn] - n mean(dn n)) / sqrt(..)       ([..]: for BSQ_NORM_LAYER)
 *   dx = c
 *   dh' = gate[g] * c, dbranch = dh' or, through the post norm, the same form with dh' * post_weight
 *   dscale[g] = sum dy (n weight + bias), dshift[g] = sum dy, dgate[g] = sum c h'   over the group's rows
 *   dweight = sum dy (1 + scale[g]) n, dbias = sum dy (1 + scale[g]), dpost_weight = sum dh' N_post(h)  over all rows
 * Each gradient whose pointer is not NULL is written, whole (zeros for groups without rows); the vectors' are fp32,
 * dense ([groups][dim], [dim]), summed in a fixed order. dx and dbranch are of dtype, their rows without a group are left as they were.
 *   dy, dx_out, x_out, branch [rows] with strides as x's of the forward; dy is NULL exactly when norm is BSQ_NORM_NONE
 *   (dx_out is then needed); branch may be NULL unless dgate or dpost_weight is asked for, or dbranch with a post norm
 *   dx [rows], may be dx_out or dy with the same stride; dbranch [rows], may be branch with the same stride
 *   dscale, dshift, dgate, dweight, dbias, dpost_weight: where the block has the vector (BSQ_ERR_ARG otherwise)
 * workspace: bsq_block_norm_workspace_bytes(rows, dim, groups) bytes (0 bytes where only dx and dbranch are asked for),
 *   256-byte aligned, not shared by calls that may overlap; nothing in it needs clearing or survives the call.
 */
size_t bsq_block_norm_workspace_bytes(int64_t rows, int64_t dim, int64_t groups);
bsq_status bsq_block_norm_backward(const bsq_block* block, const void* dy, int64_t dy_stride, const void* dx_out,
                                   int64_t dx_out_stride, const void* x_out, int64_t x_out_stride, const void* branch,
                                   int64_t branch_stride, void* dx, int64_t dx_stride, void* dbranch,
                                   int64_t dbranch_stride, float* dscale, float* dshift, float* dgate, float* dweight,
                                   float* dbias, float* dpost_weight, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/*
 * The pre-quantized linears of bsq.h (bsq_gemm_fp8r_q, bsq_gemm_nvfp4_q: operands, routes and errors as there)
 * with an epilogue:
 *   y[m][n] = bf16( residual[m][n] + gate[g(m)][n] * act( (x w^T)[m][n] + bias[n] ) )
 * where (x w^T) is their result before its rounding and every step after it is fp32, rounded once at the end. Products are
 * summed in fp32; for fp8r the e4m3 matrix instruction takes them eight at a time and first cuts each one off below 2^-13
 * of the largest of the eight (bsq.h; nvfp4's f16 instruction cuts nothing off).
 *   BSQ_ACT_NONE       v
 *   BSQ_ACT_SILU       v / (1 + exp(-v))
 *   BSQ_ACT_GELU_TANH  v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3)))
 *   BSQ_ACT_GELU       v Phi(v), Phi the normal distribution: to 2^-15 of itself for v >= -5, below that to 4e-7
 * (silu and gelu_tanh to 2^-15 of themselves, by the hardware's exp2 and reciprocal; what would be below 2^-119 may be 0.)
 *   bias     [N] bf16 or NULL (0)
 *   gate     [groups] rows of N bf16, gate_stride apart (>= N where groups > 1), 2-byte aligned, or NULL (1)
 *   residual [M][residual_stride] bf16 (residual_stride >= N), 16-byte aligned, or NULL (0); y may be residual with
 *            the same stride
 * groups, group_starts: the rows' groups (above); read with a gate only (groups is then 1 or more).
 * BSQ_ERR_ARG for an unknown activation; BSQ_ERR_SHAPE for strides and groups; bias 2-byte aligned. BSQ_ERR_NULL
 * without an epilogue.
 */
typedef enum { BSQ_ACT_NONE = 0, BSQ_ACT_SILU = 1, BSQ_ACT_GELU_TANH = 2, BSQ_ACT_GELU = 3 } bsq_act;
typedef struct {
  bsq_act act;
  const uint16_t* bias;
  const uint16_t* gate;
  int64_t gate_stride;
  const uint16_t* residual;
  int64_t residual_stride;
  int64_t groups;
  const int32_t* group_starts;
} bsq_epilogue;
bsq_status bsq_gemm_fp8r_q_epilogue(const uint8_t* xq, const float* x_scale, const uint8_t* w, const float* w_scale,
                                    const bsq_epilogue* epilogue, uint16_t* y, int64_t ldy, int64_t M, int64_t N,
                                    int64_t K, hipStream_t stream);
bsq_status bsq_gemm_nvfp4_q_epilogue(const uint8_t* xq, const uint8_t* x_bscale, const float* input_scale,
                                     const uint8_t* w, const uint8_t* w_bscale, const float* w_scale2,
                                     const bsq_epilogue* epilogue, uint16_t* y, int64_t ldy, int64_t M, int64_t N,
                                     int64_t K, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BSQ_BLOCK_H */
