/*
 * gated_act_training.h -- what training a gated MLP block needs next to the
 * forward activations of gated_act.h, in the same library:
 *
 *   8-bit checkpoints   silu_and_mul, gelu_and_mul and gelu_and_mul_sparse that
 *                       keep their input in 8 bits for the backward pass, and
 *                       the backward passes that read it back;
 *   layer norm          forward, and backward with the reduction of the
 *                       parameters' gradients over the rows;
 *   balance loss        a router's auxiliary loss, its per-expert counts and
 *                       the gradient of its logits.
 *
 * Conventions, where not said otherwise, are those of gated_act.h: memory is
 * the caller's (device, managed or page-locked host memory the current device
 * can reach), every call launches only on `stream`, allocates nothing, never
 * synchronizes and can be captured in a CUDA graph; every layout is accepted
 * (16-byte aligned rows take vector paths); the status codes are the same.
 * Element types are a gated_act_dtype.  Arithmetic is fp32; each output
 * element is rounded once, to nearest even.  Results do not depend on the
 * order in which blocks run: there are no floating-point atomics.
 * Strides count elements.
 */
#ifndef GATED_ACT_TRAINING_H
#define GATED_ACT_TRAINING_H

#include "gated_act.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * 8-bit checkpoints.
 *
 * The checkpoint of rows [M, 2d] (gate = columns [0, d), up = [d, 2d)) is
 *   codes   int8  [M, 2d], laid out as the rows;
 *   scales  uint8 [M, 2B], B = ceil(d / 32): one byte for each block of 32
 *           consecutive elements of the gate half, then of the up half (the
 *           last block of a half holds what is left).
 * A code q under a scale byte e stands for q * 2^(e - 127).  In each block
 * k = e - 127 is the smallest integer in [-127, 121] for which the largest
 * magnitude v gives rint(|v| 2^-k) <= 127, and q = rint(v 2^-k), ties to even
 * (a magnitude of 127.5 * 2^121 or more, at the very end of the types' range,
 * has k = 121 and q = +-127).  The scale is a power of two, so codes and
 * values are exact functions of the input, and every value is exact in bf16.
 * A block that holds an infinity or a NaN has e = 255 and q = 0 and stands for
 * NaN.
 * (Blocks of 32 with a power-of-two scale and 8-bit integers are those of the
 * OCP Microscaling Formats specification v1.0, MXINT8.)
 *
 * gelu_and_mul_sparse keeps gate - cutoff in the gate half instead of the
 * gate, and there the code is at least 1 wherever gate > cutoff: the mask
 * that the backward pass reads is exactly the forward pass's.
 * ------------------------------------------------------------------------ */

/* Scale bytes of one row, 2 * ceil(d / 32). */
int64_t gated_act_checkpoint_scales(int64_t d);

/*
 * silu_and_mul / gelu_and_mul that also write the checkpoint of their input.
 *   out     [M, d] contiguous.    codes, scales  as above, contiguous.
 *   in      [M, row_stride], row_stride >= 2d.
 *   dtype   element type of in and out.
 *   n_rows  null, or a device pointer to the live row count (as in
 *           silu_and_mul_bounded): rows past it are neither read nor written.
 */
int silu_and_mul_checkpoint(void *out, int8_t *codes, uint8_t *scales, const void *in, int64_t M,
                            int64_t d, int64_t row_stride, int dtype, const int32_t *n_rows,
                            cudaStream_t stream);
int gelu_and_mul_checkpoint(void *out, int8_t *codes, uint8_t *scales, const void *in, int64_t M,
                            int64_t d, int64_t row_stride, int dtype, const int32_t *n_rows,
                            cudaStream_t stream);

/*
 * Their backward passes: the gradient at the checkpoint's values (g, u),
 *   grad_gate = grad_out * u * act'(g),   grad_up = grad_out * act(g).
 *   grad_in   [M, 2d] contiguous.
 *   out       null, or [M, d] contiguous: act(g) * u is written there (the
 *             weight gradient of the product that follows the activation
 *             needs it; it need not be kept from the forward pass).
 *   grad_out  [M, grad_stride], grad_stride >= d.
 *   dtype     element type of grad_in, out and grad_out.
 */
int silu_and_mul_backward(void *grad_in, void *out, const void *grad_out, const int8_t *codes,
                          const uint8_t *scales, int64_t M, int64_t d, int64_t grad_stride,
                          int dtype, const int32_t *n_rows, cudaStream_t stream);
int gelu_and_mul_backward(void *grad_in, void *out, const void *grad_out, const int8_t *codes,
                          const uint8_t *scales, int64_t M, int64_t d, int64_t grad_stride,
                          int dtype, const int32_t *n_rows, cudaStream_t stream);

/*
 * gelu_and_mul_sparse that also writes its checkpoint.
 *   std  [T] fp32: each row's population standard deviation; exactly 0 for a row
 *        of one value, of which nothing passes the mask.
 *   Other arguments as gelu_and_mul_sparse_typed and above.
 */
int gelu_and_mul_sparse_checkpoint(void *out, int8_t *codes, uint8_t *scales, float *std,
                                   const void *in, int64_t T, int64_t d, int64_t row_stride,
                                   double z, int dtype, cudaStream_t stream);

/*
 * Its backward pass.  With delta = gate - cutoff and u from the checkpoint,
 * s = max(delta, 0) and h = [delta > 0] grad_out u gelu_tanh'(s):
 *   grad_gate_i = h_i - (sum_j h_j / d) (1 + z (g_i - mean) / std),
 *   g_i - mean  = delta_i + z std,
 *   grad_up     = grad_out * gelu_tanh(s).
 * The cutoff's own dependence on the row is the second term.  A row with
 * std = 0 has no derivative of std; the z term is then left out (every h of a
 * row of one value is 0).  A position with delta <= 0 adds nothing to the sum,
 * whatever grad_out and u hold there.
 */
int gelu_and_mul_sparse_backward(void *grad_in, void *out, const void *grad_out,
                                 const int8_t *codes, const uint8_t *scales, const float *std,
                                 int64_t T, int64_t d, int64_t grad_stride, double z, int dtype,
                                 cudaStream_t stream);

/*
 * The values that a checkpoint stands for: values [M, 2d] contiguous, of type
 * GATED_ACT_BF16 or GATED_ACT_F32 (both exact).
 */
int gated_act_checkpoint_values(void *values, const int8_t *codes, const uint8_t *scales,
                                int64_t M, int64_t d, int dtype, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Layer norm over rows of width d:
 *   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
 *   out = (x - mean) rstd * weight + bias.
 * A row of one value has it as its mean and, with eps > 0, the bias as its output.
 * Squares of deviations are fp32 numbers: past 1.8e19 they are infinite (rstd =
 * 0), and below 1e-19 they lose bits.
 * ------------------------------------------------------------------------ */

/*
 *   out     [T, d] contiguous, of type dtype.   mean, rstd  [T] fp32.
 *   in      [T, row_stride], row_stride >= d, of type dtype.
 *   weight  [d] of type param_dtype: dtype or GATED_ACT_F32.
 *   bias    [d] of type param_dtype, or null for none.
 *   eps     >= 0.
 */
int layer_norm(void *out, float *mean, float *rstd, const void *in, const void *weight,
               const void *bias, int64_t T, int64_t d, int64_t row_stride, double eps, int dtype,
               int param_dtype, cudaStream_t stream);

/* Bytes of workspace that layer_norm_backward needs for T rows of width d on
 * the current device. */
size_t layer_norm_backward_workspace_bytes(int64_t T, int64_t d);

/*
 * With hat = (in - mean) rstd and g = grad_out * weight:
 *   grad_in     = rstd (g - sum g / d - hat sum (g hat) / d)   [T, d], dtype;
 *   grad_weight = sum over rows of grad_out * hat              [d] fp32;
 *   grad_bias   = sum over rows of grad_out                    [d] fp32, or
 *                 null where it is not wanted.
 *   workspace   device memory of the size above, 16-byte aligned; what it
 *               holds before does not matter, and calls that may overlap on
 *               the GPU need one each.
 * T = 0 writes zero parameter gradients.
 */
int layer_norm_backward(void *grad_in, float *grad_weight, float *grad_bias, const void *grad_out,
                        const void *in, const void *weight, const float *mean, const float *rstd,
                        int64_t T, int64_t d, int64_t row_stride, int64_t grad_stride, int dtype,
                        int param_dtype, void *workspace, size_t workspace_bytes,
                        cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Balance loss of a router over E experts (Fedus, Zoph and Shazeer, "Switch
 * Transformers", 2021, section 2.2, for k choices per token): with p the
 * softmax of a token's logits, N live tokens, c_e the number of times that
 * expert e was chosen by them and P_e the mean of p_e over them,
 *   loss = coef * E * sum_e c_e / (N k) * P_e,
 *   d loss / d logit_j of a token = coef E / (N^2 k) p_j (c_j - sum_e p_e c_e).
 * The counts are constants to the gradient.  N = 0 gives loss 0 and gradients
 * 0.  A token whose logits are all -infinity has p = 0.
 * ------------------------------------------------------------------------ */

/* Bytes of workspace that moe_balance_loss needs on the current device. */
size_t moe_balance_loss_workspace_bytes(int64_t T, int64_t E);

/*
 *   loss    [1] fp32.      counts  [E] int32.    tokens  [1] int32: N.
 *   mean_p  [E] fp32: P.
 *   logits  [T, logits_stride], logits_stride >= E, of type dtype; E <= 1024.
 *   ids     [T, k] contiguous expert ids, int32 (ids64 = 0) or int64 (else).
 *           An id outside [0, E) is a choice that was dropped: it is not
 *           counted.
 *   live    null, or [T] bytes: a token whose byte is 0 takes no part, and
 *           its logits and ids are not used.
 *   workspace  as for layer_norm_backward.
 * T * k < 2^31.
 */
int moe_balance_loss(float *loss, int32_t *counts, int32_t *tokens, float *mean_p,
                     const void *logits, const void *ids, const uint8_t *live, int64_t T,
                     int64_t E, int64_t k, int64_t logits_stride, int dtype, int ids64,
                     double coef, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 *   grad_logits [T, E] contiguous, of type dtype: grad_loss times the gradient
 *               above; 0 in the rows of tokens that are not live.
 *   grad_loss   [1] fp32, read on the device; where it is not finite, the rows
 *               that are not live are 0 all the same.
 *   counts, tokens  what moe_balance_loss wrote.
 */
int moe_balance_loss_backward(void *grad_logits, const float *grad_loss, const void *logits,
                              const int32_t *counts, const int32_t *tokens, const uint8_t *live,
                              int64_t T, int64_t E, int64_t k, int64_t logits_stride, int dtype,
                              double coef, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GATED_ACT_TRAINING_H */
