/*
 * gated_act_linear.h -- the matrix products next to the gated activations, in the
 * same library:
 *
 *   gated projections   act(x Wg') * (x Wu'): the products that feed an activation,
 *                       with the activation as their epilogue, for one block or a
 *                       batch of experts, and the backward pass;
 *   cross entropy       of x W' against targets in a large vocabulary, without the
 *                       logits, and the backward pass.
 *
 * Conventions, where not said otherwise, are those of gated_act_training.h.  What
 * differs:
 *   - element types are GATED_ACT_BF16 and GATED_ACT_F16 (the tensor cores'; others:
 *     GATED_ACT_ERR_DTYPE); products are summed in fp32;
 *   - every buffer is device or managed memory (page-locked host memory:
 *     GATED_ACT_ERR_HOST): the operands are read many times;
 *   - rows whose base and strides are multiples of 16 bytes are read in place; others
 *     are first copied into the workspace, whose size depends on that.
 * The kernels wait inside for copies, products and their own warps.  Such a wait gives up
 * after a second by the clock (for the end of a sum of n terms after n x 0.3 us more); the kernel
 * then sets bit 0 of gated_act_device_status and ends, and the outputs of the call, which returned
 * GATED_ACT_OK long before, and of what was computed from them are undefined.  A kernel that
 * something else holds up for that long (pages of managed memory on their way, another process's
 * time slice) gives up as well.  Two waits have no limit: for tensor memory, until the kernels that
 * hold it on the same SM have ended, and those of a pair of blocks for each other.
 */
#ifndef GATED_ACT_LINEAR_H
#define GATED_ACT_LINEAR_H

#include "gated_act_training.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most experts of one call. */
#define GATED_ACT_MAX_EXPERTS 1024

/* The operands of a call on E experts (E = 1: one block) with T rows each. */
typedef struct gated_act_linear {
    const void *in;         /* [E, T, k]: rows in_stride apart, experts in_batch apart */
    const void *weight;     /* [E, 2d, k], gate rows [0, d), up rows [d, 2d)           */
    int64_t E, T, k, d;
    int64_t in_stride;      /* >= k                                                    */
    int64_t in_batch;       /* >= (T - 1) in_stride + k, where E > 1: rows that all experts
                               share (0) are refused, GATED_ACT_ERR_STRIDE; so is a shared weight */
    int64_t weight_stride;  /* >= k                                                    */
    int64_t weight_batch;   /* >= (2d - 1) weight_stride + k, where E > 1              */
    int dtype;
    const int32_t *n_rows;  /* null, or [E] on the device: live rows of each expert    */
} gated_act_linear;

/* ------------------------------------------------------------------------
 * Gated projections: g = in Wg', u = in Wu' (the weight's two halves), out = act(g) u.
 * Rows past n_rows[e] (taken within [0, T]) have no effect, and what is
 * returned per row is not written there.
 *
 * For the backward pass the forward pass keeps g and u in 16 bits: int16 codes
 * with one scale byte for each block of 32 consecutive elements of a row's gate
 * half, then of its up half, laid out as the 8-bit checkpoint is.  A code q
 * under a scale byte e stands for q * 2^(e - 127); k = e - 127 is the smallest
 * integer >= -126 for which the block's largest magnitude v gives
 * rint(|v| 2^-k) <= 32767.  A block that holds an infinity or a NaN has e = 255 and
 * q = 0 and stands for NaN.  (Why not the element type: bf16's 8 bits would add an error
 * of the gradients' own rounding to each factor that they are computed from.)
 * What one scale for 32 means: a code is off by up to 2^-15 of its block's largest magnitude.  An
 * element r times smaller than that is off by up to r 2^-15 of itself, past r = 128 more than in
 * bf16: one of the 32 that is 1000 times the others leaves these up to 3% off, in the factors of
 * the gradients of their own columns alone.
 * ------------------------------------------------------------------------ */

/* Bytes of workspace that the forward pass needs. */
size_t linear_and_mul_workspace_bytes(const gated_act_linear *a);

/*
 *   out     [E, T, d] contiguous, of type dtype.
 *   codes   null, or int16 [E, T, 2d] contiguous.
 *   scales  uint8 [E, T, 2 ceil(d / 32)], where codes are kept.
 *   workspace  device memory of the size above, 16-byte aligned (null where that is 0);
 *           calls that may overlap on the GPU need one each.
 */
int linear_silu_and_mul(void *out, int16_t *codes, uint8_t *scales, const gated_act_linear *a,
                        void *workspace, size_t workspace_bytes, cudaStream_t stream);
int linear_gelu_and_mul(void *out, int16_t *codes, uint8_t *scales, const gated_act_linear *a,
                        void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace that the backward pass needs: dg and du (4 E T d), where n_rows are given 64 rows of k
 * for each expert, where few long sums of grad_in are split these in fp32, and the copies of operands. */
size_t linear_and_mul_backward_workspace_bytes(const gated_act_linear *a);

/*
 * With dg = grad_out u act'(g) and du = grad_out act(g) at the kept g and u, each rounded once
 * to the element type as an operand of the products (in fp16 under a power of two per expert, so
 * that neither small nor large ones leave the type's range; below 2^-25 of an expert's largest
 * they lose bits):
 *   grad_in      = dg Wg + du Wu            [E, T, k] contiguous, of type dtype;
 *   grad_weight  = (dg' in, du' in)         [E, 2d, k] contiguous, of type dtype: sums over
 *                  the live rows (zeros for an expert without any).
 *   grad_out     [E, T, d] of type dtype, rows grad_stride >= d apart, experts grad_batch apart.
 */
int linear_silu_and_mul_backward(void *grad_in, void *grad_weight, const void *grad_out,
                                 int64_t grad_stride, int64_t grad_batch, const int16_t *codes,
                                 const uint8_t *scales, const gated_act_linear *a, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream);
int linear_gelu_and_mul_backward(void *grad_in, void *grad_weight, const void *grad_out,
                                 int64_t grad_stride, int64_t grad_batch, const int16_t *codes,
                                 const uint8_t *scales, const gated_act_linear *a, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Cross entropy of logits l = in W' over a vocabulary of V:
 *   lse = log sum_v exp(l_v),  loss = lse - l_target.
 * A token whose target lies outside [0, V) takes no part: its loss and lse are
 * 0, its row is not used, and its gradient is 0.
 * ------------------------------------------------------------------------ */

typedef struct gated_act_vocabulary {
    const void *in;         /* [T, k], rows in_stride >= k apart        */
    const void *weight;     /* [V, k], rows weight_stride >= k apart    */
    const void *targets;    /* [T] contiguous int32, or int64           */
    int64_t T, k, V;
    int64_t in_stride, weight_stride;
    int dtype;
    int targets64;          /* 0: int32 targets, else int64             */
} gated_act_vocabulary;

/* Bytes of workspace that the forward pass needs: T V / 16 (up to 128 tokens T V / 4), the live rows (2 T k), and
 * the copy of a weight that is not read in place. */
size_t linear_cross_entropy_workspace_bytes(const gated_act_vocabulary *a);

/*   loss, lse  [T] fp32. */
int linear_cross_entropy(float *loss, float *lse, const gated_act_vocabulary *a, void *workspace,
                         size_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace that the backward pass needs: grad_in's sums in fp32 (4 T k; few rows, up to 32 times that), the
 * rows with and without their slopes (4 T k), a piece of the vocabulary's y, and the copy of a weight that is
 * not read in place.  A piece's y takes about 256 MB up to 16384 tokens; past that a piece keeps 8192
 * columns (a quarter more at most), and y grows with the tokens as the other parts do, 16 KB a token: 1 GB at
 * 65536 of them. */
size_t linear_cross_entropy_backward_workspace_bytes(const gated_act_vocabulary *a);

/*
 * With p = exp(l - lse), c = 1 - p_target (from the loss) and a token's slope f = grad_loss c,
 *   grad_in      = f y W                     [T, k] contiguous, of type dtype;
 *   grad_weight  = sum_t y_t' (f_t in_t)     [V, k] contiguous, of type dtype,
 * where y = (p - [v = target]) / c and f in (by a power of two from the batch's largest: of |f| in bf16; of |f in| in fp16,
 * whose upper end it is put to; the sums are multiplied with it at their end) are each rounded once to the element type
 * as operands of the products; with T <= 256 what the second rounding takes off is an operand too.  In fp16 a product
 * f in below 2^-29 of the batch's largest loses bits (the second operand, with T <= 256, below 2^-18 of it), and so does
 * a y below 2^-28.
 *   grad_loss    [T] fp32, read on the device; not used at tokens that take no part.
 *   loss, lse    what linear_cross_entropy wrote.
 * The logits are computed again, in pieces of the vocabulary.
 */
int linear_cross_entropy_backward(void *grad_in, void *grad_weight, const float *grad_loss,
                                  const float *loss, const float *lse, const gated_act_vocabulary *a,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GATED_ACT_LINEAR_H */
