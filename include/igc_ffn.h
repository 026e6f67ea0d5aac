/*
 * igc_ffn.h -- feed-forward operators of libigc.so: a matrix product with bias,
 * activation and residual in its epilogue, the gated pair of projections, the
 * gradients of both, and the clipping of a global gradient norm.
 *
 * The conventions of igc.h hold here too (ownership, asynchrony, errors,
 * device, launch).  In addition:
 *  - Element type: `dtype` (IGC_F16 or IGC_BF16) is the type of every matrix of
 *    a call except where an argument says otherwise.  Products are summed in
 *    fp32; a result is rounded once, to nearest even, where it is stored.
 *  - Matrices are row-major with a row stride (ld*) in elements, at least their
 *    number of columns.  X, W, Wg and Wu, which are read by TMA, must be 16-byte
 *    aligned with row strides that are multiples of 8; every other matrix and
 *    every vector may start at any multiple of its element's size and have any
 *    stride.  Anything else is IGC_ERR_MISALIGNED.
 *  - Sizes: any M, N, F, K >= 0 that fit 32 bits.  An empty output is a no-op.
 *    A contraction of length zero is an empty sum: zeros.
 *  - Aliasing: outputs must not overlap inputs or each other (the kernels of a call
 *    may run side by side), with one exception: a residual may be the output itself
 *    (same pointer, type and row stride).  An output pointer that equals another
 *    pointer of the call is refused; other overlaps are not detected.
 *  - Activations (z is fp32, c = sqrt(2 / pi)):
 *      IGC_ACT_NONE       z
 *      IGC_ACT_RELU       max(z, 0)                     derivative 0 at z = 0
 *      IGC_ACT_GELU       z (1 + erf(z / sqrt(2))) / 2
 *      IGC_ACT_GELU_TANH  z (1 + tanh(c (z + 0.044715 z^3))) / 2
 *      IGC_ACT_SILU       z / (1 + exp(-z))
 *    They are computed in fp32 with approximate exponentials and reciprocals (relative errors
 *    of 2^-22 and 2^-23) and are within 1e-5 |z|, their derivatives within 1e-5 (1 + |z|):
 *    no more than the rounding of a 16-bit result hides, but visible in an fp32 Y.
 *  - Workspaces: 256-byte aligned device memory of at least the size that the
 *    *_workspace_size function gives, not shared with a concurrent call; nothing
 *    in one need survive between calls.
 *  - Results do not vary from run to run: every sum has a fixed order.
 *  - Schedule: each product runs on 256-row tiles or, for few rows or small outputs, on
 *    the kernel for those, whichever is estimated to be done sooner (igc_plan_ffn).  A
 *    width set through igc_set_tile_width (igc_debug.h) takes the calling thread's later
 *    products to the 256-row tiles, 128 or 256 columns wide where it is one of these.
 */
#ifndef IGC_FFN_H
#define IGC_FFN_H

#include "igc.h"

#ifdef __cplusplus
extern "C" {
#endif

#define IGC_ACT_NONE 0
#define IGC_ACT_RELU 1
#define IGC_ACT_GELU 2
#define IGC_ACT_GELU_TANH 3
#define IGC_ACT_SILU 4

/*
 * linear_act -- matrix product with bias, activation and residual.
 *
 *   Z[i,j] = sum_{k<K} X[i,k] W[j,k] + bias[j]        0 <= i < M, 0 <= j < N
 *   Y[i,j] = act(Z[i,j]) + R[i,j]
 *
 *  X, W     device, M x K and N x K.
 *  bias     device vector of N elements of type bias_dtype (IGC_F32 or dtype), or NULL.
 *  R        device M x N, or NULL.  May be Y itself when y_dtype is dtype.
 *  Z        device M x N, or NULL: the pre-activation, kept for linear_act_backward.
 *  Y        device M x N of type y_dtype (IGC_F32 or dtype).
 *
 *  Z is rounded to dtype where it is stored; Y is computed from the fp32 Z.
 */
int linear_act(int64_t M, int64_t N, int64_t K, int dtype,
               const void *X, int64_t ldx, const void *W, int64_t ldw,
               const void *bias, int bias_dtype, int act,
               const void *R, int64_t ldr, void *Z, int64_t ldz,
               void *Y, int64_t ldy, int y_dtype, igc_stream_t stream);

/*
 * linear_act_backward -- gradients of linear_act.
 *
 *   dZ[i,j] = dY[i,j] act'(Z[i,j])
 *   dX = dZ W   (M x K)      dW = dZ^T X   (N x K)      dbias[j] = sum_i dZ[i,j]
 *
 *  (The residual's gradient is dY.)  dX, dW and dbias may each be NULL: it is then
 *  not computed.
 *
 *  dY, Z    device, M x N; Z may be NULL when act is IGC_ACT_NONE.
 *  X, W     device, as in linear_act; X is needed for dW, W for dX (else NULL).
 *  dX       device M x K of type dtype.
 *  dW       device N x K of type dw_dtype (IGC_F32 or dtype).
 *  dbias    device vector of N elements of type dbias_dtype (IGC_F32 or dtype).
 *
 *  dZ is rounded to dtype before the two products (it is an operand of the tensor
 *  cores), to the type's precision and range: in fp16 a dZ past 65504 is infinite and one
 *  below 2^-25 is 0, and so is its part in dX and dW.  dbias sums the unrounded values in
 *  fp32.
 */
size_t linear_act_backward_workspace_size(int64_t M, int64_t N, int64_t K);
int linear_act_backward(int64_t M, int64_t N, int64_t K, int dtype,
                        const void *dY, int64_t lddy, const void *Z, int64_t ldz, int act,
                        const void *X, int64_t ldx, const void *W, int64_t ldw,
                        void *dX, int64_t lddx, void *dW, int64_t lddw, int dw_dtype,
                        void *dbias, int dbias_dtype,
                        void *workspace, size_t workspace_bytes, igc_stream_t stream);

/*
 * gated_ffn -- both projections of a gated feed-forward block, the activation and
 * the product, in one kernel.
 *
 *   G[i,j] = sum_{k<K} X[i,k] Wg[j,k] + bg[j]         0 <= i < M, 0 <= j < F
 *   U[i,j] = sum_{k<K} X[i,k] Wu[j,k] + bu[j]
 *   H[i,j] = act(G[i,j]) U[i,j]
 *
 *  X        device, M x K.
 *  Wg, Wu   device, F x K, one row stride ldw (they may be the halves of one 2F x K
 *           matrix).
 *  bg, bu   device vectors of F elements of type bias_dtype (IGC_F32 or dtype); either
 *           may be NULL.
 *  H        device M x F.
 *  G, U     device M x F (row stride ldgu), both or neither: the pre-activations, kept
 *           for gated_ffn_backward.
 */
int gated_ffn(int64_t M, int64_t F, int64_t K, int dtype,
              const void *X, int64_t ldx, const void *Wg, const void *Wu, int64_t ldw,
              const void *bg, const void *bu, int bias_dtype, int act,
              void *G, void *U, int64_t ldgu, void *H, int64_t ldh, igc_stream_t stream);

/*
 * gated_ffn_backward -- gradients of gated_ffn.
 *
 *   dU = dH * act(G)       dG = dH * U * act'(G)               (M x F)
 *   dX = dG Wg + dU Wu     dWg = dG^T X     dWu = dU^T X
 *   dbg[j] = sum_i dG[i,j]     dbu[j] = sum_i dU[i,j]
 *
 *  dX, the pair dWg / dWu, and the pair dbg / dbu may each be NULL: not computed.
 *
 *  dH       device M x F; G, U: device M x F (row stride ldgu).
 *  X, Wg, Wu  device, as in gated_ffn; X is needed for dWg / dWu, Wg and Wu for dX.
 *  dX       device M x K of type dtype.
 *  dWg, dWu device F x K of type dw_dtype (IGC_F32 or dtype), row stride lddw.
 *  dbg, dbu device vectors of F elements of type dbias_dtype (IGC_F32 or dtype).
 *
 *  dG and dU are rounded to dtype before the products, with the range that dZ has in
 *  linear_act_backward: fp16 gradients want a loss scale that keeps dH U act'(G) within
 *  65504.  dbg and dbu sum the unrounded values in fp32.
 */
size_t gated_ffn_backward_workspace_size(int64_t M, int64_t F, int64_t K);
int gated_ffn_backward(int64_t M, int64_t F, int64_t K, int dtype,
                       const void *dH, int64_t lddh, const void *G, const void *U, int64_t ldgu,
                       int act, const void *X, int64_t ldx,
                       const void *Wg, const void *Wu, int64_t ldw,
                       void *dX, int64_t lddx, void *dWg, void *dWu, int64_t lddw, int dw_dtype,
                       void *dbg, void *dbu, int dbias_dtype,
                       void *workspace, size_t workspace_bytes, igc_stream_t stream);

/*
 * grad_norm_clip -- the global 2-norm of many tensors, and their clipping.
 *
 *   norm = sqrt(sum_t sum_i g_t[i]^2)
 *   out_t[i] = g_t[i] * min(1, max_norm / (norm + eps))
 *
 *  count    number of tensors (0: the norm of nothing, 0).
 *  grads    host array of `count` device pointers, each to sizes[t] elements of type
 *           dtypes[t] (IGC_F32, IGC_F16 or IGC_BF16), aligned to its element.
 *  sizes, dtypes  host arrays; a size may be 0 (its pointer is not used).
 *  out      host array of `count` device pointers, or NULL: the norm alone.  out[t] has
 *           the type and size of grads[t] and may be grads[t] itself (in place).
 *  norm     device fp32 scalar.
 *
 *  The tensors must be distinct.  The host arrays may be freed once the call has
 *  returned.  Squares and each thread's sums of them are fp32, what is joined after that
 *  fp64: a value over 2^64 in magnitude makes the norm infinite, one under 2^-75 adds
 *  nothing to it.  A NaN makes the norm and every output NaN; an infinite norm makes
 *  every finite output 0 and the infinite ones NaN, as the formula has it.
 */
size_t grad_norm_clip_workspace_size(int64_t count);
int grad_norm_clip(int64_t count, const void *const *grads, const int64_t *sizes,
                   const int32_t *dtypes, void *const *out, float max_norm, float eps,
                   float *norm, void *workspace, size_t workspace_bytes, igc_stream_t stream);

/*
 * igc_plan_ffn -- the schedule that one of the products above runs with, on a GPU of
 * `sms` SMs, computed on the host by the launches' own decision functions.
 *
 *  op     IGC_PLAN_FFN_LINEAR, _GATED (the forward products), _GRAD_X, _GRAD_W (the
 *         products of the backward passes); M, N (or F), K are the operator's sizes.  A
 *         call's forward product goes by its own operands' alignment too; here their rows
 *         are taken to start on 128-byte lines.  The products of a backward pass go by the
 *         sizes alone, in the call and here.
 *  count  1 for linear_act_backward's products, 2 for gated_ffn_backward's.
 *  out    int32[7]: 0 = 256-row tiles, 1 = the kernel for small outputs; output rows of a
 *         tile or block; their number; its columns of the MMA (of both weights for _GATED);
 *         CTAs that share the contraction of a block; the estimated times of the small and
 *         of the tile kernel in nanoseconds.  The shorter of these is the choice, but for
 *         _GRAD_X, which also goes to the tiles where its own then run beside dW's.
 */
#define IGC_PLAN_FFN_LINEAR 0
#define IGC_PLAN_FFN_GATED 1
#define IGC_PLAN_FFN_GRAD_X 2
#define IGC_PLAN_FFN_GRAD_W 3
int igc_plan_ffn(int op, int64_t M, int64_t N, int64_t K, int count, int sms, int32_t *out);

#ifdef __cplusplus
}
#endif

#endif /* IGC_FFN_H */
