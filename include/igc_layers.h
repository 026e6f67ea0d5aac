/*
 * igc_layers.h -- operators of libigc.so that a training step needs around its
 * feed-forward products: embedding, layer norm and dropout, with their gradients.
 *
 * The conventions of igc.h hold here too (ownership, asynchrony, errors, device,
 * launch).  In addition:
 *  - Element types are IGC_F32, IGC_F16 or IGC_BF16.  Sums, statistics and what is
 *    computed between loads and stores are fp32; a result is rounded once, to nearest
 *    even, where it is stored.
 *  - Matrices are row-major with a row stride (ld*) in elements, at least their number
 *    of columns, and may start at any multiple of their element's size (anything else is
 *    IGC_ERR_MISALIGNED).  Rows that start on 16-byte boundaries (of every matrix of the call)
 *    are read and written 16 bytes at a time.  Others take up to eight times as long (most at
 *    257 to 512 columns), and layer_norm on rows of up to 256 columns, which then has a block to
 *    each row, 9 to 28 times: 65536 rows of 63 bf16 columns 167 us, of 64 columns 6; of 201
 *    columns 196, of 208 22.
 *  - Sizes: up to 2^31 - 512 rows, columns, positions and rows of a table; more, and what would
 *    need more than 2^31 - 1 blocks, is IGC_ERR_UNSUPPORTED.  An empty output is a no-op.
 *  - Aliasing: outputs must not overlap inputs or each other, but for the pairs that an
 *    entry names; those are the same pointer, type and row stride.  An output pointer that
 *    equals another pointer of the call is refused; other overlaps are not detected.
 *  - Results do not vary from run to run: every sum has a fixed order.
 *  - Nothing past a row's last column is written.
 *  - Workspaces: 256-byte aligned device memory of at least the size that the
 *    *_workspace_size function gives, not shared with a concurrent call; nothing in one
 *    need survive between calls.
 *
 * Dropout.  Where an entry takes (p, seed, offset, step), drop(X) below is
 *
 *   drop(X)[i,j] = X[i,j] * 65536 / T  where keep[i,j], else 0,     T = rint((1 - p) 65536)
 *
 *  An element is kept with probability T / 65536: p to 2^-17, and the scale has the exact
 *  expectation.  (A p under 2^-17 drops nothing, one over 1 - 2^-17 everything.)  A dropped
 *  element is 0 whatever X holds there, an infinity or NaN too.  keep comes from a
 *  counter-based generator and is never stored; a backward pass computes it again from the
 *  same four values:
 *
 *   (w0, w1, w2, w3) = Philox4x32-10(counter = (j / 8, i, offset mod 2^32, offset / 2^32),
 *                                    key = (seed mod 2^32, seed / 2^32))
 *   keep[i,j] = (j even ? w mod 65536 : w / 65536) < T,    w = w[(j mod 8) / 2]
 *
 *  (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011.)
 *  It depends on the element's row and column alone, not on the matrix's size, strides or
 *  type.  step, if not NULL, is a device uint64 that is read when the kernels run and added to
 *  offset (mod 2^64): a captured graph draws new elements at each replay if something in it
 *  or between replays changes *step.
 *  Calls (and replays) are independent of one another where (seed, offset + *step mod 2^64)
 *  differ, and draw the same where they are the same.  Layers that share a seed and a counter
 *  and have offsets 0, 1, 2, ... repeat one another's masks a step later: give each layer a
 *  seed of its own, or offsets further apart than there are steps.
 */
#ifndef IGC_LAYERS_H
#define IGC_LAYERS_H

#include "igc.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * dropout_add -- dropout, and the sum with a residual.
 *
 *   Y[i,j] = R[i,j] + drop(X)[i,j]          0 <= i < M, 0 <= j < N
 *
 *  X        device, M x N of type x_dtype.
 *  R        device, M x N of type y_dtype, or NULL (0).
 *  Y        device, M x N of type y_dtype.  May be R; may be X where x_dtype is y_dtype.
 *
 *  Types: x_dtype and y_dtype are the same, or one of them is IGC_F32.  The gradient of X is
 *  the same call on dY without R; that of R is dY.
 */
int dropout_add(int64_t M, int64_t N, const void *X, int64_t ldx, int x_dtype,
                const void *R, int64_t ldr, double p, uint64_t seed, uint64_t offset,
                const uint64_t *step, void *Y, int64_t ldy, int y_dtype, igc_stream_t stream);

/*
 * layer_norm -- dropout, residual sum and layer norm of a block's rows in one pass.
 *
 *   S[i,j] = R[i,j] + drop(X)[i,j]          0 <= i < M, 0 <= j < N
 *   mean[i] = sum_j S[i,j] / N              rstd[i] = 1 / sqrt(sum_j (S[i,j] - mean[i])^2 / N + eps)
 *   Y[i,j] = (S[i,j] - mean[i]) rstd[i] w[j] + b[j]
 *
 *  X        device, M x N of type dtype, or NULL: S = R.
 *  R        device, M x N of type s_dtype, or NULL: S = drop(X).  Not both NULL.
 *  w, b     device vectors of N elements of type w_dtype (IGC_F32 or dtype); either may be
 *           NULL (1 and 0).
 *  S        device, M x N of type s_dtype, or NULL: not stored.  May be R.
 *  Y        device, M x N of type dtype.
 *  mean, rstd  device fp32 vectors of M elements; either may be NULL: not stored.
 *
 *  dtype: any; s_dtype: dtype or IGC_F32 (a residual stream kept in fp32).  N >= 1.  The
 *  statistics and Y are those of the fp32 S, before it is rounded where it is stored.  The mean
 *  is an fp32 sum divided by N: a row of one value whose sums fp32 holds gives Y = b.  The
 *  variance is a sum of squared differences from the mean in fp32: a row whose values differ by
 *  more than 2^63 has an infinite one (rstd 0, Y = b), one whose sum overflows a mean that is not
 *  finite (Y NaN).
 */
int layer_norm(int64_t M, int64_t N, int dtype, const void *X, int64_t ldx,
               const void *R, int64_t ldr, int s_dtype, double p, uint64_t seed,
               uint64_t offset, const uint64_t *step, const void *w, const void *b, int w_dtype,
               float eps, void *S, int64_t lds, void *Y, int64_t ldy, float *mean, float *rstd,
               igc_stream_t stream);

/*
 * layer_norm_backward -- gradients of layer_norm.
 *
 *   h = (S - mean) rstd      g = dY w
 *   dS[i,j] = rstd[i] (g[i,j] - sum_k g[i,k] / N - h[i,j] sum_k g[i,k] h[i,k] / N) + A[i,j]
 *   dX = drop(dS)   (the same elements as in the forward pass; p = 0: dX = dS in dtype)
 *   dw[j] = sum_i dY[i,j] h[i,j]            db[j] = sum_i dY[i,j]
 *
 *  dY       device, M x N of type dtype.
 *  S        device, M x N of type s_dtype (dtype or IGC_F32), as layer_norm stored or read it.
 *  mean, rstd  device fp32 vectors of M elements, as layer_norm stored them.
 *  w        device vector of N elements of type w_dtype (IGC_F32 or dtype), or NULL (1).
 *  A        device, M x N of type s_dtype, or NULL (0): the gradient that reaches S past the
 *           norm, along the residual stream.
 *  dS       device, M x N of type s_dtype, or NULL.  May be A.  It is the gradient of R.
 *  dX       device, M x N of type dtype, or NULL.
 *  dw, db   device vectors of N elements of type dw_dtype (IGC_F32 or dtype); either may be NULL.
 *
 *  dX is rounded from the fp32 dS.  N >= 1; M == 0 writes zeros to dw and db.
 */
size_t layer_norm_backward_workspace_size(int64_t M, int64_t N);
int layer_norm_backward(int64_t M, int64_t N, int dtype, const void *dY, int64_t lddy,
                        const void *S, int64_t lds, int s_dtype, const float *mean,
                        const float *rstd, const void *w, int w_dtype,
                        const void *A, int64_t lda, double p, uint64_t seed, uint64_t offset,
                        const uint64_t *step, void *dS, int64_t ldds, void *dX, int64_t lddx,
                        void *dw, void *db, int dw_dtype, void *workspace,
                        size_t workspace_bytes, igc_stream_t stream);

/*
 * embedding_lookup -- rows of a table, scaled.
 *
 *   Y[i,j] = scale W[token[i], j]           0 <= i < M, 0 <= j < D
 *
 *  tokens   device vector of M integers: int32 (token_bytes 4) or int64 (token_bytes 8).
 *           A token outside [0, V) (padding, or a part of the vocabulary that is elsewhere)
 *           gives a row of zeros.
 *  W        device, V x D of type w_dtype.
 *  Y        device, M x D of type y_dtype: w_dtype or IGC_F32.
 */
int embedding_lookup(int64_t M, int64_t V, int64_t D, const void *tokens, int token_bytes,
                     const void *W, int64_t ldw, int w_dtype, float scale,
                     void *Y, int64_t ldy, int y_dtype, igc_stream_t stream);

/*
 * embedding_backward -- gradient of embedding_lookup's table.
 *
 *   dW[v,j] = scale sum_{i: token[i] = v} dY[i,j]      (+ dW[v,j] when accumulate)
 *
 *  tokens   as in embedding_lookup; a token outside [0, V) adds nothing.
 *  dY       device, M x D of type y_dtype.
 *  dW       device, V x D of type dw_dtype: y_dtype or IGC_F32.  Without accumulate (0) all of
 *           it is written, zeros where no token points; with it (1) only the rows that a
 *           token points to are read and written.
 *
 *  The sum of a row is formed in an order that depends on the tokens and sizes alone.
 */
size_t embedding_backward_workspace_size(int64_t M, int64_t V, int64_t D);
int embedding_backward(int64_t M, int64_t V, int64_t D, const void *tokens, int token_bytes,
                       const void *dY, int64_t lddy, int y_dtype, float scale, int accumulate,
                       void *dW, int64_t lddw, int dw_dtype, void *workspace,
                       size_t workspace_bytes, igc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* IGC_LAYERS_H */
