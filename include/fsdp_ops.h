/*
 * fsdp_ops.h -- C ABI of the training-step operators around a sharded unit
 * (GB300, sm_103a): what produces the gradients that the shard engine
 * reduces, and a matrix-aware update that uses them.
 *
 *   fsdp_layer_norm, fsdp_layer_norm_backward
 *   fsdp_linear_cross_entropy      loss of a linear head, with its gradients
 *   fsdp_newton_schulz             orthogonalises matrices
 *   fsdp_muon                      rank reduction + momentum + Newton-Schulz
 *                                  + update of master and parameter
 *
 * Conventions (beyond those of fsdp_shard.h, whose status codes, dtypes and
 * fsdp_last_error these calls share):
 *  - Matrices are row-major with a row stride in elements (ld >= columns);
 *    the elements of a row are adjacent.
 *  - Rows, columns and vocabulary are at most 2^31 - 65536 each, and matrices
 *    have at most 2^40 elements (FSDP_ERANGE above).
 *  - Numbers are doubles that the kernels take as fp32: one that fp32 cannot
 *    hold (infinite in it, or an eps that is 0 in it) is FSDP_EINVAL.
 *  - Pointers need the alignment of their element only; 16-byte aligned
 *    bases and strides take the vector and tensor-copy paths directly, others
 *    go through scalar accesses or one packing copy.
 *  - Every call checks its arguments on the host before it launches anything:
 *    sizes, strides, NULL, alignment, that no output's range overlaps any
 *    other buffer's, and that every buffer is device memory of one device.
 *    A range runs from the first to the last element of a matrix, the gaps
 *    between its rows included.
 *  - Calls are asynchronous on `stream` and never synchronise. They allocate
 *    nothing: scratch memory is the caller's `workspace`, of at least the
 *    bytes that the operator's _workspace query returns, 256-byte aligned.
 *    It may be reused as soon as the call's work on the stream is done, and
 *    holds nothing that a later call needs.
 *  - Sums, statistics and products accumulate in fp32 or wider. Their order is
 *    fixed by the sizes, by whether rows start on 16 bytes, by the device's
 *    number of multiprocessors and, for the loss, by the number of rows that
 *    count: the same call gives the same bits every time. The same values in
 *    buffers of another alignment may be summed in another order.
 *  - No kernel traps. The matrix kernels wait on their own copies and on the
 *    tensor core; a wait that lasts ~2 s is given up, the block counts itself
 *    (fsdp_ops_wait_timeouts) and its outputs are invalid.
 */
#ifndef FSDP_OPS_H
#define FSDP_OPS_H

#include "fsdp_shard.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Layer norm over the columns of x [rows, cols]:
 *   mean = sum_j x_j / cols;  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / cols + eps)
 *   y_j = (x_j - mean) * rstd * gamma_j + beta_j
 * x, y: dtype; gamma, beta [cols]: param_dtype; beta may be NULL (no offset).
 * mean, rstd [rows] fp32: kept for the backward pass; both may be NULL.
 * rows = 0 does nothing; cols >= 1; eps > 0. Errors: FSDP_EINVAL,
 * FSDP_EALIGN, FSDP_EUNSUPPORTED (dtype), FSDP_ERANGE, FSDP_ECUDA. */
fsdp_status fsdp_layer_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                            fsdp_dtype dtype, const void *gamma, const void *beta,
                            fsdp_dtype param_dtype, double eps, void *y, int64_t ldy, float *mean,
                            float *rstd, void *stream);

/* Its gradients, with xhat = (x - mean) * rstd and g = dy * gamma:
 *   dx = rstd * (g - sum_j g_j / cols - xhat * sum_j (g_j xhat_j) / cols)
 *   dgamma_j = sum_rows dy_j * xhat_j;  dbeta_j = sum_rows dy_j
 * dy, x, dx: dtype; gamma, dgamma, dbeta: param_dtype (each sum rounded once).
 * dbeta may be NULL. rows = 0 writes zeros to dgamma and dbeta. */
fsdp_status fsdp_layer_norm_backward(int64_t rows, int64_t cols, const void *dy, int64_t lddy,
                                     const void *x, int64_t ldx, fsdp_dtype dtype,
                                     const void *gamma, fsdp_dtype param_dtype, const float *mean,
                                     const float *rstd, void *dx, int64_t lddx, void *dgamma,
                                     void *dbeta, void *workspace, int64_t workspace_bytes,
                                     void *stream);
fsdp_status fsdp_layer_norm_backward_workspace(int64_t rows, int64_t cols, int64_t *bytes);

typedef enum { FSDP_MEAN = 0, FSDP_SUM = 1 } fsdp_reduction;

/* Softmax cross entropy of a linear head, without the rows x vocab logits:
 *   z = hidden weight^T;  row_loss_n = log sum_v exp(z_nv) - z_n,target_n
 *   loss = sum_n row_loss_n / count (FSDP_MEAN) or the sum (FSDP_SUM)
 * and, where dhidden is not NULL, with G = softmax(z) - onehot(target) and
 * s = grad_scale / count or grad_scale:
 *   dhidden = s G weight;  dweight = s G^T hidden
 * hidden [rows, cols], weight [vocab, cols], dhidden, dweight: bf16.
 * targets [rows] int64. A row whose target is ignore_index counts for
 * nothing, whatever its hidden holds: row_loss 0, dhidden 0, no part in
 * dweight; count is the number of the other rows. With count = 0, loss and
 * gradients are 0. A target outside [0, vocab) that is not ignore_index makes
 * row_loss and loss NaN; that row has no gradients but is counted.
 * dhidden and dweight are both given or both NULL (loss alone). dweight may
 * be a view of a unit's gradient buffer. loss [1], row_loss [rows]: fp32.
 * G is rounded to bf16 for its two products, which is where the gradients'
 * error comes from (2^-8 per element of G at most, beside their own rounding).
 * The rows are taken in pieces of piece_rows, rounded up to 64 (0: as many as
 * keep a piece's 16-bit exponentials, or without gradients its statistics of 8
 * bytes per 128 words, at 2 GiB); within a piece the softmax is formed from
 * tiles of the vocabulary, each with its own maximum and sum. */
fsdp_status fsdp_linear_cross_entropy(int64_t rows, int64_t cols, int64_t vocab,
                                      const void *hidden, int64_t ldh, const void *weight,
                                      int64_t ldw, const int64_t *targets, int64_t ignore_index,
                                      fsdp_reduction reduction, double grad_scale, float *loss,
                                      float *row_loss, void *dhidden, int64_t lddh, void *dweight,
                                      int64_t lddw, int64_t piece_rows, void *workspace,
                                      int64_t workspace_bytes, void *stream);
/* aligned_weight: weight starts on 16 bytes and ldw is a multiple of 8; else
 * the workspace holds a copy of it that does. */
fsdp_status fsdp_linear_cross_entropy_workspace(int64_t rows, int64_t cols, int64_t vocab,
                                                int with_gradients, int aligned_weight,
                                                int64_t piece_rows, int64_t *bytes);

/* Newton-Schulz iteration on `batch` matrices g [m, n] (batch stride in
 * elements), each on its own:
 *   x = g / (||g||_F + eps);  `steps` times:
 *     S = x x^T (m <= n) or x^T x;  P = b S + c S^2;  x = a x + P x (or x P)
 *   out = x
 * g: bf16 or fp32; out [batch, m, n]: bf16. steps in [0, 64].
 * The sizes and the device choose one of three forms. For a shorter side of at
 * most 32 there is one of fp32 throughout. In the others the products' operands
 * x, S and P are fp16, their sums fp32, and x is carried from step to step in
 * fp32 (few small matrices) or as two fp16 numbers, which is 22 bits, or 2^-36
 * where that is more (many or large ones). Coefficients with which an element
 * of x, S or P passes 65504 give infinities there.
 * ||g||_F has to be below 1.8e19, and below 1e-19 it counts as 0 beside eps (its
 * square is an fp32 number). */
fsdp_status fsdp_newton_schulz(int64_t batch, int64_t m, int64_t n, const void *g, int64_t ldg,
                               int64_t batch_stride, fsdp_dtype dtype, void *out, int64_t ldo,
                               int64_t out_batch_stride, int steps, double eps, double a, double b,
                               double c, void *workspace, int64_t workspace_bytes, void *stream);
fsdp_status fsdp_newton_schulz_workspace(int64_t batch, int64_t m, int64_t n, int64_t *bytes);

typedef struct {
    double lr, momentum, weight_decay;
    double eps;          /* added to the Frobenius norm */
    double update_scale; /* multiplies lr in the update; > 0 */
    int nesterov;        /* u = g + momentum * M rather than u = M */
    int steps;           /* Newton-Schulz steps */
    double a, b, c;      /* its coefficients */
} fsdp_muon_hp;

#define FSDP_MUON_MAX_MATRICES 64

/* One Muon step of n_mats matrices [m, n] (1 <= n_mats <=
 * FSDP_MUON_MAX_MATRICES), in place. For each, from R ranks' gradients
 * (grads[i*R + q], grad_dtype) with the fixed-order fold of
 * fsdp_reduce_scatter_adamw:
 *   g = (g_0 + g_1 + ... + g_{R-1}) * fl(1/R);  M = momentum * M + g
 *   u = g + momentum * M  (nesterov)  or  M
 *   w = w * (1 - lr * weight_decay) - lr * update_scale * newton_schulz(u)
 * momentum[i], master[i]: fp32; param_out: NULL, or n_mats bf16 matrices that
 * receive the rounding of the new master. All matrices are contiguous. A
 * whole matrix is needed at one place: with shards, this is the owner rank's
 * update of a ZeRO-3 layout. */
fsdp_status fsdp_muon(int n_mats, int64_t m, int64_t n, int R, const void *const *grads,
                      fsdp_dtype grad_dtype, float *const *momentum, float *const *master,
                      void *const *param_out, const fsdp_muon_hp *hp, void *workspace,
                      int64_t workspace_bytes, void *stream);
fsdp_status fsdp_muon_workspace(int n_mats, int64_t m, int64_t n, int64_t *bytes);

/* The number of thread blocks of the matrix kernels on CUDA device `device`
 * that gave up a wait since the library was loaded; 0 in every valid run.
 * Waits for all work on the device. Errors: FSDP_EINVAL, FSDP_ECUDA. */
fsdp_status fsdp_ops_wait_timeouts(int device, uint64_t *count);

#ifdef __cplusplus
}
#endif

#endif /* FSDP_OPS_H */
