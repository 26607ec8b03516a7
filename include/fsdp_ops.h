/*
 * fsdp_ops.h -- C ABI of the training-step operators around a sharded unit
 * (GB300, sm_103a): what produces the gradients that the shard engine
 * reduces, and a matrix-aware update that uses them.
 *
 *   fsdp_layer_norm, fsdp_layer_norm_backward
 *   fsdp_linear_cross_entropy      loss of a linear head, with its gradients
 *   fsdp_grouped_linear, fsdp_grouped_linear_backward
 *                                  a linear layer per expert, ragged rows
 *   fsdp_dropout                   with a mask that is never stored
 *   fsdp_preference_loss, fsdp_policy_loss
 *                                  from what tokens cost, with gradients
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
 *    count, for the experts' products by their offsets: the same call gives the
 *    same bits every time. The same values in
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

/* The same with a weight for each row (row_weights [rows], fp32; NULL: 1):
 *   loss = sum_n row_weights_n row_loss_n / count, or the sum
 * and G_n is row_weights_n times its own; row_loss itself has no weight. A row
 * of weight 0 has row_loss, and no part in the loss and the gradients, its
 * hidden being finite. Weights of ignored rows are not used. With row_weights =
 * d L / d row_loss and FSDP_SUM the gradients are those of any L of the row
 * losses (fsdp_preference_loss, fsdp_policy_loss). The workspace is
 * fsdp_linear_cross_entropy's. */
fsdp_status fsdp_linear_cross_entropy_weighted(int64_t rows, int64_t cols, int64_t vocab,
                                               const void *hidden, int64_t ldh, const void *weight,
                                               int64_t ldw, const int64_t *targets,
                                               int64_t ignore_index, const float *row_weights,
                                               fsdp_reduction reduction, double grad_scale,
                                               float *loss, float *row_loss, void *dhidden,
                                               int64_t lddh, void *dweight, int64_t lddw,
                                               int64_t piece_rows, void *workspace,
                                               int64_t workspace_bytes, void *stream);

/* A linear layer per expert, on rows that lie expert by expert: expert e has
 * the rows offsets[e] <= r < offsets[e+1], any number of them,
 *   y_r = weight_e x_r
 * x [rows, k], weight [experts, n, k] (w_stride elements from one to the
 * next), y [rows, n]: bf16, each sum rounded once. offsets [experts + 1] int64
 * are read on the device; they are taken clamped to [0, rows] and to their
 * running maximum, so none leads out of the buffers. Rows of no expert, before
 * offsets[0] or from offsets[experts] on, get y = 0, whatever x holds there.
 * rows = 0 does nothing; experts in [1, 65535], n and k >= 1. */
fsdp_status fsdp_grouped_linear(int64_t rows, int64_t experts, int64_t n, int64_t k, const void *x,
                                int64_t ldx, const void *weight, int64_t ldw, int64_t w_stride,
                                const int64_t *offsets, void *y, int64_t ldy, void *workspace,
                                int64_t workspace_bytes, void *stream);
/* x_on_16: x starts on 16 bytes and ldx is a multiple of 8; w_on_16 likewise
 * (ldw and w_stride); else the workspace holds a copy that does. It may be 0. */
fsdp_status fsdp_grouped_linear_workspace(int64_t rows, int64_t experts, int64_t n, int64_t k,
                                          int x_on_16, int w_on_16, int64_t *bytes);

/* Its gradients: dx_r = weight_e^T dy_r (0 for rows of no expert) and
 *   dweight_e = sum over the rows r of e of dy_r x_r^T (0 for an expert without)
 * dy [rows, n], dx [rows, k], dweight [experts, n, k]: bf16; dweight may be a
 * view of a unit's gradient buffer. rows = 0 writes zeros to dweight. */
fsdp_status fsdp_grouped_linear_backward(int64_t rows, int64_t experts, int64_t n, int64_t k,
                                         const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                         const void *weight, int64_t ldw, int64_t w_stride,
                                         const int64_t *offsets, void *dx, int64_t lddx,
                                         void *dweight, int64_t lddw, int64_t dw_stride,
                                         void *workspace, int64_t workspace_bytes, void *stream);
/* It may be 0. */
fsdp_status fsdp_grouped_linear_backward_workspace(int64_t rows, int64_t experts, int64_t n,
                                                   int64_t k, int dy_on_16, int x_on_16, int w_on_16,
                                                   int64_t *bytes);

/* Dropout of x [rows, cols], added to residual [rows, cols] (NULL: 0):
 *   T = round((1 - p) 65536);  y_ij = residual_ij + (draw_ij < T ? x_ij 65536 / T : 0)
 * so that the mean of y over the draws is residual + x. draw_ij is the 16-bit
 * number j % 8 (the low half of the first word first) of Philox4x32-10 for the
 * counter (j / 8, i, offset mod 2^32, offset / 2^32) and the key (seed mod
 * 2^32, seed / 2^32): the backward pass is the same call on dy, without a
 * residual, whatever the strides. What is dropped counts for nothing, infinite
 * or NaN. offset_more: NULL, or an int64 on the device that is added to offset
 * (mod 2^64) when the kernel runs, for calls that are captured and replayed.
 * x, residual, y: dtype. p in [0, 1]; T = 0 (p = 1, or nearer to it than 2^-17)
 * drops everything. */
fsdp_status fsdp_dropout(int64_t rows, int64_t cols, const void *x, int64_t ldx,
                         const void *residual, int64_t ldr, fsdp_dtype dtype, double p,
                         uint64_t seed, uint64_t offset, const int64_t *offset_more, void *y,
                         int64_t ldy, void *stream);

/* The losses below work on row_loss = -log p(token), as
 * fsdp_linear_cross_entropy leaves it, and give row_weights = d loss / d
 * row_loss, as fsdp_linear_cross_entropy_weighted takes it. Sequences are
 * ranges of rows: sequence s has the rows offsets[s] <= r < offsets[s+1]; rows
 * of none, and rows whose mask byte is 0 (mask NULL: none), count for nothing
 * whatever they hold, and have weight 0. Offsets that fall or leave [0, rows]
 * make the loss (margins, kl, clipped) NaN and the weights 0.
 *
 * Preference loss over pairs: sequence 2i is the preferred one of pair i,
 * 2i + 1 the other.
 *   s = sum over a sequence's rows of ref_row_loss - row_loss  (or their mean)
 *   m_i = beta (s_2i - s_2i+1)
 *   loss = mean (or sum) over i of -(1 - a) log sigma(m_i) - a log sigma(-m_i)
 * a = label_smoothing in [0, 1]. ref_row_loss NULL: 0. row_loss, ref_row_loss,
 * row_weights [rows], margins [pairs], loss [1]: fp32; offsets [2 pairs + 1]
 * int64. Sums over rows are held in two fp32 numbers (46 bits). The mean of no pairs, or of no rows, is 0. */
fsdp_status fsdp_preference_loss(int64_t rows, int64_t pairs, const float *row_loss,
                                 const float *ref_row_loss, const int64_t *offsets,
                                 const uint8_t *mask, double beta, double label_smoothing,
                                 int average, fsdp_reduction reduction, float *loss, float *margins,
                                 float *row_weights, void *workspace, int64_t workspace_bytes,
                                 void *stream);

typedef enum { FSDP_POLICY_MEAN = 0, FSDP_POLICY_SUM = 1, FSDP_POLICY_SEQUENCE = 2 } fsdp_policy_reduction;

/* Clipped policy loss with a KL term. For each row that counts, with
 * l = old_row_loss - row_loss, A its advantage and d = row_loss - ref_row_loss:
 *   term = -min(exp(l) A, clip(exp(l), 1 - clip_low, 1 + clip_high) A)
 *          + kl_coef (exp(d) - 1 - d)
 * (A = 0: the KL term alone; ref_row_loss NULL or kl_coef 0: without it,
 * infinite or not; a ratio at a border is not clipped, on which side one is
 * being decided without l's rounding). loss is the terms' mean over the rows
 * that count, their sum, or the mean over the sequences with such rows of their
 * means. sequences and offsets [sequences + 1] int64 may be 0 and NULL: then
 * all rows are one's, and the last reduction is refused. advantages: [rows], or
 * [sequences] where by_sequence is not 0. kl, clipped [1], fp32: the mean of
 * exp(d) - 1 - d and the share of clipped rows, both over the rows that count.
 * exp(l) and exp(d) may pass fp32's range: what comes of a row is infinite only
 * where fp32 does not hold it with A or kl_coef and the row's part of the mean. */
fsdp_status fsdp_policy_loss(int64_t rows, int64_t sequences, const float *row_loss,
                             const float *old_row_loss, const float *ref_row_loss,
                             const float *advantages, int by_sequence, const int64_t *offsets,
                             const uint8_t *mask, double clip_low, double clip_high, double kl_coef,
                             fsdp_policy_reduction reduction, float *loss, float *row_weights,
                             float *kl, float *clipped, void *workspace, int64_t workspace_bytes,
                             void *stream);
/* Of either loss; sequences: 2 pairs, or 0 without offsets. It may be 0. */
fsdp_status fsdp_tuning_loss_workspace(int64_t rows, int64_t sequences, int64_t *bytes);

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
