/*
 * cgtp_train.h -- C ABI of libcgtp.so, continued: the node-side operators that
 * a training step needs around the CGTP convolution of cgtp.h.
 *
 *   - the embedding of species (token) ids as feature rows, with a scale, and
 *     the gradient of its table;
 *   - a group normalisation with an activation over ragged segments of
 *     channels-last rows (the invariant, l = 0, rows of the atoms of each
 *     structure of a batch), and its gradient;
 *   - the orthogonalised update of a stack of weight matrices (the mixing
 *     matrices of cgtp_path_mix_fwd, say) by Newton-Schulz products.
 *
 * Conventions, beside those of cgtp.h (device pointers owned by the caller,
 * asynchronous on the given stream, outputs overwritten, every sum in a fixed
 * order so that results are bitwise reproducible, a status and never an
 * abort, no allocation, capturable into a HIP graph):
 *   - no plan: sizes are arguments, and the element type of the large arrays
 *     is a cgtp_dtype_t.  Statistics, gamma and beta and their gradients are
 *     fp32 whatever the type.  Sums over rows run in fp64, elementwise terms
 *     in fp32; Newton-Schulz products run as three fp16 products with fp32
 *     accumulation, which together carry 23 bits of their operands, for either
 *     type (in fp64 for matrices of up to 16 rows or columns and 32768
 *     elements); each result is rounded to its type once.
 *   - arrays are aligned to their element type; rows that start on 16-byte
 *     boundaries (pointer, row stride and channel count) take the wide-load
 *     kernels.  Row strides count elements and are at least the row's width.
 *     Workspaces are aligned to 256 bytes and hold nothing between calls; where
 *     the size call says 0 none is needed (NULL).
 *   - an output must not overlap an input.
 */
#ifndef CGTP_TRAIN_H
#define CGTP_TRAIN_H

#include "cgtp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CGTP_F32 = 0,
    CGTP_BF16 = 1
} cgtp_dtype_t;

typedef enum {
    CGTP_ACT_NONE = 0,
    CGTP_ACT_SILU = 1, /* z / (1 + exp(-z)) */
    CGTP_ACT_TANH = 2
} cgtp_act_t;

/* ---- embedding ---------------------------------------------------------------
 * out[n][c] = scale * table[ids[n]][c], zero where ids[n] is outside
 * [0, table_rows) (padding): table [table_rows][channels], ids [n_rows] int32,
 * out n_rows rows of `channels`, ld_out elements apart (so that out may be the
 * l = 0 rows of a [N][D][C] feature array, whose other rows are left alone).
 * The product is formed in fp32 and rounded once. */
cgtp_status_t cgtp_embed_fwd(cgtp_dtype_t dtype, int64_t n_rows, int64_t table_rows, int64_t channels,
                             const int32_t* ids, const void* table, float scale, void* out, int64_t ld_out,
                             hipStream_t stream);

/* Workspace bytes of cgtp_embed_bwd: the sorted ids and the partial sums of
 * ids whose rows span several runs. */
cgtp_status_t cgtp_embed_bwd_workspace_size(cgtp_dtype_t dtype, int64_t n_rows, int64_t table_rows,
                                            int64_t channels, size_t* bytes);

/* Gradient of the table:
 *   grad_table[v][c] = scale * sum_{n: ids[n] = v} grad_out[n][c],
 * every row written (zero for a row that no id names), ids outside
 * [0, table_rows) ignored.  grad_out rows are ld_grad elements apart.  The
 * rows are summed in fp64 by sorted ids, without atomics on values. */
cgtp_status_t cgtp_embed_bwd(cgtp_dtype_t dtype, int64_t n_rows, int64_t table_rows, int64_t channels,
                             const int32_t* ids, const void* grad_out, int64_t ld_grad, float scale,
                             void* grad_table, void* ws, size_t ws_bytes, hipStream_t stream);

/* ---- group normalisation with an activation ------------------------------------
 * The n_rows rows of `channels` values (ld_x elements apart) form n_segments
 * consecutive segments: rows seg_ptr[b] .. seg_ptr[b+1]-1 (int32 [n_segments+1],
 * seg_ptr[0] = 0, non-decreasing, seg_ptr[n_segments] = n_rows), or equal ones
 * where seg_ptr is NULL (n_rows a multiple of n_segments).  `groups` divides
 * `channels`; group g of segment b is the M = rows * channels/groups values of
 * its channels:
 *   mean[b][g], rstd[b][g] = 1 / sqrt(variance + eps)   (variance over M, biased)
 *   y = act((x - mean) * rstd * gamma[c] + beta[c])
 * gamma NULL counts as ones, beta NULL as zeros.  An empty segment has mean 0
 * and variance 0.  mean and rstd [n_segments][groups] fp32 are what the
 * backward needs.  y's rows are ld_y elements apart.
 * Offsets that break the precondition give unspecified values but no access
 * out of bounds. */

/* Workspace bytes of one direction (backward 0 or 1), with offsets (ragged 1) or
 * equal segments (0). */
cgtp_status_t cgtp_norm_act_workspace_size(cgtp_dtype_t dtype, int64_t n_rows, int64_t n_segments,
                                           int64_t channels, int64_t groups, int ragged, int backward, size_t* bytes);

cgtp_status_t cgtp_norm_act_fwd(cgtp_dtype_t dtype, cgtp_act_t act, int64_t n_rows, int64_t n_segments,
                                int64_t channels, int64_t groups, const int32_t* seg_ptr, float eps, const void* x,
                                int64_t ld_x, const float* gamma, const float* beta, void* y, int64_t ld_y,
                                float* mean, float* rstd, void* ws, size_t ws_bytes, hipStream_t stream);

/* Backward of L = <grad_y, y>, with xhat = (x - mean) * rstd and
 * dz = grad_y * act'(xhat * gamma + beta) recomputed from x and the forward's
 * statistics:
 *   grad_beta[c] = sum dz,  grad_gamma[c] = sum dz * xhat        (over all rows)
 *   grad_x = rstd * (dz * gamma - s1 - xhat * s2),
 *     s1 = sum dz * gamma / M,  s2 = sum dz * gamma * xhat / M   (over the group)
 * grad_x's rows are ld_dx elements apart.  Each gradient may be NULL. */
cgtp_status_t cgtp_norm_act_bwd(cgtp_dtype_t dtype, cgtp_act_t act, int64_t n_rows, int64_t n_segments,
                                int64_t channels, int64_t groups, const int32_t* seg_ptr, const void* x,
                                int64_t ld_x, const float* mean, const float* rstd, const float* gamma,
                                const float* beta, const void* grad_y, int64_t ld_dy, void* grad_x, int64_t ld_dx,
                                float* grad_gamma, float* grad_beta, void* ws, size_t ws_bytes,
                                hipStream_t stream);

/* ---- orthogonalised update ---------------------------------------------------------
 * out = scale * Q(G) for each of `batch` matrices [rows][cols] (contiguous), by
 * `steps` Newton-Schulz steps of the odd polynomial a x + b x^3 + c x^5:
 *   X = G / (||G||_F + eps);   steps times: A = X X^T, X <- a X + (b A + c A A) X
 * (A = X^T X, products from the other side, where rows > cols: the same
 * result).  Every singular value x of X goes through the polynomial `steps`
 * times and the singular vectors stay; with a = 3.4445, b = -4.7750,
 * c = 2.0315 and five steps all but the smallest end near 1, so that the
 * update of a weight matrix acts on all its directions alike.  A zero matrix
 * gives zeros (eps > 0); a matrix with an infinity or NaN gives NaN throughout, and the
 * others of the stack are not touched by it.
 * 1 <= steps <= 64.  The coefficients must keep the iterates bounded: over
 * singular values in [0, 1] the polynomial's maximum, followed from step to
 * step, and that of b y + c y^2 must stay within 1e-6 .. 1e6
 * (CGTP_ERR_INVALID_ARG otherwise; b = c = 0 is refused so). */

/* Workspace bytes. */
cgtp_status_t cgtp_orthogonalize_workspace_size(cgtp_dtype_t dtype, int64_t batch, int64_t rows, int64_t cols,
                                                size_t* bytes);

cgtp_status_t cgtp_orthogonalize(cgtp_dtype_t dtype, int64_t batch, int64_t rows, int64_t cols, int steps, double a,
                                 double b, double c, float eps, float scale, const void* G, void* out, void* ws,
                                 size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CGTP_TRAIN_H */
