/*
 * strata_train.h -- the ends of a training step around the sparse MoE layer:
 * the router's balance losses, token rows in and their table's gradient,
 * softmax cross entropy over the vocabulary with its gradients, and the
 * experts' updates orthogonalised by Newton-Schulz products.  With
 * strata_ops.h (the sparse block, forward and backward) they are a training
 * step of a sparse model; attention, the optimiser's momentum and its step
 * are the caller's.
 *
 * Conventions are those of strata_ops.h: [dev] and [host] pointers, memory
 * owned by the caller, kernels only on `stream` (so a call can be captured
 * in a HIP graph), host validation before any launch and nothing enqueued
 * when it fails, no allocation and no host synchronisation.  Every [dev]
 * pointer to rows, matrices or a workspace must be 16-byte aligned and rows
 * follow each other without padding; the current HIP device must be the
 * stream's.  A workspace needs no initialisation; calls that may overlap need
 * workspaces of their own (a captured graph keeps using the one it was
 * captured with).  An output shares no memory with another argument unless
 * the call says that it may.  Results are the same bits on every run.  Sums,
 * softmax statistics and norms are fp32 or more; a bf16 output is rounded
 * once (to nearest even) as it is stored.
 */
#ifndef STRATA_TRAIN_H
#define STRATA_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#include "strata_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Balance losses of a router, and the picks counted per expert.  Over the n
 * tokens that count, with p[t] = softmax(z[t]):
 *   counts[e] = picks of e,   prob[e] = (1/n) sum_t p[t][e],
 *   lse[t]    = log sum_e exp(z[t][e])
 *   losses[0] = E sum_e counts[e] / (n k) * prob[e]     (1 where even)
 *   losses[1] = (1/n) sum_t lse[t]^2
 * A token does not count where keep (nullable: all count) is 0, or where all
 * its logits are -inf: its lse is 0, its picks are not counted, and what its
 * logits hold besides is not used.  n = 0: both losses and prob are 0.
 */

/* Bytes of workspace strata_moe_balance needs; 0 for arguments it refuses. */
size_t strata_moe_balance_workspace_bytes(int32_t T, int32_t k, int32_t n_experts);

/*   z    [dev] [T][E] of zdtype: the router's logits (their product with x is the caller's).
 *   idx  [dev] [T][k] int32: the picks; ids outside 0..E-1 are not counted.
 *   keep [dev] [T] bytes, nullable.
 *   losses [2] fp32, counts [E] int32, prob [E] fp32 (nullable), lse [T] fp32, tokens [1] int32 (n): [dev].
 * T = 0 writes zeros.  EINVAL: a null or misaligned pointer (idx, counts, tokens and the fp32 vectors need
 * 4 bytes only), T < 0, k outside 1..32, E outside 1..1024, a bad dtype; EUNSUPPORTED: T > 2^23;
 * EWORKSPACE; EHIP. */
strata_status strata_moe_balance(const void *z, strata_xdtype zdtype, const int32_t *idx, const uint8_t *keep, int32_t T,
                                 int32_t k, int32_t n_experts, float *losses, int32_t *counts, float *prob, float *lse,
                                 int32_t *tokens, void *ws, size_t ws_bytes, void *stream);

/* Gradient of the logits, with lse, counts and tokens as the forward call left them (counts and tokens may
 * be sums over several calls or ranks: then the losses are those of all their tokens, counts being
 * constants) and dlosses [dev] [2] fp32 the gradients of the losses:
 *   g[e] = dlosses[0] E counts[e] / (tokens^2 k)
 *   dz[t][e] = p[t][e] (g[e] - sum_f p[t][f] g[f] + dlosses[1] 2 lse[t] / tokens)  [dev] [T][E] of zdtype
 *              + sum of dpicks[t][r] over r ascending with idx[t][r] = e
 *   dpicks [dev] [T][k] fp32, nullable: gradients of the picked logits (dz of strata_moe_combine_backward).
 * A token that does not count gets zeros, and its dpicks are not used.  dz may be z.  T = 0: no-op.
 * tokens < 1 stands for 1.  Errors as above; no workspace. */
strata_status strata_moe_balance_backward(const void *z, strata_xdtype zdtype, const int32_t *idx, const uint8_t *keep,
                                          int32_t T, int32_t k, int32_t n_experts, const float *lse,
                                          const int32_t *counts, const int32_t *tokens, const float *dlosses,
                                          const float *dpicks, void *dz, void *stream);

/* ------------------------------------------------------------------------
 * Rows of a table by token id, and the table's gradient.
 */

/* out[t] = scale * W[ids[t]]; an id outside 0..V-1 (padding) gives zeros.
 *   W [dev] [V][d] of wdtype, ids [dev] [T] int32, out [dev] [T][d] of odtype.
 * T = 0: no-op.  EINVAL: a null or misaligned pointer, T < 0, V < 1, d < 1, a bad dtype, a scale that is
 * not finite; EUNSUPPORTED: T > 2^23, d > 2^24, V > 2^24; EHIP. */
strata_status strata_embed(const void *W, strata_xdtype wdtype, int32_t V, int32_t d, const int32_t *ids, int32_t T,
                           float scale, void *out, strata_xdtype odtype, void *stream);

enum { STRATA_ACCUMULATE = 1u }; /* flags: the gradient is added to what the matrix holds */

/* Bytes of workspace the gradient needs; 0 for arguments it refuses. */
size_t strata_embed_backward_workspace_bytes(int32_t T, int32_t V, int32_t d);

/* dW[v] = scale * sum of dout[t] over the t with ids[t] = v: the tokens are sorted by id and each row's are
 * summed in an order that the ids alone decide.
 *   dout [dev] [T][d] of odtype, dW [dev] [V][d] of wdtype.
 *   flags: 0: every row is written, one without tokens with zeros (T = 0 writes all zeros);
 *          STRATA_ACCUMULATE: rows with tokens get dW + the sum (added in fp32), others are left as they were.
 * Rows of dout whose id is outside 0..V-1 are not read.  Errors as above, and EINVAL for unknown flags,
 * EUNSUPPORTED for V > 2^20 - 1 or T > 2^22; EWORKSPACE. */
strata_status strata_embed_backward(const void *dout, strata_xdtype odtype, const int32_t *ids, int32_t T, int32_t V,
                                    int32_t d, float scale, void *dW, strata_xdtype wdtype, uint32_t flags, void *ws,
                                    size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Softmax cross entropy over a vocabulary, from the hidden rows and the
 * output matrix.  With z[t] = W h[t] (bf16 operands, fp32 sums):
 *   lse[t] = log sum_v exp(z[t][v]),   loss[t] = lse[t] - z[t][targets[t]].
 * The logits are not kept: the forward call leaves each tile's maximum and
 * sum, the gradient computes them again in pieces of the vocabulary.  A token
 * whose target is outside 0..V-1 (a prompt's, padding) has loss 0 and lse 0,
 * no gradient, and costs no products; what its h, dloss and dlse hold is not
 * used.  Limits: d % 8 == 0, 8 <= d <= 16384, 1 <= V <= 2^20, T <= 2^20,
 * T*d <= 2^33, T*V <= 2^38, else EUNSUPPORTED.
 */

/* Bytes of workspace the calls need; 0 for arguments they refuse. */
size_t strata_vocab_loss_workspace_bytes(int32_t T, int32_t V, int32_t d);
size_t strata_vocab_loss_backward_workspace_bytes(int32_t T, int32_t V, int32_t d);

/*   h [dev] [T][d] bf16, W [dev] [V][d] bf16, targets [dev] [T] int32, loss and lse [dev] [T] fp32.
 * T = 0: no-op.  EINVAL: a null or misaligned pointer, T < 0; EWORKSPACE; EHIP. */
strata_status strata_vocab_loss(const void *h, const void *W, const int32_t *targets, int32_t T, int32_t V, int32_t d,
                                float *loss, float *lse, void *ws, size_t ws_bytes, void *stream);

/* Gradients, with lse as the forward call left it, dloss [dev] [T] fp32 (of loss) and dlse [dev] [T] fp32
 * (of lse, nullable: zeros):
 *   dz[t][v] = (dloss[t] + dlse[t]) exp(z[t][v] - lse[t]) - (v == targets[t] ? dloss[t] : 0)
 *   dh[t] = sum_v dz[t][v] W[v]     [dev] [T][d] of dhdtype, nullable
 *   dW[v] = sum_t dz[t][v] h[t]     [dev] [V][d] of dwdtype, nullable
 *   flags: STRATA_ACCUMULATE: dW + the sum is written to dW (added in fp32), else the sum.
 * dz enters the products as bf16 (over the first dloss's mantissa) where the output is bf16, and with all its
 * 24 bits, as three bf16 pieces, where it is fp32.  T = 0 writes zeros to dW (without the flag).  Errors as
 * above, and EINVAL for a bad dtype of an output that is given, or unknown flags. */
strata_status strata_vocab_loss_backward(const void *h, const void *W, const int32_t *targets, int32_t T, int32_t V,
                                         int32_t d, const float *lse, const float *dloss, const float *dlse, void *dh,
                                         strata_xdtype dhdtype, void *dW, strata_xdtype dwdtype, uint32_t flags, void *ws,
                                         size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Matrices orthogonalised by Newton-Schulz products: for each of n matrices
 *   X_0 = G / (|G|_F + eps)
 *   X_{i+1} = a X_i + (b A + c A^2) X_i,  A = X_i X_i^T     (i < steps)
 *   out = scale * X_steps
 * (the same polynomial from the right where N > K).  Operands of the products
 * are fp16 (11 bits), X itself is kept in two fp16 pieces (22 bits; the last of
 * several steps takes the first piece alone), so that directions that G lacks
 * are not made of its roundings; the diagonals of A and of b A + c A^2 count in
 * fp32, and sums are fp32.
 * A matrix of zeros gives zeros; infinities and NaN stay in their matrix, and
 * coefficients that take X or b A + c A^2 out of fp16's range make infinities
 * or NaN.
 */

/* Bytes of workspace the call needs; 0 for arguments it refuses. */
size_t strata_orthogonalise_workspace_bytes(int32_t n, int32_t N, int32_t K);

/*   G [dev] [n][N][K] of gdtype, out [dev] [n][N][K] bf16; out may be a bf16 G.
 *   steps 0..32; coefficients [host] {a, b, c}.
 * n = 0: no-op.  EINVAL: a null or misaligned pointer, n < 0, N or K < 1, a bad dtype, steps outside 0..32,
 * a coefficient or scale that is not finite, eps not a positive finite number, an out that shares memory with
 * G otherwise; EUNSUPPORTED: N or K > 16384,
 * n > 1024, n*N*K > 2^33; EWORKSPACE; EHIP. */
strata_status strata_orthogonalise(const void *G, strata_xdtype gdtype, int32_t n, int32_t N, int32_t K, int32_t steps,
                                   const float *coefficients, float scale, float eps, void *out, void *ws, size_t ws_bytes,
                                   void *stream);

#ifdef __cplusplus
}
#endif
#endif /* STRATA_TRAIN_H */
