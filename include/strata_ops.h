/*
 * strata_ops.h -- operators around the sparse MoE layer, each with its
 * gradient: tokens sorted by expert and back, the experts' products over the
 * sorted rows with dense bf16 weights, and the norms before and after a
 * block fused with its gate and residual scale.  With strata_moe_route they
 * are the sparse parts of a trainable block; the activation between the
 * products, the router's own gradient (from dz) and packing the trained weights
 * into the format of strata_moe.h are the caller's.
 *
 * Conventions are those of strata_moe.h: [dev] and [host] pointers, memory
 * owned by the caller, kernels only on `stream` (so a call can be captured
 * in a HIP graph), host validation before any launch and nothing enqueued
 * when it fails, no allocation and no host synchronisation.  Every [dev]
 * pointer to rows, gains, matrices or a workspace must be 16-byte aligned
 * and every row follows the one before it (no padding between rows); the
 * current HIP device must be the stream's.  A workspace needs no
 * initialisation; calls that may overlap need workspaces of their own (a
 * captured graph keeps using the one it was captured with).  An output shares
 * no memory with another argument unless the call says that it may.  Results are the
 * same bits on every run: no sum depends on the order in which blocks run.
 * All sums, norms and their statistics are fp32; a bf16 output is rounded
 * once (to nearest even) as it is stored.
 */
#ifndef STRATA_OPS_H
#define STRATA_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "strata_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Tokens sorted by expert, and back.
 *
 * A pick is an entry of idx [T][k]; its flat index is t*k + r.  Picks with
 * an id outside 0..E-1 are dropped (over capacity, padding, or experts held
 * elsewhere).  Kept picks get the slots 0, 1, ... in the order (expert asc,
 * flat index asc); pos maps a pick to its slot (-1: dropped), perm a slot to
 * its pick (-1 in the slots behind the last kept one).  Without drops the
 * four outputs are those of strata_route_out.  The same expert may appear
 * more than once in a token's picks.
 */

/* Bytes of workspace strata_moe_sort needs; 0 for arguments it refuses. */
size_t strata_moe_sort_workspace_bytes(int32_t T, int32_t k, int32_t n_experts);

/* counts [E], offsets [E+1] (exclusive prefix sum; offsets[E] = kept picks),
 * perm [T*k], pos [T*k]: [dev] int32, each nullable.  idx: [dev] [T][k].
 * T = 0 writes zero counts and offsets.  EINVAL: a null idx or workspace with
 * T > 0, T < 0, k outside 1..32, E outside 1..1024, a misaligned workspace, an
 * output that shares memory with idx, or with the workspace above 65535 picks;
 * EUNSUPPORTED: T*k > 2^31 - 1; EWORKSPACE; EHIP. */
strata_status strata_moe_sort(const int32_t *idx, int32_t T, int32_t k, int32_t n_experts, int32_t *counts,
                              int32_t *offsets, int32_t *perm, int32_t *pos, void *ws, size_t ws_bytes, void *stream);

/* xs[pos[t*k + r]] = x[t]: the token rows copied to their picks' slots.
 *   x   [dev] [T][d], xs [dev] [rows][d], both xdtype.
 *   pos [dev] [T*k] int32; entries outside 0..rows-1 copy nothing.
 * Rows of xs without a pick are left as they were; where two picks name the
 * same row, which token's values it gets is not specified.  T = 0: no-op.  EINVAL: a
 * null or misaligned pointer, T, rows < 0, d < 1, k outside 1..32, a bad
 * dtype; EUNSUPPORTED: T > 2^23, d > 2^24 or T*k > 2^31 - 1; EHIP. */
strata_status strata_moe_dispatch(const void *x, strata_xdtype xdtype, int32_t T, int32_t k, int32_t d,
                                  const int32_t *pos, void *xs, int32_t rows, void *stream);

/* Its gradient: dx[t] = sum over r ascending of dxs[pos[t*k + r]]; a token
 * whose picks are all dropped gets zeros.  Errors as above. */
strata_status strata_moe_dispatch_backward(const void *dxs, strata_xdtype xdtype, int32_t rows, const int32_t *pos,
                                           int32_t T, int32_t k, int32_t d, void *dx, void *stream);

/* out[t] = base[t] + sum over r ascending of w[t][r] * ys[pos[t*k + r]].
 *   ys   [dev] [rows][d] of ydtype; base (nullable: zeros) and out [dev] [T][d]
 *        of odtype; out may be base.
 *   w    [dev] [T][k] fp32, or NULL for weights of 1.
 * A pick with pos outside 0..rows-1 is skipped: its weight and row are not
 * read as numbers, whatever they hold.  Errors as for strata_moe_dispatch. */
strata_status strata_moe_combine(const void *ys, strata_xdtype ydtype, int32_t rows, const int32_t *pos,
                                 const float *w, int32_t T, int32_t k, int32_t d, const void *base, void *out,
                                 strata_xdtype odtype, void *stream);

/* Gradient of the combine with weights (the gradient of base is dout):
 *   dys[pos[t*k + r]] = w[t][r] * dout[t]           [dev] [rows][d] of ydtype
 *   dw[t][r] = <dout[t], ys[pos[t*k + r]]>, 0 for a skipped pick   [dev] [T][k] fp32
 *   dz[t][r] = w[t][r] * (dw[t][r] - sum_s w[t][s] dw[t][s])       [dev] [T][k] fp32
 * dz is the gradient of the picked logits when the weights are their softmax
 * over the k picks (the gates of strata_moe_route); a skipped pick's weight
 * enters its own dz alone.  Each output is nullable; rows of dys without a pick are left as they were.  dys may be
 * ys.  pos must name no row twice.  Errors as above, and EINVAL for a null w. */
strata_status strata_moe_combine_backward(const void *dout, strata_xdtype odtype, const void *ys,
                                          strata_xdtype ydtype, int32_t rows, const int32_t *pos, const float *w,
                                          int32_t T, int32_t k, int32_t d, void *dys, float *dw, float *dz,
                                          void *stream);

/* ------------------------------------------------------------------------
 * The experts' products over rows sorted by expert.  Rows offsets[e] ..
 * offsets[e+1]-1 belong to expert e; W [E][N][K] bf16 (out x in, row-major).
 * offsets: [dev] int32 [E+1] as strata_moe_sort and strata_moe_route give
 * them, ascending.  Entries outside 0..rows are cut to it; which rows an
 * expert gets from offsets that do not ascend is not specified, but nothing
 * outside the buffers is touched.  Matrix-core products of bf16 operands,
 * summed in fp32.
 * Limits: N % 8 == 0, K % 8 == 0, 8 <= N, K <= 65536, N*K <= 2^29, 1 <= E <=
 * 1024, E*N*K <= 2^37, rows <= 2^22, else EUNSUPPORTED.  EINVAL: a null or
 * misaligned pointer, rows < 0, a bad dtype, an output that shares memory with
 * the workspace; EWORKSPACE; EHIP.  Rows behind
 * the last expert's are not read and their outputs are left as they were.
 */

/* Bytes of workspace each of the three calls needs; 0 for arguments they refuse. */
size_t strata_moe_grouped_workspace_bytes(int32_t rows, int32_t n_experts, int32_t N, int32_t K);

/* y[s] = W_e x[s]: x [dev] [rows][K] bf16, y [dev] [rows][N] of ydtype. */
strata_status strata_moe_grouped_product(const void *x, const void *W, const int32_t *offsets, int32_t rows,
                                         int32_t n_experts, int32_t N, int32_t K, void *y, strata_xdtype ydtype,
                                         void *ws, size_t ws_bytes, void *stream);

/* dx[s] = W_e^T dy[s]: dy [dev] [rows][N] bf16, dx [dev] [rows][K] of xdtype. */
strata_status strata_moe_grouped_dgrad(const void *dy, const void *W, const int32_t *offsets, int32_t rows,
                                       int32_t n_experts, int32_t N, int32_t K, void *dx, strata_xdtype xdtype,
                                       void *ws, size_t ws_bytes, void *stream);

/* dW_e = sum over e's rows of dy[s] x[s]^T: dW [dev] [E][N][K] of wdtype; every
 * expert is written, one without rows with zeros (rows = 0 writes all zeros). */
strata_status strata_moe_grouped_wgrad(const void *dy, const void *x, const int32_t *offsets, int32_t rows,
                                       int32_t n_experts, int32_t N, int32_t K, void *dW, strata_xdtype wdtype,
                                       void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Norms before and after a block, fused with the branch's gate and the
 * residual scale.  Per row, with y the block's output and x the residual row:
 *   n = y                         or with STRATA_POST_NORM  y * rstd(y) * g_post
 *   r = resid_scale * x + branch_scale * G * n
 *   u = r * rstd(r) * g_pre       with STRATA_PRE_NORM: the next block's input
 *   rstd(v) = 1 / sqrt(mean(v^2) + eps)
 * G = 1, a gate value for the row (STRATA_GATE_TOKEN) or one per element
 * (STRATA_GATE_CHANNEL); with STRATA_GATE_SIGMOID the sigmoid of it.
 * u is the norm of r before r is rounded for its store.
 */
enum {
    STRATA_POST_NORM = 1u,
    STRATA_PRE_NORM = 2u,
    STRATA_GATE_TOKEN = 4u,    /* gate: [T] fp32 */
    STRATA_GATE_CHANNEL = 8u,  /* gate: [T][d] of y_dtype */
    STRATA_GATE_SIGMOID = 16u  /* with one of the two */
};

/* [host] 1 <= d <= 8192; eps > 0. */
typedef struct {
    int32_t T, d;
    int32_t x_dtype; /* strata_xdtype of x, r, dr, dx */
    int32_t y_dtype; /* of y, dy and a channel gate */
    int32_t u_dtype; /* of u, du */
    uint32_t flags;
    float resid_scale, branch_scale, eps;
} strata_block_norm_args;

/* x [T][d]; y [T][d], or NULL for no branch (r = resid_scale * x; then no
 * post norm and no gate); g_post, g_pre [d] fp32, NULL for gains of 1.
 * Outputs: r [T][d] (nullable; may be x), u [T][d] (required with
 * STRATA_PRE_NORM, else NULL), rstd_y and rstd_r [T] fp32 (nullable; what
 * the gradient needs).  T = 0: no-op.  EINVAL: a null required pointer, a
 * pointer that the flags give no meaning to, a misaligned one, a bad dtype,
 * unknown or contradictory flags, T < 0, d < 1, eps not a positive finite
 * number, a scale that is not finite; EUNSUPPORTED: d > 8192, T > 2^23; EHIP. */
strata_status strata_block_norm(const strata_block_norm_args *args, const void *x, const void *y, const void *gate,
                                const float *g_post, const float *g_pre, void *r, void *u, float *rstd_y,
                                float *rstd_r, void *stream);

/* Bytes of workspace the gradient needs; 0 for arguments it refuses. */
size_t strata_block_norm_backward_workspace_bytes(const strata_block_norm_args *args);

/* Gradient, from dr (of r, nullable: zeros) and du (of u; required with
 * STRATA_PRE_NORM, else NULL), with r (needed with STRATA_PRE_NORM), y, gate,
 * gains and both rstd as the forward call had or left them:
 *   dx [T][d], dy [T][d], dgate as the gate, dg_post and dg_pre [d] fp32,
 * each nullable.  dx may be dr.  T = 0 writes zeros to dg_post and dg_pre.
 * Errors as above, and EINVAL for an output without its input (dy, dgate,
 * dg_post without y; dg_post without STRATA_POST_NORM; dg_pre without
 * STRATA_PRE_NORM; rstd_y or rstd_r missing); EWORKSPACE. */
strata_status strata_block_norm_backward(const strata_block_norm_args *args, const void *dr, const void *du,
                                         const void *r, const void *y, const void *gate, const float *g_post,
                                         const float *g_pre, const float *rstd_y, const float *rstd_r, void *dx,
                                         void *dy, void *dgate, float *dg_post, float *dg_pre, void *ws,
                                         size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* STRATA_OPS_H */
