/*
 * moe_ops.h -- operators around the sparse MoE layer of moe_layer.h, for
 * models that train their experts, serve them in 8 bits or build the
 * transformer block around the layer (AMD Instinct MI355X, gfx950).
 *
 *   grouped products   y[p] = x[row(p)] . W_e^T for the rows p of each expert's
 *                      group (ragged sizes), and the gradients of that product
 *   8-bit products     tokens quantised to int8 with one scale a token, weights
 *                      int8 with one scale a channel, exact int32 sums; dense or
 *                      grouped by expert
 *   block norms        RMSNorm before a block; RMSNorm after it fused with its
 *                      gate, the residual scale, the residual sum and the next
 *                      block's norm; and their gradients
 *   gated products     h = silu(x G^T) * (x U^T) grouped by expert in one kernel,
 *                      and the gradient through it and the projection behind it
 *   combine            a token's weighted sum over its grouped rows, and its
 *                      gradients
 *   clipping           the norm over all gradients of a model, and their scaling
 *   cross entropy      the loss of tokens against a vocabulary from hidden states
 *                      and vocabulary weights, without keeping the logits, and
 *                      its gradients
 *
 * The conventions of moe_layer.h hold for every entry point: device pointers
 * owned by the caller and 16-byte aligned (workspaces 256-byte), nothing
 * allocated, no state between calls, asynchronous on `stream`, arguments
 * checked before anything is enqueued, outputs and workspaces disjoint from
 * every input and from each other (element by element where both are column
 * slices with rows the same number of bytes apart, else as whole extents).  Work runs on the current device: make the
 * stream's device current.  A call with no rows returns MOE_OK without reading
 * its input rows; gradients of weights are then written as zeros.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ grouped products */

/* Rows grouped by expert.  `offsets` are the group offsets and `perm` the
 * permutation that moe_route reports: rows offsets[e] <= p < offsets[e+1] of
 * the grouped order belong to expert e, and row p reads row perm[p] / top_k of
 * x (the token of that assignment).  Without perm, row p reads row p of x.
 * Both are device data that the host does not see; the kernels stay in bounds
 * for any contents: offsets are limited to [0, rows], an expert whose end is
 * not above its start is empty, and a perm entry outside [0, x_rows * top_k)
 * stands for a row of zeros.  Rows p >= offsets[E] of an output are left as
 * they were. */
typedef struct {
  int64_t rows;           /* rows of the grouped order (of y, dy and dx) */
  int64_t x_rows;         /* rows of x; without perm >= rows */
  int64_t ldx;            /* elements from a row of x (or dx) to the next: >= K */
  int64_t ldy;            /* elements from a row of y (or dy) to the next: >= N */
  int32_t E;              /* experts, 1 .. 1024 */
  int32_t N;              /* rows of a weight matrix = output features */
  int32_t K;              /* columns of a weight matrix = input features */
  int32_t top_k;          /* assignments per token, 1 .. 32; not used without perm */
  const int32_t* offsets; /* [E+1]; NULL with E == 1: all rows belong to it */
  const int32_t* perm;    /* [rows] or NULL */
} moe_groups_t;

/* Element types of outputs that have a choice. */
typedef enum { MOE_DT_BF16 = 0, MOE_DT_FP32 = 1 } moe_dtype_t;

/* Shapes of the bf16 products: N and K multiples of 8, 8 <= N <= 2^20,
 * 8 <= K <= 16384, ldx and ldy multiples of 8 and at most 2^20, rows and
 * x_rows < 2^31, and at most 2^22 output tiles of 256 x 256.  Products accumulate in fp32 and
 * are rounded once to the output's type. */

/* y[p][n] = sum_k x[row(p)][k] w[e][n][k].  x bf16 [x_rows][ldx], w bf16
 * [E][N][K], y bf16 or fp32 [rows][ldy]. */
moe_status_t moe_grouped_matmul(const moe_groups_t* g, const void* x, const void* w, void* y, moe_dtype_t y_type,
                                hipStream_t stream);

/* dx[p][k] = sum_n dy[p][n] w[e][n][k]: the gradient of the grouped rows (of
 * the copies that row(p) took: a token's own gradient is the sum over its
 * assignments).  dy bf16 [rows][ldy], w as above, dx bf16 or fp32
 * [rows][ldx].  perm, top_k and x_rows are not used, but have to be within their ranges. */
moe_status_t moe_grouped_matmul_grad_input(const moe_groups_t* g, const void* dy, const void* w, void* dx,
                                           moe_dtype_t dx_type, hipStream_t stream);

/* dw[e][n][k] = sum_p dy[p][n] x[row(p)][k] over the expert's rows, in a fixed
 * order; zeros for an expert without rows.  dw bf16 or fp32 [E][N][K]. */
moe_status_t moe_grouped_matmul_grad_weight(const moe_groups_t* g, const void* x, const void* dy, void* dw,
                                            moe_dtype_t dw_type, hipStream_t stream);

/* ------------------------------------------------------------ 8-bit products */

/* codes[t][k] = rint(127 x[t][k] / max|x[t]|), half to even, in [-127, 127],
 * and scale[t] = max|x[t]| / 127.  A row of zeros has codes and scale 0; a row
 * that holds an infinity or NaN has codes 0 and that infinity or NaN as scale,
 * so that products of the row are NaN.  x bf16 [rows][ldx], codes int8
 * [rows][K], scale fp32 [rows].  K a multiple of 16, 16 <= K <= 16384, ldx a
 * multiple of 8. */
moe_status_t moe_quantize_i8(int64_t rows, int32_t K, int64_t ldx, const void* x, void* codes, float* scale,
                             hipStream_t stream);

/* y[p][n] = (sum_k q[row(p)][k] w[e][n][k]) * (x_scale[row(p)] * w_scale[e][n])
 *           + bias[n].
 * The sum is exact in int32; the rest is fp32, rounded once to y's type.
 *   x        bf16 [x_rows][ldx] with x_scale NULL: quantised by the call as
 *            moe_quantize_i8 does; or int8 codes [x_rows][ldx] with x_scale
 *            fp32 [x_rows]
 *   w        int8 [E][N][K], w_scale fp32 [E][N]
 *   bias     fp32 [N], or NULL; only with E == 1
 *   y        bf16 or fp32 [rows][ldy]
 * Shapes: N a multiple of 8, K a multiple of 16, ldx a multiple of 8 (codes:
 * 16), ldy a multiple of 8, the other limits as for the bf16 products.
 * workspace: moe_matmul_i8_workspace_size bytes (0 for a few bf16 rows, and not
 * used with codes), 256-byte aligned; calls sharing one must be ordered. */
size_t moe_matmul_i8_workspace_size(const moe_groups_t* g);
moe_status_t moe_matmul_i8(const moe_groups_t* g, const void* x, const float* x_scale, const void* w,
                           const float* w_scale, const float* bias, void* y, moe_dtype_t y_type, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------ block norms */

/* How a block's output is gated: by nothing, by one value a token (gate
 * [rows]) or by one value an element (gate [rows][H]). */
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_TOKEN = 1, MOE_GATE_ELEMENT = 2 } moe_gate_t;

/* Shapes and types of the norms: H a multiple of 8, 8 <= H <= 16384.  The
 * residual stream (residual, out and their gradients) is bf16 or fp32; h, y,
 * the gate and their gradients are bf16; norm weights are bf16 or fp32 [H],
 * all of one call of the same type; gradients of weights are fp32 [H].
 * Statistics are fp32, so that a row's sum of squares has to stay below fp32's
 * largest value (elements up to 1e17 do at every H); each result is rounded once
 * to its type. */
typedef struct {
  int64_t rows;            /* tokens, < 2^31 */
  int32_t H;
  moe_dtype_t stream_type; /* residual stream */
  moe_dtype_t weight_type; /* norm weights */
  moe_gate_t gate_mode;
  float eps;               /* added to the mean square; > 0, finite */
  float scale;             /* residual scale of the block's output; finite */
} moe_norm_t;

/* A [rows][H] matrix: its first element and the elements from a row to the
 * next, a multiple of 8 and >= H.  data NULL: the argument is not given.  A
 * token gate and its gradient are vectors [rows]; their ld is not used. */
typedef struct {
  void* data;
  int64_t ld;
} moe_mat_t;

/* h = x * rsqrt(mean(x^2) + eps) * weight, the norm before a block.  x in the
 * stream's type, h bf16. */
moe_status_t moe_block_norm(const moe_norm_t* d, moe_mat_t x, const void* weight, moe_mat_t h, hipStream_t stream);

/* Its gradients: dx = d_add + (gradient through the norm), with d_add the
 * gradient that reaches x beside the norm (or not given), and d_weight. */
moe_status_t moe_block_norm_grad(const moe_norm_t* d, moe_mat_t d_h, moe_mat_t x, const void* weight, moe_mat_t d_add,
                                 moe_mat_t dx, float* d_weight, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* out = residual + scale * sigmoid(gate) * y * rsqrt(mean(y^2) + eps) * weight,
 * the norm after a block, its gate and the residual sum; with next_weight
 * also h = out * rsqrt(mean(out^2) + eps) * next_weight of the stored out, the
 * norm before the next block (next_weight and h both given, or neither). */
moe_status_t moe_block_merge(const moe_norm_t* d, moe_mat_t residual, moe_mat_t y, const void* weight, moe_mat_t gate,
                             const void* next_weight, moe_mat_t out, moe_mat_t h, hipStream_t stream);

/* Gradients of every input of moe_block_merge, from d_out (of out; not given =
 * 0) and d_h (of h; not given without a next norm; at least one of the two),
 * with the forward call's y, weight, gate and, for d_h, its out and
 * next_weight.
 *   d_residual, d_y, d_gate (shape of gate; not given without one), d_weight
 *   and d_next_weight (fp32 [H]; d_next_weight NULL without d_h). */
moe_status_t moe_block_merge_grad(const moe_norm_t* d, moe_mat_t d_out, moe_mat_t d_h, moe_mat_t y, const void* weight,
                                  moe_mat_t gate, moe_mat_t out, const void* next_weight, moe_mat_t d_residual,
                                  moe_mat_t d_y, moe_mat_t d_gate, float* d_weight, float* d_next_weight,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace of the two gradient calls (partial sums of the weight gradients);
 * 0 when the arguments are invalid. */
size_t moe_norm_grad_workspace_size(const moe_norm_t* d);

/* ------------------------------------------------------------ gated products */

/* g[p] = x[row(p)] . G_e^T, u[p] = x[row(p)] . U_e^T, h[p] = silu(g[p]) * u[p],
 * silu(z) = z / (1 + exp(-z)): the two input projections of a gated
 * feed-forward block with the activation and the product.  The groups as for
 * moe_grouped_matmul with N the features of each of the two matrices:
 *   x        bf16 [x_rows][ldx]
 *   w        bf16 [E][2 N][K]: G_e, then U_e
 *   h        bf16 [rows][ldy]
 *   gate_up  not given, or bf16 [rows][ld] of 2 N columns: g, then u, rounded,
 *            for the backward pass */
moe_status_t moe_gated_matmul(const moe_groups_t* g, const void* x, const void* w, void* h, moe_mat_t gate_up,
                              hipStream_t stream);

/* The gradient through y[p] = h[p] . W_e^T and the gate, in one kernel:
 *   dh[p] = dy[p] . W_e,  s = 1 / (1 + exp(-g)),
 *   d_gate_up = (dh u s (1 + g (1 - s)), dh g s),  h = g s u
 * with g and u as gate_up holds them, and h again for the gradient of W.  dh is
 * not rounded on the way.  N are the columns of dy, K the features:
 *   dy         bf16 [rows][ldy]
 *   w          bf16 [E][N][K]
 *   gate_up, d_gate_up  bf16 [rows][ld] of 2 K columns
 *   h          bf16 [rows][ldx]
 * perm, top_k and x_rows are not used, but have to be within their ranges. */
moe_status_t moe_gated_matmul_grad(const moe_groups_t* g, const void* dy, const void* w, moe_mat_t gate_up,
                                   moe_mat_t d_gate_up, void* h, hipStream_t stream);

/* A gated feed-forward block: y[p] = h[p] . D_e^T of H columns with h of I features from
 * moe_gated_matmul.  K, H and I multiples of 8, K and I at most 16384, 2 I and H at most
 * 2^20; the other fields as in moe_groups_t. */
typedef struct {
  int64_t rows, x_rows;
  int64_t ldx;            /* of x */
  int64_t ld_dy;          /* of dy, >= H */
  int32_t E, I, K, H;
  int32_t top_k;
  const int32_t* offsets;
  const int32_t* perm;
} moe_feed_forward_t;

/* Its gradients from dy, with moe_gated_matmul_grad's d_gate_up and h:
 *   dx = d_gate_up . W_e (of each grouped row, as moe_grouped_matmul_grad_input),
 *   dw_gate_up = d_gate_up^T x[row(p)],  dw_down = dy^T h (as ..._grad_weight).
 * dy bf16 [rows][ld_dy], x bf16 [x_rows][ldx], w_gate_up bf16 [E][2 I][K], w_down bf16
 * [E][H][I], gate_up bf16 [rows][ld] of 2 I columns as the forward call kept it, dx bf16
 * [rows][ld], dw_gate_up and dw_down in dw_type, of the weights' shapes.  workspace:
 * moe_feed_forward_grad_workspace_size bytes, which hold d_gate_up, h and, where few experts have
 * long groups, parts of the weight gradients.  d_gate_up and h are operands of the matrix units
 * and so rounded to bf16, as where they are tensors between calls: the gradients are off by 0.17%
 * of their norm before their own rounding, another 0.17% in bf16 (both: 0.23%).  Calls of at most
 * 32 rows in which rows times weights, and experts times weights, are at most 2^28 keep them in fp32. */
size_t moe_feed_forward_grad_workspace_size(const moe_feed_forward_t* d);
moe_status_t moe_feed_forward_grad(const moe_feed_forward_t* d, const void* dy, const void* x, const void* w_gate_up,
                                   const void* w_down, moe_mat_t gate_up, moe_mat_t dx, void* dw_gate_up, void* dw_down,
                                   moe_dtype_t dw_type, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------ combine */

/* inverse[a] = the row p with perm[p] == a, the lowest of several, for the
 * assignments 0 <= a < n; -1 where no row has it.  Rows from the end of the last
 * group on (offsets[E], when offsets are given; E is else not used) and entries of
 * perm outside [0, n) count for nothing.  perm int32 [rows], inverse int32 [n];
 * rows, n < 2^31, E 1 .. 1024. */
moe_status_t moe_invert_permutation(int64_t rows, const int32_t* perm, const int32_t* offsets, int32_t E, int64_t n,
                                    int32_t* inverse, hipStream_t stream);

/* Tokens and the grouped rows of their assignments.  H a multiple of 8, 8 <= H <=
 * 16384; top_k 1 .. 32; tokens * top_k < 2^31. */
typedef struct {
  int64_t tokens;
  int64_t rows;           /* grouped rows */
  int32_t H;
  int32_t top_k;
  int32_t E;              /* with offsets: 1 .. 1024 */
  moe_dtype_t out_type;   /* of out and add */
  const int32_t* inverse; /* [tokens * top_k]: as moe_invert_permutation gives it; entries outside [0, rows) have no row */
  const int32_t* perm;    /* [rows]; gradient only */
  const int32_t* offsets; /* [E+1] or NULL: all rows; gradient only */
} moe_combine_t;

/* out[t] = add[t] + sum_s weight[t][s] y[inverse[t * top_k + s]], in the order of
 * s in fp32, rounded once; an assignment without a row adds nothing, whatever its
 * weight.  y bf16 [rows][ld], weight fp32 [tokens][top_k] or NULL (ones), add
 * [tokens][ld] in out's type or not given, out bf16 or fp32 [tokens][ld]. */
moe_status_t moe_combine(const moe_combine_t* d, moe_mat_t y, const float* weight, moe_mat_t add, moe_mat_t out,
                         hipStream_t stream);

/* Its gradients: dy[p] = weight[t][s] d_out[t] for the row p of assignment (t, s),
 * zeros for a row in front of offsets[E] that no assignment has, rows behind it
 * left as they were; d_weight[t][s] = <d_out[t], y[p]>, 0 for an assignment without
 * a row.  d_out and y bf16, dy bf16 [rows][ld], d_weight fp32 [tokens][top_k].
 * Without weight, y is not read and d_weight is NULL; with it d_weight may be
 * NULL. */
moe_status_t moe_combine_grad(const moe_combine_t* d, moe_mat_t d_out, moe_mat_t y, const float* weight, moe_mat_t dy,
                              float* d_weight, hipStream_t stream);

/* ------------------------------------------------------------ clipping */

/* One of many gradients: n elements in a row, aligned as their type only; at most 2^40
 * elements in all tensors of a call. */
typedef struct {
  const void* in;
  void* out;              /* moe_clip_grads only; in place: out == in of the same type */
  int64_t n;              /* >= 0; the addresses of a tensor without elements are not used */
  moe_dtype_t in_type;
  moe_dtype_t out_type;
} moe_tensor_t;

/* *norm = sqrt(sum over all elements of all tensors of in^2), fp32.  The sum is of
 * 64 bits and repeats bit for bit; an infinity or NaN among the elements gives one.
 * The addresses are read from `tensors` (host memory) during the call.  workspace:
 * moe_grad_norm_workspace_size bytes (0 when the arguments are invalid). */
size_t moe_grad_norm_workspace_size(const moe_tensor_t* tensors, int32_t count);
moe_status_t moe_grad_norm(const moe_tensor_t* tensors, int32_t count, float* norm, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* out = in * min(1, max_norm / (norm + eps)), rounded once; in place nothing is
 * written where that factor is 1.  norm_given = 0: *norm is computed and written
 * first, as above; else it is read (of gradients that other devices hold too, say)
 * and the workspace is not used.  max_norm >= 0, eps > 0, both finite.  An infinite norm scales
 * to 0, a NaN to NaN. */
moe_status_t moe_clip_grads(const moe_tensor_t* tensors, int32_t count, float max_norm, float eps, float* norm,
                            int32_t norm_given, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------ cross entropy */

/* Tokens against a vocabulary: 1 <= V <= 2^20, H a multiple of 8, 8 <= H <= 16384,
 * ldx a multiple of 8, H <= ldx <= 2^20, rows < 2^31, and at most 2^21 tiles of
 * 256 x 256 in a matrix of as many rows and of V, or of H, columns.  A token whose target is ignore_index or lies outside
 * [0, V) has no target: its loss is 0 and it has no part in the gradients. */
typedef struct {
  int64_t rows;           /* tokens */
  int64_t ldx;            /* elements from a row of x to the next */
  int32_t V;
  int32_t H;
  int64_t ignore_index;
} moe_loss_t;

/* z = x[t] . w^T in fp32, lse[t] = log(sum_v exp(z[v])), loss[t] = lse[t] -
 * z[target[t]].  x bf16 [rows][ldx], w bf16 [V][H], target int64 [rows], loss and
 * lse fp32 [rows] (lse may be NULL).  workspace:
 * moe_cross_entropy_workspace_size bytes. */
size_t moe_cross_entropy_workspace_size(const moe_loss_t* d);
moe_status_t moe_cross_entropy(const moe_loss_t* d, const void* x, const void* w, const int64_t* target, float* loss,
                               float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* dz[t][v] = exp(z[t][v] - lse[t]) - (v == target[t]), rounded to bf16; dx[t] =
 * d_loss[t] sum_v dz[t][v] w[v], dw[v] = m sum_t dz[t][v] r[t] with m the d_loss
 * of largest magnitude of the tokens that have a target and r[t] = x[t] d_loss[t] / m, rounded to bf16.  lse as the forward call
 * gave it, d_loss fp32 [rows]; dx bf16 or fp32 [rows][ld] or not given, dw bf16 or
 * fp32 [V][H] or NULL.  The vocabulary goes by in pieces; the workspace
 * (moe_cross_entropy_grad_workspace_size bytes) holds one piece's dz (at most 256 MB, or 4 KB a
 * token above 65536 tokens), one to 32 sums of dx in fp32, r, and where a vocabulary is small
 * parts of dw.  Either gradient is the same, bit for bit, with and without the other. */
size_t moe_cross_entropy_grad_workspace_size(const moe_loss_t* d);
moe_status_t moe_cross_entropy_grad(const moe_loss_t* d, const float* d_loss, const void* x, const void* w,
                                    const int64_t* target, const float* lse, moe_mat_t dx, moe_dtype_t dx_type, void* dw,
                                    moe_dtype_t dw_type, void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
