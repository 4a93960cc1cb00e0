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
 * [rows][ldx].  perm, top_k and x_rows are not used. */
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

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
