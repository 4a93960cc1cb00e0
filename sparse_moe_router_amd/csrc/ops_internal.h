// Declarations shared by the kernels and the host code of the operators in
// moe_ops.h (gfx950 only).
#pragma once

#include "moe_internal.h"
#include "moe_ops.h"

namespace moe {

typedef __attribute__((__vector_size__(4 * sizeof(int32_t)))) int32_t i32x4_t;
typedef __attribute__((__vector_size__(16 * sizeof(int32_t)))) int32_t i32x16_t;

constexpr int kOpTile = 256;              // tile edge of the matrix-matrix kernels
constexpr int64_t kOpMaxUnits = 1 << 22;  // output tiles of one launch (threads of a launch stay below 2^32)

// The rows of one grouped product, as the kernels take them.
struct Groups {
  int64_t rows, x_rows;
  int64_t ldx, ldy;  // elements
  int E, N, K, k;
  const int32_t* offsets;  // NULL: one group of all rows
  const int32_t* perm;     // NULL: row p of x
};

// Rows lo <= p < hi.
struct Range {
  int64_t lo, hi;
  __device__ __forceinline__ int64_t size() const { return hi - lo; }
};

// Rows a <= p < b, limited to [0, rows]; empty when the end is not above the start.
__device__ __forceinline__ Range limited(const Groups& g, int64_t a, int64_t b) {
  a = a < 0 ? 0 : a > g.rows ? g.rows : a;
  b = b < a ? a : b > g.rows ? g.rows : b;
  return Range{a, b};
}

// The rows of group e.
__device__ __forceinline__ Range group_range(const Groups& g, int e) {
  return g.offsets ? limited(g, g.offsets[e], g.offsets[e + 1]) : Range{0, g.rows};
}

// Row of x that row p of the grouped order reads; -1: none (a row of zeros).
__device__ __forceinline__ int64_t source_row(const Groups& g, int64_t p) {
  if (!g.perm) return p;
  const int32_t v = g.perm[p];
  if (v < 0) return -1;
  const int64_t t = (uint32_t)v / (uint32_t)g.k;
  return t < g.x_rows ? t : -1;
}

// Scales of the 8-bit products (NULL members: bf16 products).
struct Scales {
  const float* x;     // [x_rows]
  const float* w;     // [E][N]
  const float* bias;  // [N] or NULL
};

enum OpKind { OP_NT = 0, OP_NN = 1, OP_TN = 2 };

// Matrix-matrix kernels: y = x W^T, dx = dy W, dw = dy^T x.  i8: y from codes.
hipError_t launch_op_tile(OpKind kind, bool i8, const Groups& g, const void* a, const void* b, const Scales& sc,
                          void* out, bool fp32, hipStream_t s);
// Matrix-vector kernel for few rows an expert: y = x W^T.  quantize: x is bf16,
// w int8, and every workgroup quantises its rows itself.
hipError_t launch_op_skinny(bool i8, bool quantize, const Groups& g, const void* x, const void* w, const Scales& sc, void* y,
                            bool fp32, hipStream_t s);
hipError_t launch_quantize_i8(int64_t rows, int K, int64_t ldx, const uint16_t* x, int8_t* codes, float* scale,
                              hipStream_t s);

// Output tiles of a launch; 0 rows give 0.
int64_t op_tile_units(OpKind kind, const Groups& g);

// Gated products, g.N features of each of the two matrices: h (rows g.ldy apart) from x, and with
// pre the products themselves; by matrix-matrix tiles or for few rows.
hipError_t launch_gated(const Groups& g, const void* x, const void* w, void* h, void* pre, int64_t ldp, hipStream_t s);
hipError_t launch_gated_skinny(const Groups& g, const void* x, const void* w, void* h, void* pre, int64_t ldp,
                               hipStream_t s);
int64_t gated_units(const Groups& g);
// The gradients of a gated feed-forward block: of its rows and both weights, from d_pre and h.
struct FfnArgs {
  Groups g;  // of x and w_gate_up: N = 2 I
  int I, H;
  const void *dy, *x, *w_gate_up, *d_pre, *h;
  int64_t ld_dy, ld_dpre, ld_h;
  void *dx, *dw_gate_up, *dw_down;
  int64_t ld_dx;
  bool dw32;
};
// Parts that the reduction of each weight gradient is cut into, and their bytes of workspace.
int ffn_splits(const FfnArgs& a);
size_t ffn_split_bytes(const FfnArgs& a);
int64_t ffn_units(const FfnArgs& a);
hipError_t launch_ffn_products(const FfnArgs& a, float* part, hipStream_t s);
// The whole backward pass for few rows, d [rows][2 I] and h [rows][I] in fp32.
hipError_t launch_few_rows(const FfnArgs& a, const void* w_down, const void* pre, int64_t ldp, float* d, float* h,
                           hipStream_t s);
// dy W through the gate: d_pre and h of g.K features.
hipError_t launch_gated_grad(const Groups& g, const void* dy, const void* w, const void* pre, int64_t ldp, void* d_pre,
                             int64_t ldd, void* h, int64_t ldh, hipStream_t s);

// Block norms: the arguments as the kernels take them (d_* only in the gradients).
struct NormArgs {
  int64_t rows;
  int H;
  bool stream32, weight32;
  int gate_mode;
  float eps, scale;
  moe_mat_t residual, y, gate, out, h;
  moe_mat_t d_out, d_h, d_residual, d_y, d_gate;
  const void *weight, *next_weight;
  float *d_weight, *d_next_weight;
  float* part;  // [groups][2][H] partial sums of the weight gradients
};
hipError_t launch_norm_fwd(const NormArgs& a, bool merge, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, bool merge, hipStream_t s);
// Workgroups of the gradient kernel = partial sums of each weight gradient.
int norm_grad_groups(int64_t rows, int H);

// A token's sum over its grouped rows, and its gradients (d_* and dy only there).
struct CombineArgs {
  int64_t tokens, rows;
  int H, k, E;
  const int32_t *perm, *inverse, *offsets;
  const float* weight;  // [tokens][k] or NULL: ones
  moe_mat_t y, add, out;
  moe_mat_t d_out, dy;
  float* d_weight;
};
hipError_t launch_invert(const int32_t* perm, const int32_t* offsets, int E, int64_t rows, int32_t* inverse, int64_t n,
                         hipStream_t s);
hipError_t launch_combine(const CombineArgs& a, bool fp32, hipStream_t s);
hipError_t launch_combine_grad(const CombineArgs& a, hipStream_t s);

// Tensors of one launch over many gradients, cut into pieces; as kernel arguments (below 4 KB).
constexpr int kClipTensors = 120;
constexpr int kClipGroups = 2048;  // workgroups of a launch at most
constexpr int kClipParts = 2 * kClipGroups;  // sums of workgroups that each workgroup of the scaling adds itself
struct GradTable {
  const void* in[kClipTensors];
  void* out[kClipTensors];
  int64_t n[kClipTensors];
  int32_t first[kClipTensors];  // first piece
  uint32_t types[2][4];         // bit j: tensor j of in (0) or out (1) is fp32
  int32_t count;
  int32_t pieces;
  int32_t shift;                // elements of a piece: 2^shift
};
static_assert(kClipTensors <= 128 && sizeof(GradTable) < 3840, "kernel arguments");
int64_t clip_pieces(int64_t n, int shift);
int clip_shift(int64_t elements);  // of all tensors of a call
int clip_groups(int64_t pieces);
hipError_t launch_squares(const GradTable& t, double* part, hipStream_t s);
hipError_t launch_norm(const double* part, int parts, float* norm, hipStream_t s);
// part NULL: *norm is given; else it is the root of the parts' sum, and stored if store.
hipError_t launch_clip(const GradTable& t, const double* part, int parts, float* norm, float max_norm, float eps,
                       bool store, hipStream_t s);

// Softmax cross entropy against a vocabulary (lse, d_loss, dx and dw only in the gradient).
struct LossArgs {
  int64_t rows, ldx;
  int V, H;
  const void *x, *w;
  const int64_t* target;
  int64_t ignore;
  float *loss, *lse_out;
  const float *lse, *d_loss;
  void* dx;  // or NULL
  int64_t lddx;
  bool dx32, dw32;
  void* dw;  // or NULL
};
// The tokens as the kernels of the logits take them.
struct LossTokens {
  const int64_t* target;
  int64_t ignore;
  int V, v0;      // vocabulary; first column of the piece
  float2* part;   // forward: [panel][rows] maximum, sum of exp(z - maximum)
  float* hit;     // forward: [rows] z at the target
  const float *lse, *d_loss;  // gradient
  uint16_t* d;                // gradient: [rows][ldd]
  int64_t ldd;
};
// The logits of few tokens: 16 columns a workgroup and a panel.
constexpr int kSkinnyColumns = 16;
hipError_t launch_loss_skinny(const Groups& g, const void* x, const void* w, const LossTokens& loss, bool grad,
                              hipStream_t s);
// The gradient goes through the vocabulary in pieces whose d (bf16) takes at most kLossPieceBytes,
// but at least kLossPieceColumns columns; dx is summed in `slices` buffers, each over `slice` columns
// of a piece.
constexpr int64_t kLossPieceBytes = 256 << 20;
constexpr int kLossPieceColumns = 2048;
struct LossPlan {
  int piece, slice, slices;
  int splits;  // parts of the reduction of dw
  size_t d_bytes, part_bytes, x_bytes, dw_bytes, bytes;
};
LossPlan loss_plan(int64_t rows, int V, int H);
size_t loss_workspace(int64_t rows, int V);
hipError_t launch_loss(const LossArgs& a, void* workspace, hipStream_t s);
hipError_t launch_loss_grad(const LossArgs& a, void* workspace, hipStream_t s);

}  // namespace moe
