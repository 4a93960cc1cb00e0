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

}  // namespace moe
