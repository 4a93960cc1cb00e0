// C ABI of the operators in moe_ops.h: argument checks and launches on the
// caller's stream.  No allocation, no host synchronisation, no state kept.
#include <math.h>

#include "ops_checks.h"
#include "ops_paths.h"

using namespace moe;

namespace {

bool skinny(const Groups& g) { return takes_matrix_vector(g.rows, g.E, g.N); }
bool quantize_inside(const Groups& g) { return quantizes_inside(g.rows, g.x_rows, g.E, g.N, g.K); }

// The forward product of either kind on checked arguments.
moe_status_t run_forward(bool i8, const Groups& g, const void* x, const void* w, const Scales& sc, void* y, bool fp32,
                         hipStream_t s) {
  const hipError_t e = skinny(g) ? launch_op_skinny(i8, false, g, x, w, sc, y, fp32, s)
                                 : launch_op_tile(OP_NT, i8, g, x, w, sc, y, fp32, s);
  return e == hipSuccess ? MOE_OK : hip_fail(e);
}

moe_status_t run_tile(OpKind kind, const Groups& g, const void* a, const void* b, void* out, bool fp32, hipStream_t s) {
  const hipError_t e = launch_op_tile(kind, false, g, a, b, Scales{}, out, fp32, s);
  return e == hipSuccess ? MOE_OK : hip_fail(e);
}

size_t codes_bytes(const moe_groups_t* d) { return ((size_t)d->x_rows * d->K + 255) & ~(size_t)255; }

moe_status_t check_norm(const moe_norm_t* d) {
  if (!d || d->rows < 0) return MOE_ERR_INVALID_ARG;
  if (d->rows > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->H < 8 || d->H > kMaxK || d->H % 8) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!check_type(d->stream_type) || !check_type(d->weight_type)) return MOE_ERR_INVALID_ARG;
  if (d->gate_mode != MOE_GATE_NONE && d->gate_mode != MOE_GATE_TOKEN && d->gate_mode != MOE_GATE_ELEMENT)
    return MOE_ERR_INVALID_ARG;
  if (!(d->eps > 0.0f) || !isfinite(d->eps) || !isfinite(d->scale)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

NormArgs norm_args(const moe_norm_t* d) {
  NormArgs a{};
  a.rows = d->rows;
  a.H = d->H;
  a.stream32 = d->stream_type == MOE_DT_FP32;
  a.weight32 = d->weight_type == MOE_DT_FP32;
  a.gate_mode = d->gate_mode;
  a.eps = d->eps;
  a.scale = d->scale;
  return a;
}

// Checks a norm call's buffers one by one and collects their ranges.
struct NormBuffers {
  const moe_norm_t* d;
  Regions r;
  moe_status_t st = MOE_OK;
  enum Kind { STREAM, ACT, GATE };
  Region check(const moe_mat_t& m, Kind k) {
    if (!m.data) return bytes_at(nullptr, 0);
    if (!aligned(m.data, 16)) fail(MOE_ERR_MISALIGNED);
    if (k == GATE && d->gate_mode == MOE_GATE_TOKEN) return bytes_at(m.data, (size_t)d->rows * 2);
    if (m.ld < d->H) fail(MOE_ERR_INVALID_ARG);
    if (m.ld > ((int64_t)1 << 31)) fail(MOE_ERR_UNSUPPORTED_SHAPE);
    if (m.ld % 8) fail(MOE_ERR_MISALIGNED);
    return matrix_at(m.data, d->rows, m.ld, d->H, k == STREAM && d->stream_type == MOE_DT_FP32 ? 4 : 2);
  }
  void fail(moe_status_t s) {
    if (st == MOE_OK) st = s;
  }
  void in(const moe_mat_t& m, Kind k) { r.input(check(m, k)); }
  void out(const moe_mat_t& m, Kind k) { r.output(check(m, k)); }
  void weight(const void* w) {
    if (!aligned(w, 16)) fail(MOE_ERR_MISALIGNED);
    r.input(w, (size_t)d->H * (d->weight_type == MOE_DT_FP32 ? 4 : 2));
  }
  void d_weight(const void* w) {
    if (!aligned(w, 16)) fail(MOE_ERR_MISALIGNED);
    r.output(w, (size_t)d->H * 4);
  }
  void workspace(const void* w, size_t have) {
    const size_t need = moe_norm_grad_workspace_size(d);
    if (!aligned(w, 256)) fail(MOE_ERR_MISALIGNED);
    if (have < need) fail(MOE_ERR_WORKSPACE_TOO_SMALL);
    r.output(w, need);
  }
  moe_status_t done() {
    if (st == MOE_OK && !r.disjoint()) st = MOE_ERR_INVALID_ARG;
    return st;
  }
};

}  // namespace

extern "C" {

moe_status_t moe_grouped_matmul(const moe_groups_t* d, const void* x, const void* w, void* y, moe_dtype_t y_type,
                                hipStream_t stream) {
  Checked c;
  moe_status_t st = check_groups(d, 8, 8, &c);
  if (st == MOE_OK) st = check_x_rows(d);
  if (st != MOE_OK) return st;
  if (!check_type(y_type)) return MOE_ERR_INVALID_ARG;
  if (op_tile_units(OP_NT, c.g) > kOpMaxUnits) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->rows == 0) return MOE_OK;
  if (!w || !y || (!x && d->x_rows > 0)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({x, w, y})) return MOE_ERR_MISALIGNED;
  const bool f32 = y_type == MOE_DT_FP32;
  Regions r;
  r.input(matrix_at(x, d->x_rows, d->ldx, d->K, 2));
  r.input(w, c.w_elems * 2);
  group_regions(&r, c.g);
  r.output(matrix_at(y, d->rows, d->ldy, d->N, f32 ? 4 : 2));
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  return run_forward(false, c.g, x, w, Scales{}, y, f32, stream);
}

moe_status_t moe_grouped_matmul_grad_input(const moe_groups_t* d, const void* dy, const void* w, void* dx,
                                           moe_dtype_t dx_type, hipStream_t stream) {
  Checked c;
  const moe_status_t st = check_groups(d, 8, 8, &c);
  if (st != MOE_OK) return st;
  if (!check_type(dx_type)) return MOE_ERR_INVALID_ARG;
  if (op_tile_units(OP_NN, c.g) > kOpMaxUnits) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->rows == 0) return MOE_OK;
  if (!dy || !w || !dx) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({dy, w, dx})) return MOE_ERR_MISALIGNED;
  const bool f32 = dx_type == MOE_DT_FP32;
  c.g.perm = nullptr;
  Regions r;
  r.input(matrix_at(dy, d->rows, d->ldy, d->N, 2));
  r.input(w, c.w_elems * 2);
  group_regions(&r, c.g);
  r.output(matrix_at(dx, d->rows, d->ldx, d->K, f32 ? 4 : 2));
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  return run_tile(OP_NN, c.g, dy, w, dx, f32, stream);
}

moe_status_t moe_grouped_matmul_grad_weight(const moe_groups_t* d, const void* x, const void* dy, void* dw,
                                            moe_dtype_t dw_type, hipStream_t stream) {
  Checked c;
  moe_status_t st = check_groups(d, 8, 8, &c);
  if (st == MOE_OK) st = check_x_rows(d);
  if (st != MOE_OK) return st;
  if (!check_type(dw_type)) return MOE_ERR_INVALID_ARG;
  if (op_tile_units(OP_TN, c.g) > kOpMaxUnits) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dw || (d->rows > 0 && (!dy || (!x && d->x_rows > 0)))) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({x, dy, dw})) return MOE_ERR_MISALIGNED;
  const bool f32 = dw_type == MOE_DT_FP32;
  Regions r;
  r.input(matrix_at(x, d->x_rows, d->ldx, d->K, 2));
  r.input(matrix_at(dy, d->rows, d->ldy, d->N, 2));
  group_regions(&r, c.g);
  r.output(dw, c.w_elems * (f32 ? 4 : 2));
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  return run_tile(OP_TN, c.g, dy, x, dw, f32, stream);
}

moe_status_t moe_quantize_i8(int64_t rows, int32_t K, int64_t ldx, const void* x, void* codes, float* scale,
                             hipStream_t stream) {
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows || K < 16 || K > kMaxK || K % 16) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (ldx < K) return MOE_ERR_INVALID_ARG;
  if (ldx > ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (ldx % 8) return MOE_ERR_MISALIGNED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scale) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({x, codes, scale})) return MOE_ERR_MISALIGNED;
  Regions r;
  r.input(matrix_at(x, rows, ldx, K, 2));
  r.output(codes, (size_t)rows * K);
  r.output(scale, (size_t)rows * 4);
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  const hipError_t e = launch_quantize_i8(rows, K, ldx, (const uint16_t*)x, (int8_t*)codes, scale, stream);
  return e == hipSuccess ? MOE_OK : hip_fail(e);
}

size_t moe_matmul_i8_workspace_size(const moe_groups_t* d) {
  Checked c;
  if (check_groups(d, 16, 8, &c) != MOE_OK || check_x_rows(d) != MOE_OK || quantize_inside(c.g)) return 0;
  return codes_bytes(d) + (((size_t)d->x_rows * 4 + 255) & ~(size_t)255);
}

moe_status_t moe_matmul_i8(const moe_groups_t* d, const void* x, const float* x_scale, const void* w,
                           const float* w_scale, const float* bias, void* y, moe_dtype_t y_type, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  Checked c;
  moe_status_t st = check_groups(d, 16, x_scale ? 16 : 8, &c);
  if (st == MOE_OK) st = check_x_rows(d);
  if (st != MOE_OK) return st;
  if (!check_type(y_type) || (bias && d->E != 1)) return MOE_ERR_INVALID_ARG;
  if (op_tile_units(OP_NT, c.g) > kOpMaxUnits) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->rows == 0) return MOE_OK;
  if (!w || !w_scale || !y || (!x && d->x_rows > 0)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({x, x_scale, w, w_scale, bias, y})) return MOE_ERR_MISALIGNED;
  const bool f32 = y_type == MOE_DT_FP32;
  Regions r;
  r.input(matrix_at(x, d->x_rows, d->ldx, d->K, x_scale ? 1 : 2));
  r.input(x_scale, (size_t)d->x_rows * 4);
  r.input(w, c.w_elems);
  r.input(w_scale, (size_t)d->E * d->N * 4);
  r.input(bias, (size_t)d->N * 4);
  group_regions(&r, c.g);
  r.output(matrix_at(y, d->rows, d->ldy, d->N, f32 ? 4 : 2));
  Scales sc{x_scale, w_scale, bias};
  if (!x_scale) {
    const size_t need = moe_matmul_i8_workspace_size(d);
    if (need > 0 && !workspace) return MOE_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    r.output(workspace, need);
  }
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  if (!x_scale && quantize_inside(c.g)) {
    const hipError_t e = launch_op_skinny(true, true, c.g, x, w, sc, y, f32, stream);
    return e == hipSuccess ? MOE_OK : hip_fail(e);
  }
  if (!x_scale) {
    float* scale = (float*)((char*)workspace + codes_bytes(d));
    if (d->x_rows > 0) {
      const hipError_t e =
          launch_quantize_i8(d->x_rows, d->K, d->ldx, (const uint16_t*)x, (int8_t*)workspace, scale, stream);
      if (e != hipSuccess) return hip_fail(e);
    }
    x = workspace;
    sc.x = scale;
    c.g.ldx = d->K;
  }
  return run_forward(true, c.g, x, w, sc, y, f32, stream);
}

moe_status_t moe_block_norm(const moe_norm_t* d, moe_mat_t x, const void* weight, moe_mat_t h, hipStream_t stream) {
  const moe_status_t st = check_norm(d);
  if (st != MOE_OK) return st;
  if (d->gate_mode != MOE_GATE_NONE) return MOE_ERR_INVALID_ARG;
  if (d->rows == 0) return MOE_OK;
  if (!x.data || !weight || !h.data) return MOE_ERR_INVALID_ARG;
  NormBuffers b{d};
  b.in(x, b.STREAM);
  b.weight(weight);
  b.out(h, b.ACT);
  if (b.done() != MOE_OK) return b.st;
  NormArgs a = norm_args(d);
  a.residual = x;
  a.weight = weight;
  a.h = h;
  const hipError_t e = launch_norm_fwd(a, false, stream);
  return e == hipSuccess ? MOE_OK : hip_fail(e);
}

size_t moe_norm_grad_workspace_size(const moe_norm_t* d) {
  if (check_norm(d) != MOE_OK) return 0;
  const size_t n = (size_t)norm_grad_groups(d->rows, d->H);
  return (n > 0 ? n : 1) * 2 * d->H * 4;
}

moe_status_t moe_block_norm_grad(const moe_norm_t* d, moe_mat_t d_h, moe_mat_t x, const void* weight, moe_mat_t d_add,
                                 moe_mat_t dx, float* d_weight, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  const moe_status_t st = check_norm(d);
  if (st != MOE_OK) return st;
  if (d->gate_mode != MOE_GATE_NONE) return MOE_ERR_INVALID_ARG;
  if (!weight || !d_weight || !workspace) return MOE_ERR_INVALID_ARG;
  if (d->rows > 0 && (!d_h.data || !x.data || !dx.data)) return MOE_ERR_INVALID_ARG;
  NormBuffers b{d};
  b.in(d_h, b.ACT);
  b.in(x, b.STREAM);
  b.weight(weight);
  b.in(d_add, b.STREAM);
  b.out(dx, b.STREAM);
  b.d_weight(d_weight);
  b.workspace(workspace, workspace_bytes);
  if (b.done() != MOE_OK) return b.st;
  NormArgs a = norm_args(d);
  a.d_h = d_h;
  a.out = x;
  a.weight = weight;
  a.d_out = d_add;
  a.d_residual = dx;
  a.d_weight = d_weight;
  a.part = (float*)workspace;
  const hipError_t e = launch_norm_bwd(a, false, stream);
  return e == hipSuccess ? MOE_OK : hip_fail(e);
}

moe_status_t moe_block_merge(const moe_norm_t* d, moe_mat_t residual, moe_mat_t y, const void* weight, moe_mat_t gate,
                             const void* next_weight, moe_mat_t out, moe_mat_t h, hipStream_t stream) {
  const moe_status_t st = check_norm(d);
  if (st != MOE_OK) return st;
  if (d->rows == 0) return MOE_OK;
  if (!residual.data || !y.data || !weight || !out.data) return MOE_ERR_INVALID_ARG;
  if ((next_weight == nullptr) != (h.data == nullptr)) return MOE_ERR_INVALID_ARG;
  if ((d->gate_mode == MOE_GATE_NONE) != (gate.data == nullptr)) return MOE_ERR_INVALID_ARG;
  NormBuffers b{d};
  b.in(residual, b.STREAM);
  b.in(y, b.ACT);
  b.weight(weight);
  b.in(gate, b.GATE);
  b.weight(next_weight);
  b.out(out, b.STREAM);
  b.out(h, b.ACT);
  if (b.done() != MOE_OK) return b.st;
  NormArgs a = norm_args(d);
  a.residual = residual;
  a.y = y;
  a.weight = weight;
  a.gate = gate;
  a.next_weight = next_weight;
  a.out = out;
  a.h = h;
  const hipError_t e = launch_norm_fwd(a, true, stream);
  return e == hipSuccess ? MOE_OK : hip_fail(e);
}

moe_status_t moe_block_merge_grad(const moe_norm_t* d, moe_mat_t d_out, moe_mat_t d_h, moe_mat_t y, const void* weight,
                                  moe_mat_t gate, moe_mat_t out, const void* next_weight, moe_mat_t d_residual,
                                  moe_mat_t d_y, moe_mat_t d_gate, float* d_weight, float* d_next_weight,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const moe_status_t st = check_norm(d);
  if (st != MOE_OK) return st;
  const bool next = next_weight != nullptr, gated = d->gate_mode != MOE_GATE_NONE;
  if (!weight || !d_weight || !workspace || next != (d_next_weight != nullptr)) return MOE_ERR_INVALID_ARG;
  if (d->rows > 0) {
    if (!y.data || !d_residual.data || !d_y.data) return MOE_ERR_INVALID_ARG;
    if (next != (d_h.data != nullptr) || (next ? !out.data : !d_out.data)) return MOE_ERR_INVALID_ARG;
    if (gated != (gate.data != nullptr) || gated != (d_gate.data != nullptr)) return MOE_ERR_INVALID_ARG;
  }
  if (!next) out = moe_mat_t{nullptr, 0};  // not read
  NormBuffers b{d};
  b.in(d_out, b.STREAM);
  b.in(d_h, b.ACT);
  b.in(y, b.ACT);
  b.weight(weight);
  b.in(gate, b.GATE);
  b.in(out, b.STREAM);
  b.weight(next_weight);
  b.out(d_residual, b.STREAM);
  b.out(d_y, b.ACT);
  b.out(d_gate, b.GATE);
  b.d_weight(d_weight);
  b.d_weight(d_next_weight);
  b.workspace(workspace, workspace_bytes);
  if (b.done() != MOE_OK) return b.st;
  NormArgs a = norm_args(d);
  a.d_out = d_out;
  a.d_h = d_h;
  a.y = y;
  a.weight = weight;
  a.gate = gate;
  a.out = out;
  a.next_weight = next_weight;
  a.d_residual = d_residual;
  a.d_y = d_y;
  a.d_gate = d_gate;
  a.d_weight = d_weight;
  a.d_next_weight = d_next_weight;
  a.part = (float*)workspace;
  const hipError_t e = launch_norm_bwd(a, true, stream);
  return e == hipSuccess ? MOE_OK : hip_fail(e);
}

}  // extern "C"
