// C ABI of the operators of a training step in moe_ops.h (gated products,
// combine, clipping, cross entropy): argument checks and launches on the
// caller's stream.  No device allocation, no host synchronisation, no state kept.
#include <math.h>

#include <algorithm>
#include <memory>
#include <new>

#include "ops_checks.h"
#include "ops_paths.h"

using namespace moe;

namespace {

// A matrix argument: rows of at least `cols` columns, chunks of 16 bytes.
moe_status_t check_mat(const moe_mat_t& m, int64_t cols) {
  if (!aligned(m.data, 16)) return MOE_ERR_MISALIGNED;
  if (m.ld < cols) return MOE_ERR_INVALID_ARG;
  if (m.ld > ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return m.ld % 8 ? MOE_ERR_MISALIGNED : MOE_OK;
}
Region mat_region(const moe_mat_t& m, int64_t rows, int64_t cols, moe_dtype_t t) {
  return matrix_at(m.data, rows, m.ld, cols, t == MOE_DT_FP32 ? 4 : 2);
}
moe_status_t status_of(hipError_t e) { return e == hipSuccess ? MOE_OK : hip_fail(e); }

// A feed-forward block on checked shapes, and its workspace.
struct Ffn {
  FfnArgs a;
  bool few;  // kernels for few rows, which keep d and h in fp32
  size_t d_pre_bytes, h_bytes, bytes;
};
moe_status_t check_ffn(const moe_feed_forward_t* d, Ffn* f) {
  if (!d) return MOE_ERR_INVALID_ARG;
  const moe_groups_t gu{d->rows, d->x_rows, d->ldx, 2 * (int64_t)std::max(d->I, 0), d->E, 2 * std::min(d->I, kMaxN), d->K,
                        d->top_k, d->offsets, d->perm};
  const moe_groups_t down{d->rows, d->rows, std::max<int64_t>(d->I, 0), d->ld_dy, d->E, d->H, d->I, 1, d->offsets, nullptr};
  Checked c, e;
  moe_status_t st = check_groups(&gu, 8, 8, &c);
  if (st == MOE_OK) st = check_groups(&down, 8, 8, &e);
  if (st == MOE_OK) st = check_x_rows(&gu);
  if (st != MOE_OK) return st;
  *f = Ffn{};
  f->a.g = c.g;
  f->a.I = d->I;
  f->a.H = d->H;
  f->a.ld_dy = d->ld_dy;
  f->a.ld_dpre = 2 * (int64_t)d->I;
  f->a.ld_h = d->I;
  if (op_tile_units(OP_NN, e.g) > kOpMaxUnits || ffn_units(f->a) > kOpMaxUnits) return MOE_ERR_UNSUPPORTED_SHAPE;
  f->few = takes_few_rows(d->rows, d->E, d->H, d->I, d->K);
  const size_t size = f->few ? 4 : 2;
  f->d_pre_bytes = ((size_t)d->rows * 2 * d->I * size + 255) & ~(size_t)255;
  f->h_bytes = ((size_t)d->rows * d->I * size + 255) & ~(size_t)255;
  f->bytes = f->d_pre_bytes + f->h_bytes + (f->few ? 0 : ffn_split_bytes(f->a));
  return MOE_OK;
}

moe_status_t check_combine(const moe_combine_t* d) {
  if (!d || d->tokens < 0 || d->rows < 0) return MOE_ERR_INVALID_ARG;
  if (d->H < 8 || d->H > kMaxK || d->H % 8 || d->top_k < 1 || d->top_k > kMaxTopK) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->rows > kMaxRows || d->tokens > kMaxRows || d->tokens * d->top_k > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!check_type(d->out_type)) return MOE_ERR_INVALID_ARG;
  if (!aligned(d->inverse, 4)) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}
CombineArgs combine_args(const moe_combine_t* d) {
  CombineArgs a{};
  a.tokens = d->tokens;
  a.rows = d->rows;
  a.H = d->H;
  a.k = d->top_k;
  a.E = d->E;
  a.perm = d->perm;
  a.inverse = d->inverse;
  a.offsets = d->offsets;
  return a;
}

size_t type_size(moe_dtype_t t) { return t == MOE_DT_FP32 ? 4 : 2; }

constexpr int64_t kMaxElements = (int64_t)1 << 40;  // of all tensors of a call
moe_status_t check_tensors(const moe_tensor_t* t, int32_t count, bool outs) {
  if (count < 0 || (count > 0 && !t)) return MOE_ERR_INVALID_ARG;
  int64_t elements = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || !check_type(t[i].in_type) || (outs && !check_type(t[i].out_type))) return MOE_ERR_INVALID_ARG;
    if (t[i].n > kMaxElements - elements) return MOE_ERR_UNSUPPORTED_SHAPE;
    elements += t[i].n;
    if (t[i].n == 0) continue;
    if (!t[i].in || (outs && !t[i].out)) return MOE_ERR_INVALID_ARG;
    if (!aligned(t[i].in, type_size(t[i].in_type)) || (outs && !aligned(t[i].out, type_size(t[i].out_type))))
      return MOE_ERR_MISALIGNED;
  }
  return MOE_OK;
}

constexpr int64_t kClipPieces = 1 << 30;  // of a launch
// Calls f(table) for the tensors, as many at a time as a launch takes.
template <class F>
moe_status_t each_table(const moe_tensor_t* t, int32_t count, bool outs, F&& f) {
  GradTable g;
  g.count = g.pieces = 0;
  auto reset = [&] {
    g.count = g.pieces = 0;
    for (auto& a : g.types)
      for (uint32_t& w : a) w = 0;
  };
  reset();
  int64_t elements = 0;
  for (int32_t i = 0; i < count; ++i) elements += t[i].n;
  g.shift = clip_shift(elements);
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const int64_t pieces = clip_pieces(t[i].n, g.shift);  // at most 2^25
    if (g.count == kClipTensors || g.pieces + pieces > kClipPieces) {
      const moe_status_t st = f(g);
      if (st != MOE_OK) return st;
      reset();
    }
    const int j = g.count++;
    g.in[j] = t[i].in;
    g.out[j] = outs ? t[i].out : nullptr;
    g.n[j] = t[i].n;
    g.first[j] = g.pieces;
    g.pieces += (int32_t)pieces;
    if (t[i].in_type == MOE_DT_FP32) g.types[0][j >> 5] |= 1u << (j & 31);
    if (outs && t[i].out_type == MOE_DT_FP32) g.types[1][j >> 5] |= 1u << (j & 31);
  }
  return g.count ? f(g) : MOE_OK;
}

// Bytes that a call over many tensors reads or writes.
struct Extent {
  uintptr_t lo, hi;
  bool out;
};
// Whether an output shares a byte with anything else.
bool overlapping(Extent* x, size_t n) {
  std::sort(x, x + n, [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
  uintptr_t any = 0, outs = 0;  // ends of what came before
  for (size_t i = 0; i < n; ++i) {
    if (x[i].lo < (x[i].out ? any : outs)) return true;
    any = std::max(any, x[i].hi);
    if (x[i].out) outs = std::max(outs, x[i].hi);
  }
  return false;
}
moe_status_t check_disjoint(const moe_tensor_t* t, int32_t count, bool outs, const float* norm, bool norm_out,
                            const void* workspace, size_t workspace_bytes) {
  Extent few[128];
  std::unique_ptr<Extent[]> many;
  Extent* x = few;
  if ((size_t)count * 2 + 2 > 128) {
    many.reset(new (std::nothrow) Extent[(size_t)count * 2 + 2]);
    if (!many) return hip_fail(hipErrorOutOfMemory);
    x = many.get();
  }
  size_t n = 0;
  auto add = [&](const void* p, size_t bytes, bool out) {
    if (p && bytes) x[n++] = Extent{(uintptr_t)p, (uintptr_t)p + bytes, out};
  };
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const bool in_place = outs && t[i].in == t[i].out && t[i].in_type == t[i].out_type;
    if (!in_place) add(t[i].in, (size_t)t[i].n * type_size(t[i].in_type), false);
    if (outs) add(t[i].out, (size_t)t[i].n * type_size(t[i].out_type), true);
  }
  add(norm, 4, norm_out);
  add(workspace, workspace_bytes, true);
  return overlapping(x, n) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

// Bytes of the parts of the sum of squares of checked tensors: each_table's launches.
size_t parts_bytes(const moe_tensor_t* t, int32_t count) {
  int64_t elements = 0, pieces = 0, parts = 0;
  for (int32_t i = 0; i < count; ++i) elements += t[i].n;
  const int shift = clip_shift(elements);
  int tensors = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const int64_t n = clip_pieces(t[i].n, shift);
    if (tensors == kClipTensors || pieces + n > kClipPieces) {
      parts += clip_groups(pieces);
      tensors = 0, pieces = 0;
    }
    ++tensors, pieces += n;
  }
  parts += clip_groups(pieces);
  return ((size_t)(parts > 0 ? parts : 1) * 8 + 255) & ~(size_t)255;
}

// The parts of the sum of squares into the workspace; their number.
moe_status_t run_squares(const moe_tensor_t* t, int32_t count, double* part, int* parts, hipStream_t s) {
  *parts = 0;
  return each_table(t, count, false, [&](const GradTable& g) {
    const hipError_t e = launch_squares(g, part + *parts, s);
    *parts += clip_groups(g.pieces);
    return status_of(e);
  });
}

moe_status_t check_norm_call(const float* norm, const void* workspace, size_t workspace_bytes, size_t need) {
  if (!norm || !workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned(norm, 4) || !aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
  return workspace_bytes < need ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

moe_status_t check_loss(const moe_loss_t* d) {
  if (!d || d->rows < 0) return MOE_ERR_INVALID_ARG;
  if (d->rows > kMaxRows || d->V < 1 || d->V > kMaxN || d->H < 8 || d->H > kMaxK || d->H % 8)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->ldx < d->H) return MOE_ERR_INVALID_ARG;
  if (d->ldx % 8) return MOE_ERR_MISALIGNED;
  if (d->ldx > kMaxLd) return MOE_ERR_UNSUPPORTED_SHAPE;
  // tiles of the logits and of dx
  const int64_t rows = (d->rows + kOpTile - 1) / kOpTile, cols = std::max(d->V, d->H) / kOpTile + 1;
  return rows * cols > kOpMaxUnits / 2 ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}
LossArgs loss_args(const moe_loss_t* d, const void* x, const void* w, const int64_t* target) {
  LossArgs a{};
  a.rows = d->rows;
  a.ldx = d->ldx;
  a.V = d->V;
  a.H = d->H;
  a.x = x;
  a.w = w;
  a.target = target;
  a.ignore = d->ignore_index;
  return a;
}
void loss_regions(Regions* r, const moe_loss_t* d, const void* x, const void* w, const int64_t* target) {
  r->input(matrix_at(x, d->rows, d->ldx, d->H, 2));
  r->input(w, (size_t)d->V * d->H * 2);
  r->input(target, (size_t)d->rows * 8);
}

}  // namespace

extern "C" {

moe_status_t moe_gated_matmul(const moe_groups_t* d, const void* x, const void* w, void* h, moe_mat_t gate_up,
                              hipStream_t stream) {
  Checked c;
  moe_status_t st = check_groups(d, 8, 8, &c);
  if (st == MOE_OK) st = check_x_rows(d);
  if (st != MOE_OK) return st;
  if (gated_units(c.g) > kOpMaxUnits) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->rows == 0) return MOE_OK;
  if (!w || !h || (!x && d->x_rows > 0)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({x, w, h})) return MOE_ERR_MISALIGNED;
  if (gate_up.data && (st = check_mat(gate_up, 2 * (int64_t)d->N)) != MOE_OK) return st;
  Regions r;
  r.input(matrix_at(x, d->x_rows, d->ldx, d->K, 2));
  r.input(w, c.w_elems * 4);
  group_regions(&r, c.g);
  r.output(matrix_at(h, d->rows, d->ldy, d->N, 2));
  r.output(mat_region(gate_up, d->rows, 2 * (int64_t)d->N, MOE_DT_BF16));
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  // the rule of the products, for the rows of both matrices
  return status_of(takes_matrix_vector(d->rows, d->E, 2 * d->N)
                       ? launch_gated_skinny(c.g, x, w, h, gate_up.data, gate_up.ld, stream)
                       : launch_gated(c.g, x, w, h, gate_up.data, gate_up.ld, stream));
}

moe_status_t moe_gated_matmul_grad(const moe_groups_t* d, const void* dy, const void* w, moe_mat_t gate_up,
                                   moe_mat_t d_gate_up, void* h, hipStream_t stream) {
  Checked c;
  moe_status_t st = check_groups(d, 8, 8, &c);
  if (st != MOE_OK) return st;
  if (op_tile_units(OP_NN, c.g) > kOpMaxUnits) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->rows == 0) return MOE_OK;
  if (!dy || !w || !gate_up.data || !d_gate_up.data || !h) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({dy, w, h})) return MOE_ERR_MISALIGNED;
  const int64_t cols = 2 * (int64_t)d->K;
  if ((st = check_mat(gate_up, cols)) != MOE_OK || (st = check_mat(d_gate_up, cols)) != MOE_OK) return st;
  c.g.perm = nullptr;
  Regions r;
  r.input(matrix_at(dy, d->rows, d->ldy, d->N, 2));
  r.input(w, c.w_elems * 2);
  group_regions(&r, c.g);
  r.input(mat_region(gate_up, d->rows, cols, MOE_DT_BF16));
  r.output(mat_region(d_gate_up, d->rows, cols, MOE_DT_BF16));
  r.output(matrix_at(h, d->rows, d->ldx, d->K, 2));
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  return status_of(launch_gated_grad(c.g, dy, w, gate_up.data, gate_up.ld, d_gate_up.data, d_gate_up.ld, h, d->ldx,
                                     stream));
}

size_t moe_feed_forward_grad_workspace_size(const moe_feed_forward_t* d) {
  Ffn f;
  return check_ffn(d, &f) == MOE_OK ? f.bytes : 0;
}

moe_status_t moe_feed_forward_grad(const moe_feed_forward_t* d, const void* dy, const void* x, const void* w_gate_up,
                                   const void* w_down, moe_mat_t gate_up, moe_mat_t dx, void* dw_gate_up, void* dw_down,
                                   moe_dtype_t dw_type, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  Ffn f;
  moe_status_t st = check_ffn(d, &f);
  if (st != MOE_OK) return st;
  if (!check_type(dw_type)) return MOE_ERR_INVALID_ARG;
  if (!w_gate_up || !w_down || !dw_gate_up || !dw_down) return MOE_ERR_INVALID_ARG;
  if (d->rows > 0 && (!dy || !gate_up.data || !dx.data || !workspace || (!x && d->x_rows > 0))) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({dy, x, w_gate_up, w_down, dw_gate_up, dw_down}) || !aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
  const int64_t cols = 2 * (int64_t)d->I;
  if (d->rows > 0 && ((st = check_mat(gate_up, cols)) != MOE_OK || (st = check_mat(dx, d->K)) != MOE_OK)) return st;
  if (dx.ld > kMaxLd) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->rows > 0 && workspace_bytes < f.bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const size_t gu = (size_t)d->E * cols * d->K, down = (size_t)d->E * d->H * d->I;
  Regions r;
  r.input(matrix_at(dy, d->rows, d->ld_dy, d->H, 2));
  r.input(matrix_at(x, d->x_rows, d->ldx, d->K, 2));
  r.input(w_gate_up, gu * 2);
  r.input(w_down, down * 2);
  r.input(mat_region(gate_up, d->rows, cols, MOE_DT_BF16));
  group_regions(&r, f.a.g);
  r.output(mat_region(dx, d->rows, d->K, MOE_DT_BF16));
  r.output(dw_gate_up, gu * type_size(dw_type));
  r.output(dw_down, down * type_size(dw_type));
  r.output(workspace, d->rows > 0 ? f.bytes : 0);
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  // workspace: d_pre, h, parts of the weight gradients
  char* const d_pre = (char*)workspace;
  char* const h = d_pre + f.d_pre_bytes;
  if (d->rows > 0 && !f.few) {
    Groups g = f.a.g;  // of the down projection
    g.N = d->H;
    g.K = d->I;
    g.ldy = d->ld_dy;
    g.perm = nullptr;
    st = status_of(launch_gated_grad(g, dy, w_down, gate_up.data, gate_up.ld, d_pre, cols, h, d->I, stream));
    if (st != MOE_OK) return st;
  }
  FfnArgs a = f.a;
  a.dy = dy;
  a.x = x;
  a.w_gate_up = w_gate_up;
  a.d_pre = d_pre;
  a.h = h;
  a.dx = dx.data;
  a.ld_dx = dx.ld;
  a.dw_gate_up = dw_gate_up;
  a.dw_down = dw_down;
  a.dw32 = dw_type == MOE_DT_FP32;
  if (f.few) return status_of(launch_few_rows(a, w_down, gate_up.data, gate_up.ld, (float*)d_pre, (float*)h, stream));
  return status_of(launch_ffn_products(a, (float*)(h + f.h_bytes), stream));
}

moe_status_t moe_invert_permutation(int64_t rows, const int32_t* perm, const int32_t* offsets, int32_t E, int64_t n,
                                    int32_t* inverse, hipStream_t stream) {
  if (rows < 0 || n < 0) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows || n > kMaxRows || (offsets && (E < 1 || E > kMaxE))) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (n == 0) return MOE_OK;
  if (!inverse || (rows > 0 && !perm)) return MOE_ERR_INVALID_ARG;
  if (!aligned(perm, 4) || !aligned(offsets, 4) || !aligned(inverse, 4)) return MOE_ERR_MISALIGNED;
  Regions r;
  r.input(perm, (size_t)rows * 4);
  r.input(offsets, (size_t)(E + 1) * 4);
  r.output(inverse, (size_t)n * 4);
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  return status_of(launch_invert(perm, offsets, E, rows, inverse, n, stream));
}

moe_status_t moe_combine(const moe_combine_t* d, moe_mat_t y, const float* weight, moe_mat_t add, moe_mat_t out,
                         hipStream_t stream) {
  moe_status_t st = check_combine(d);
  if (st != MOE_OK) return st;
  if (d->tokens == 0) return MOE_OK;
  if (!d->inverse || !out.data || (!y.data && d->rows > 0)) return MOE_ERR_INVALID_ARG;
  if (!aligned(weight, 4)) return MOE_ERR_MISALIGNED;
  for (const moe_mat_t* m : {&y, &add, &out})
    if (m->data && (st = check_mat(*m, d->H)) != MOE_OK) return st;
  Regions r;
  r.input(mat_region(y, d->rows, d->H, MOE_DT_BF16));
  r.input(d->inverse, (size_t)d->tokens * d->top_k * 4);
  r.input(weight, (size_t)d->tokens * d->top_k * 4);
  r.input(mat_region(add, d->tokens, d->H, d->out_type));
  r.output(mat_region(out, d->tokens, d->H, d->out_type));
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  CombineArgs a = combine_args(d);
  a.y = y;
  a.weight = weight;
  a.add = add;
  a.out = out;
  return status_of(launch_combine(a, d->out_type == MOE_DT_FP32, stream));
}

moe_status_t moe_combine_grad(const moe_combine_t* d, moe_mat_t d_out, moe_mat_t y, const float* weight, moe_mat_t dy,
                              float* d_weight, hipStream_t stream) {
  moe_status_t st = check_combine(d);
  if (st != MOE_OK) return st;
  if (d->offsets && (d->E < 1 || d->E > kMaxE)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d_weight && !weight) return MOE_ERR_INVALID_ARG;
  if (d->tokens == 0 && d->rows == 0) return MOE_OK;
  if (d->tokens > 0 && (!d->inverse || !d_out.data)) return MOE_ERR_INVALID_ARG;
  if (d->rows > 0 && (!d->perm || !dy.data || (weight && !y.data))) return MOE_ERR_INVALID_ARG;
  if (!aligned(weight, 4) || !aligned(d_weight, 4) || !aligned(d->perm, 4) || !aligned(d->offsets, 4))
    return MOE_ERR_MISALIGNED;
  if (!weight) y = moe_mat_t{nullptr, 0};
  for (const moe_mat_t* m : {&d_out, &y, &dy})
    if (m->data && (st = check_mat(*m, d->H)) != MOE_OK) return st;
  const size_t n = (size_t)d->tokens * d->top_k * 4;
  Regions r;
  r.input(mat_region(d_out, d->tokens, d->H, MOE_DT_BF16));
  r.input(mat_region(y, d->rows, d->H, MOE_DT_BF16));
  r.input(d->inverse, n);
  r.input(d->perm, (size_t)d->rows * 4);
  r.input(d->offsets, d->offsets ? (size_t)(d->E + 1) * 4 : 0);
  r.input(weight, n);
  r.output(mat_region(dy, d->rows, d->H, MOE_DT_BF16));
  r.output(d_weight, n);
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  CombineArgs a = combine_args(d);
  a.d_out = d_out;
  a.y = y;
  a.weight = weight;
  a.dy = dy;
  a.d_weight = d_weight;
  return status_of(launch_combine_grad(a, stream));
}

size_t moe_grad_norm_workspace_size(const moe_tensor_t* t, int32_t count) {
  return check_tensors(t, count, false) == MOE_OK ? parts_bytes(t, count) : 0;
}

moe_status_t moe_grad_norm(const moe_tensor_t* t, int32_t count, float* norm, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  moe_status_t st = check_tensors(t, count, false);
  if (st != MOE_OK) return st;
  const size_t need = parts_bytes(t, count);
  st = check_norm_call(norm, workspace, workspace_bytes, need);
  if (st == MOE_OK) st = check_disjoint(t, count, false, norm, true, workspace, need);
  if (st != MOE_OK) return st;
  int parts;
  st = run_squares(t, count, (double*)workspace, &parts, stream);
  return st != MOE_OK ? st : status_of(launch_norm((const double*)workspace, parts, norm, stream));
}

moe_status_t moe_clip_grads(const moe_tensor_t* t, int32_t count, float max_norm, float eps, float* norm,
                            int32_t norm_given, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  moe_status_t st = check_tensors(t, count, true);
  if (st != MOE_OK) return st;
  if (!(max_norm >= 0.0f) || !isfinite(max_norm) || !(eps > 0.0f) || !isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (norm_given) {
    if (!norm) return MOE_ERR_INVALID_ARG;
    if (!aligned(norm, 4)) return MOE_ERR_MISALIGNED;
    workspace = nullptr;
  }
  const size_t need = norm_given ? 0 : parts_bytes(t, count);
  if (!norm_given && (st = check_norm_call(norm, workspace, workspace_bytes, need)) != MOE_OK) return st;
  st = check_disjoint(t, count, true, norm, !norm_given, workspace, need);
  if (st != MOE_OK) return st;
  int parts = 0;
  if (!norm_given) {
    st = run_squares(t, count, (double*)workspace, &parts, stream);
    if (st != MOE_OK) return st;
  }
  const double* part = (const double*)workspace;
  if (!norm_given && (parts == 0 || parts > kClipParts)) {  // no elements, or more parts than each workgroup adds
    st = status_of(launch_norm(part, parts, norm, stream));
    if (st != MOE_OK || parts == 0) return st;
    part = nullptr;
  }
  bool store = true;
  return each_table(t, count, true, [&](const GradTable& g) {
    const hipError_t e = launch_clip(g, part, parts, norm, max_norm, eps, store, stream);
    store = false;
    return status_of(e);
  });
}

size_t moe_cross_entropy_workspace_size(const moe_loss_t* d) {
  return check_loss(d) == MOE_OK ? loss_workspace(d->rows, d->V) : 0;
}

moe_status_t moe_cross_entropy(const moe_loss_t* d, const void* x, const void* w, const int64_t* target, float* loss,
                               float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const moe_status_t st = check_loss(d);
  if (st != MOE_OK) return st;
  if (d->rows == 0) return MOE_OK;
  if (!x || !w || !target || !loss || !workspace) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({x, w}) || !aligned(target, 8) || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(workspace, 256))
    return MOE_ERR_MISALIGNED;
  const size_t need = loss_workspace(d->rows, d->V);
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  Regions r;
  loss_regions(&r, d, x, w, target);
  r.output(loss, (size_t)d->rows * 4);
  r.output(lse, (size_t)d->rows * 4);
  r.output(workspace, need);
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  LossArgs a = loss_args(d, x, w, target);
  a.loss = loss;
  a.lse_out = lse;
  return status_of(launch_loss(a, workspace, stream));
}

size_t moe_cross_entropy_grad_workspace_size(const moe_loss_t* d) {
  return check_loss(d) == MOE_OK ? loss_plan(d->rows, d->V, d->H).bytes : 0;
}

moe_status_t moe_cross_entropy_grad(const moe_loss_t* d, const float* d_loss, const void* x, const void* w,
                                    const int64_t* target, const float* lse, moe_mat_t dx, moe_dtype_t dx_type, void* dw,
                                    moe_dtype_t dw_type, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  moe_status_t st = check_loss(d);
  if (st != MOE_OK) return st;
  if (!check_type(dx_type) || !check_type(dw_type)) return MOE_ERR_INVALID_ARG;
  if (d->rows == 0 && !dw) return MOE_OK;
  if (!dx.data && !dw) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({x, w, dw}) || !aligned(target, 8) || !aligned(lse, 4) || !aligned(d_loss, 4) ||
      !aligned(workspace, 256))
    return MOE_ERR_MISALIGNED;
  if (dx.data && (st = check_mat(dx, d->H)) != MOE_OK) return st;
  if (d->rows > 0 && (!x || !w || !target || !lse || !d_loss || !workspace)) return MOE_ERR_INVALID_ARG;
  const size_t need = loss_plan(d->rows, d->V, d->H).bytes;
  if (d->rows > 0 && workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  Regions r;
  loss_regions(&r, d, x, w, target);
  r.input(lse, (size_t)d->rows * 4);
  r.input(d_loss, (size_t)d->rows * 4);
  r.output(mat_region(dx, d->rows, d->H, dx_type));
  r.output(dw, (size_t)d->V * d->H * type_size(dw_type));
  r.output(workspace, d->rows > 0 ? need : 0);
  if (!r.disjoint()) return MOE_ERR_INVALID_ARG;
  LossArgs a = loss_args(d, x, w, target);
  a.lse = lse;
  a.d_loss = d_loss;
  a.dx = dx.data;
  a.lddx = dx.ld;
  a.dx32 = dx_type == MOE_DT_FP32;
  a.dw = dw;
  a.dw32 = dw_type == MOE_DT_FP32;
  return status_of(launch_loss_grad(a, workspace, stream));
}

}  // extern "C"
