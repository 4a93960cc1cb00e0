// Argument checks shared by the operators' C-ABI sources.
#pragma once

#include <initializer_list>

#include "api_checks.h"
#include "ops_internal.h"

namespace moe {

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int kMaxN = 1 << 20, kMaxK = 16384;
constexpr int64_t kMaxLd = 1 << 20;  // 256 rows stay within the range of a buffer descriptor

struct Checked {
  Groups g;
  size_t w_elems;
};

// Shapes of a grouped product.  x_unit: elements that K and ldx are multiples
// of (16 bytes of x).
inline moe_status_t check_groups(const moe_groups_t* d, int k_unit, int ldx_unit, Checked* c) {
  if (!d || d->rows < 0 || d->x_rows < 0) return MOE_ERR_INVALID_ARG;
  if (d->rows > kMaxRows || d->x_rows > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->E < 1 || d->E > kMaxE) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->N < 8 || d->N > kMaxN || d->N % 8) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->K < k_unit || d->K > kMaxK || d->K % k_unit) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->top_k < 1 || d->top_k > kMaxTopK) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->ldx < d->K || d->ldy < d->N) return MOE_ERR_INVALID_ARG;
  if (d->ldx % ldx_unit || d->ldy % 8) return MOE_ERR_MISALIGNED;
  if (d->ldx > kMaxLd || d->ldy > kMaxLd) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!d->offsets && d->E != 1) return MOE_ERR_INVALID_ARG;
  if (!aligned(d->offsets, 4) || !aligned(d->perm, 4)) return MOE_ERR_MISALIGNED;
  c->g = Groups{d->rows, d->x_rows, d->ldx, d->ldy, d->E, d->N, d->K, d->top_k, d->offsets, d->perm};
  c->w_elems = (size_t)d->E * d->N * d->K;
  return MOE_OK;
}

// Rows of x that a product with gathered rows reads.
inline moe_status_t check_x_rows(const moe_groups_t* d) {
  if (!d->perm && d->x_rows < d->rows) return MOE_ERR_INVALID_ARG;
  if (d->perm && d->x_rows * d->top_k > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

inline void group_regions(Regions* r, const Groups& g) {
  r->input(g.offsets, (size_t)(g.E + 1) * 4);
  r->input(g.perm, (size_t)g.rows * 4);
}

inline bool check_type(moe_dtype_t t) { return t == MOE_DT_BF16 || t == MOE_DT_FP32; }

inline bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 16)) return false;
  return true;
}

}  // namespace moe
