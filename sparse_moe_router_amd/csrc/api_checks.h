// Argument checks and error records shared by the C-ABI sources.
#pragma once

#include "moe_internal.h"
#include "moe_layer.h"

namespace moe {

// MOE_ERR_HIP, with e kept for moe_last_hip_error() of this thread.
moe_status_t hip_fail(hipError_t e);

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

// Byte ranges of one call's buffers.  Every output range must be disjoint
// from every input range and from every other output range.
struct Region {
  const void* p;
  size_t n;
};
struct Regions {
  Region in[8], out[12];
  int nin = 0, nout = 0;
  void input(const void* p, size_t n) {
    if (p && n) in[nin++] = Region{p, n};
  }
  void output(const void* p, size_t n) {
    if (p && n) out[nout++] = Region{p, n};
  }
  bool disjoint() const {
    for (int i = 0; i < nout; ++i) {
      for (int j = 0; j < nin; ++j)
        if (overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return false;
      for (int j = i + 1; j < nout; ++j)
        if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return false;
    }
    return true;
  }
};

}  // namespace moe
