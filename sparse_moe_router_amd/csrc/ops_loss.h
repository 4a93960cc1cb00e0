// Device code that the kernels of the cross entropy share.
#pragma once

#include "ops_internal.h"

namespace moe {
namespace {

// exp(x - m), 0 where both are -inf.
__device__ __forceinline__ float exp_from(float x, float m) { return x == -INFINITY ? 0.0f : __expf(x - m); }

// d_loss of a token, 0 without a target.
__device__ __forceinline__ float scale_of(const LossTokens& a, int64_t t) {
  const int64_t g = a.target[t];
  return g >= 0 && g < a.V && g != a.ignore ? a.d_loss[t] : 0.0f;
}

}  // namespace
}  // namespace moe
