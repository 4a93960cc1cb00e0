// out = the sum of `parts` arrays of n fp32 values, one after the other, in their
// order, times *factor if given; up to two results in a launch.  Bound by the
// parts' bytes, most of which are still in the last-level cache.
#pragma once

#include "ops_internal.h"

namespace moe {
namespace {

struct SumOf {
  const float* part;
  int64_t n;  // a multiple of 8
  void* out;
};
struct SumArgs {
  SumOf of[2];
  int parts, fp32;
  const float* factor;
  unsigned groups;  // workgroups of the first
};

__global__ __launch_bounds__(256) void k_sum_parts(SumArgs a) {
  const bool second = blockIdx.x >= a.groups;
  const SumOf s = a.of[second];
  const int64_t group = blockIdx.x - (second ? a.groups : 0), groups = second ? gridDim.x - a.groups : a.groups;
  const float f = a.factor ? *a.factor : 1.0f;
  for (int64_t i = (group * 256 + threadIdx.x) * 8; i < s.n; i += groups * 256 * 8) {
    float v[8] = {};
    for (int p = 0; p < a.parts; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t q = *(const f32x4_t*)(s.part + p * s.n + i + 4 * h);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * h + k] += q[k];
      }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= f;
    if (a.fp32) {
      *(f32x4_t*)((float*)s.out + i) = f32x4_t{v[0], v[1], v[2], v[3]};
      *(f32x4_t*)((float*)s.out + i + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
      *(u32x4_t*)((uint16_t*)s.out + i) = u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
  }
}

// b.n 0: one result
inline hipError_t launch_sum_parts(int parts, const SumOf& a, const SumOf& b, const float* factor, bool fp32, hipStream_t s) {
  auto groups = [](int64_t n) {
    const int64_t g = (n / 8 + 255) / 256;
    return (unsigned)(g < 8192 ? g : 8192);
  };
  const SumArgs args{{a, b}, parts, (int)fp32, factor, groups(a.n)};
  return launch(Launch{s, nullptr, nullptr}, k_sum_parts, dim3(groups(a.n) + groups(b.n)), dim3(256), args);
}

}  // namespace
}  // namespace moe
