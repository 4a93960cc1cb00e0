// out = the sum of `parts` arrays of n fp32 values, one after the other, in their
// order, times *factor if given.
#pragma once

#include "ops_internal.h"

namespace moe {
namespace {

__global__ __launch_bounds__(256) void k_sum_parts(const float* part, int parts, int64_t n, const float* factor, void* out,
                                                   int fp32) {
  const float f = factor ? *factor : 1.0f;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
    float v[8] = {};
    for (int s = 0; s < parts; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t q = *(const f32x4_t*)(part + s * n + i + 4 * h);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * h + k] += q[k];
      }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= f;
    if (fp32) {
      *(f32x4_t*)((float*)out + i) = f32x4_t{v[0], v[1], v[2], v[3]};
      *(f32x4_t*)((float*)out + i + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
      *(u32x4_t*)((uint16_t*)out + i) = u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
  }
}

// n a multiple of 8
inline hipError_t launch_sum_parts(const float* part, int parts, int64_t n, const float* factor, void* out, bool fp32,
                                   hipStream_t s) {
  const int64_t groups = (n / 8 + 255) / 256;
  return launch(Launch{s, nullptr, nullptr}, k_sum_parts, dim3((unsigned)(groups < 8192 ? groups : 8192)), dim3(256), part,
                parts, n, factor, out, (int)fp32);
}

}  // namespace
}  // namespace moe
