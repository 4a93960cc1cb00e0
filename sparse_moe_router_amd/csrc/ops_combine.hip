// A token's sum over its grouped rows (gfx950, wave64):
//   inverse[perm[p]] = p
//   out[t] = add[t] + sum_s weight[t][s] y[inverse[t k + s]]
//   dy[p] = weight[perm[p]] d_out[perm[p] / k],  d_weight[t][s] = <d_out[t], y[inverse[t k + s]]>
// All are bound by HBM: each grouped row is read (and its gradient written) once,
// whole, 16 bytes a lane (4096 x 8 rows of 2048: 151 MB in 31 us = 4.8 TB/s; gradients of 4099 x 8 rows: 285 MB
// in 52 us = 5.5 TB/s; a copy reaches 4.97).  The inverse gives every sum its terms in a fixed order
// without atomics; only its own making uses one (the lowest of rows that name the
// same assignment, whatever order they come in).
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kMaxBlocks = 1 << 22;  // threads of a launch stay below 2^32

// rows in front of the end of the last group
__device__ __forceinline__ int64_t rows_end(int64_t rows, const int32_t* offsets, int E) {
  if (!offsets) return rows;
  const int64_t n = offsets[E];
  return n < 0 ? 0 : n < rows ? n : rows;
}

__global__ __launch_bounds__(256) void k_invert_fill(int32_t* inverse, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) inverse[i] = -1;
}

__global__ __launch_bounds__(256) void k_invert(const int32_t* perm, const int32_t* offsets, int E, int64_t rows,
                                                int32_t* inverse, int64_t n) {
  const int64_t end = rows_end(rows, offsets, E);
  for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < end; p += (int64_t)gridDim.x * 256) {
    const int32_t a = perm[p];
    if (a >= 0 && a < n) atomicMin((unsigned*)inverse + a, (unsigned)p);  // -1 is the largest
  }
}

__device__ __forceinline__ void unpack(u32x4_t q, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(q[j]);
    f[2 * j + 1] = bf16_hi(q[j]);
  }
}
__device__ __forceinline__ u32x4_t pack(const float (&f)[8]) {
  return u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// A thread takes eight columns of a token's row; rows of up to 1024 elements share a workgroup (WIDE, from
// 2048 on: one row, and the token's indexes and weights come by scalar loads: 4096 x 8 rows of 2048 36.2 ->
// 31.4 us, 4.8 TB/s).  Between the two a workgroup has one row and threads without columns.  4096 x 8 rows, other
// ones in each call but in part still cached: of 1024 elements 5.0 TB/s, 1032 3.6, 1536 5.0, 2040 4.5, 2048 5.6, 2056
// 5.3.  Eight grouped rows are in flight at a time.
template <class T>
__device__ __forceinline__ T read_uniform(const T* p, int64_t i) {
  return ((const __attribute__((address_space(4))) T*)p)[i];
}
template <bool F32, bool WIDE>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a) {
  const int chunks = a.H / 8, per = WIDE ? 1 : 256 / chunks;
  const int mine = WIDE ? 0 : (int)threadIdx.x / chunks, first = threadIdx.x - mine * chunks;
  if (mine >= per) return;
  for (int64_t t = (int64_t)blockIdx.x * per + mine; t < a.tokens; t += (int64_t)gridDim.x * per)
    for (int c = first; c < chunks; c += 256) {
      float v[8] = {};
      if (a.add.data) {
        if (F32) {
          const f32x4_t* q = (const f32x4_t*)((const float*)a.add.data + t * a.add.ld + 8 * c);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = q[j >> 2][j & 3];
        } else {
          unpack(*(const u32x4_t*)((const uint16_t*)a.add.data + t * a.add.ld + 8 * c), v);
        }
      }
      for (int s0 = 0; s0 < a.k; s0 += 8) {
        u32x4_t q[8];
        float w[8];
        bool in[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int64_t i = t * a.k + s0 + s;
          int64_t p = -1;
          if (s0 + s < a.k) p = WIDE ? read_uniform(a.inverse, i) : a.inverse[i];
          in[s] = p >= 0 && p < a.rows;
          w[s] = 1.0f;
          if (in[s] && a.weight) w[s] = WIDE ? read_uniform(a.weight, i) : a.weight[i];
          q[s] = u32x4_t{0, 0, 0, 0};
          if (in[s]) q[s] = *(const u32x4_t*)((const uint16_t*)a.y.data + p * a.y.ld + 8 * c);
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          float f[8];
          unpack(q[s], f);
          if (in[s])
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = fmaf(w[s], f[j], v[j]);
        }
      }
      if (F32) {
        f32x4_t* o = (f32x4_t*)((float*)a.out.data + t * a.out.ld + 8 * c);
        o[0] = f32x4_t{v[0], v[1], v[2], v[3]};
        o[1] = f32x4_t{v[4], v[5], v[6], v[7]};
      } else {
        *(u32x4_t*)((uint16_t*)a.out.data + t * a.out.ld + 8 * c) = pack(v);
      }
    }
}

// A workgroup of four waves takes a token, a wave one of its rows at a time; d_out's row comes from
// the caches after the first.  A workgroup also looks at k grouped rows of its own place: those that
// no assignment has become zeros.
constexpr int GW = 4;
__global__ __launch_bounds__(64 * GW) void k_combine_grad(CombineArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), chunks = a.H / 8;
  const int64_t end = rows_end(a.rows, a.offsets, a.E), n = a.tokens * a.k;
  const int64_t units = a.tokens > (a.rows + a.k - 1) / a.k ? a.tokens : (a.rows + a.k - 1) / a.k;
  for (int64_t t = blockIdx.x; t < units; t += gridDim.x) {
    for (int s = wave; s < a.k; s += GW) {
      const int64_t i = t * a.k + s;
      if (i < end) {
        const int64_t g = a.perm[i];
        if (g < 0 || g >= n || a.inverse[g] != i)
          for (int c = lane; c < chunks; c += 64)
            *(u32x4_t*)((uint16_t*)a.dy.data + i * a.dy.ld + 8 * c) = u32x4_t{0, 0, 0, 0};
      }
      if (t >= a.tokens) continue;
      const int64_t p = a.inverse[i];
      const bool has = p >= 0 && p < end && a.perm[p] == i;
      float dot = 0.0f;
      if (has) {
        const float w = a.weight ? a.weight[i] : 1.0f;
        const uint16_t* d = (const uint16_t*)a.d_out.data + t * a.d_out.ld;
        const uint16_t* y = a.weight ? (const uint16_t*)a.y.data + p * a.y.ld : d;
        uint16_t* dy = (uint16_t*)a.dy.data + p * a.dy.ld;
        for (int c0 = lane; c0 < chunks; c0 += 256) {
          u32x4_t qd[4], qy[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int c = c0 + 64 * u < chunks ? c0 + 64 * u : c0;
            qd[u] = *(const u32x4_t*)(d + 8 * c);
            qy[u] = *(const u32x4_t*)(y + 8 * c);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (c0 + 64 * u >= chunks) continue;
            float fd[8], fy[8];
            unpack(qd[u], fd);
            unpack(qy[u], fy);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              dot = fmaf(fd[j], fy[j], dot);
              fd[j] *= w;
            }
            *(u32x4_t*)(dy + 8 * (c0 + 64 * u)) = pack(fd);
          }
        }
      }
      if (a.d_weight) {
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) dot += __shfl_xor(dot, m, 64);
        if (lane == 0) a.d_weight[i] = dot;
      }
    }
  }
}

unsigned blocks(int64_t n) { return (unsigned)(n < 1 ? 1 : n < kMaxBlocks ? n : kMaxBlocks); }

}  // namespace

hipError_t launch_invert(const int32_t* perm, const int32_t* offsets, int E, int64_t rows, int32_t* inverse, int64_t n,
                         hipStream_t s) {
  const Launch lc{s, nullptr, nullptr};
  if (n == 0) return hipSuccess;
  const hipError_t e = launch(lc, k_invert_fill, dim3(blocks((n + 255) / 256)), dim3(256), inverse, n);
  if (e != hipSuccess || rows == 0) return e;
  return launch(lc, k_invert, dim3(blocks((rows + 255) / 256)), dim3(256), perm, offsets, E, rows, inverse, n);
}

hipError_t launch_combine(const CombineArgs& a, bool fp32, hipStream_t s) {
  const int chunks = a.H / 8, per = chunks < 256 ? 256 / chunks : 1;
  const bool wide = chunks >= 256;
  const dim3 grid(blocks((a.tokens + per - 1) / per));
  const Launch lc{s, nullptr, nullptr};
  if (fp32) return wide ? launch(lc, k_combine<true, true>, grid, dim3(256), a) : launch(lc, k_combine<true, false>, grid, dim3(256), a);
  return wide ? launch(lc, k_combine<false, true>, grid, dim3(256), a) : launch(lc, k_combine<false, false>, grid, dim3(256), a);
}

hipError_t launch_combine_grad(const CombineArgs& a, hipStream_t s) {
  const int64_t rows = (a.rows + a.k - 1) / a.k, units = a.tokens > rows ? a.tokens : rows;
  return launch(Launch{s, nullptr, nullptr}, k_combine_grad, dim3(blocks(units)), dim3(64 * GW), a);
}

}  // namespace moe
