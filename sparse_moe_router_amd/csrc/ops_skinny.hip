// y = x W^T for few rows an expert (gfx950, wave64): the decode and
// small-batch form of the grouped and 8-bit products, bound by the stream of
// the weights.
//
// A four-wave workgroup takes 16 rows of one expert's weights and all rows of
// the expert's group, 16, 32 or 64 at a time.  The waves split the reduction,
// each in runs of 1 KB of every weight row, straight from global memory into
// the MFMA operands (16x16 blocks: lane l holds 16 bytes of row l % 16),
// sixteen weight loads in flight a wave; the four partial sums meet in LDS and
// are added in wave order.  The weights are read once for each 64 rows of a group
// (once in all for most calls: the host gives it at most 256 rows), and so with
// the non-temporal hint; the few activation rows come from the caches.  Tokens in
// bf16 for int8 weights are quantised by every workgroup for itself while its
// first weights are on their way, when they are few: a launch of its own and
// its results' way through memory cost more.
#include <type_traits>

#include "ops_internal.h"
#include "ops_paths.h"
#include "quantize8.h"

namespace moe {
namespace {

constexpr int SN = 16;  // weight rows of a workgroup
constexpr int SW = 4;   // waves
constexpr int SUN = 16;  // 64-byte steps of a wave's run
constexpr int QR = kInsideRows;  // rows quantised at a time by a workgroup

__device__ __align__(16) const uint32_t kZero[4] = {0, 0, 0, 0};

struct SkinnyArgs {
  Groups g;
  const char* x;
  const char* w;
  Scales sc;
  void* y;
  int fp32;
  int by_row;  // workgroup row = row of the grouped order (else the expert)
};

// The codes and scales of up to QR rows into LDS (rows at a stride of K + 16
// bytes), by the whole workgroup: the arithmetic of moe_quantize_i8.
__device__ __forceinline__ void quantize_rows(const SkinnyArgs& p, int64_t p0, int rows, int8_t* codes, float* scale,
                                              uint32_t* maxima) {
  const Groups& g = p.g;
  const int tid = threadIdx.x, nc = g.K / 8;
  const uint16_t* src[QR];
  uint32_t m[QR];
#pragma unroll
  for (int r = 0; r < QR; ++r) {
    const int64_t t = r < rows ? source_row(g, p0 + r) : -1;
    src[r] = t < 0 ? nullptr : (const uint16_t*)p.x + t * g.ldx;
    m[r] = 0;
  }
  for (int c = tid; c < nc; c += 64 * SW)
#pragma unroll
    for (int r = 0; r < QR; ++r)
      if (src[r]) {
        const uint32_t o = max_magnitude(*(const u32x4_t*)(src[r] + 8 * c));
        m[r] = m[r] > o ? m[r] : o;
      }
#pragma unroll
  for (int r = 0; r < QR; ++r) {
    if (r >= rows) break;  // uniform
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      const uint32_t o = __shfl_xor(m[r], d, 64);
      m[r] = m[r] > o ? m[r] : o;
    }
    if ((tid & 63) == 0) maxima[(tid >> 6) * QR + r] = m[r];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < QR; ++r) {
    if (r >= rows) break;
    for (int w = 0; w < SW; ++w) m[r] = m[r] > maxima[w * QR + r] ? m[r] : maxima[w * QR + r];
    const float big = __uint_as_float(m[r]);
    if (tid == 0) scale[r] = big / 127.0f;
    for (int c = tid; c < nc; c += 64 * SW)
      *(uint64_t*)(codes + r * (g.K + 16) + 8 * c) = src[r] ? quantize8(*(const u32x4_t*)(src[r] + 8 * c), big) : 0;
  }
  __syncthreads();
}

// QX: x is bf16 and quantised here (rows <= QR, NB = 1).
template <bool I8, int NB, bool QX>
__device__ __forceinline__ void skinny_block(const SkinnyArgs& p, int e, int n0, int64_t p0, int rows, float* red,
                                             int8_t* codes, float* qscale) {
  typedef typename std::conditional<I8, i32x4_t, f32x4_t>::type acc_t;
  constexpr int ES = I8 ? 1 : 2;
  const Groups& g = p.g;
  const int lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int KC = g.K * ES / 16;        // 16-byte chunks of a row
  const int steps = (KC + 3) / 4;      // 64-byte steps
  const int n = n0 + l16;
  const char* wrow = p.w + ((int64_t)e * g.N + (n < g.N ? n : 0)) * g.K * ES + quad * 16;
  const int wlim = n < g.N ? KC : 0;
  u32x4_t wf[SUN];
  auto load_w = [&](int s0) {
#pragma unroll
    for (int u = 0; u < SUN; ++u) {
      const int c = 4 * (s0 + u) + quad;
      wf[u] = __builtin_nontemporal_load((const u32x4_t*)(c < wlim ? wrow + (int64_t)(s0 + u) * 64 : (const char*)kZero));
    }
  };
  load_w(SUN * wave);
  const char* xrow[NB];
  int xlim[NB];
  if (QX) quantize_rows(p, p0, rows, codes, qscale, (uint32_t*)red);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = 16 * b + l16;
    if (QX) {
      xlim[b] = r < rows ? KC : 0;
      continue;
    }
    const int64_t t = r < rows ? source_row(g, p0 + r) : -1;
    xrow[b] = p.x + (t < 0 ? 0 : t) * g.ldx * ES + quad * 16;
    xlim[b] = t < 0 ? 0 : KC;
  }
  acc_t acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = (acc_t){};
  for (int s0 = SUN * wave; s0 < steps; s0 += SUN * SW) {
    constexpr int XU = NB == 1 ? SUN : 4;  // steps of x in registers at a time
#pragma unroll
    for (int v = 0; v < SUN; v += XU) {
      u32x4_t xf[NB][XU];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int u = 0; u < XU; ++u) {
          const int c = 4 * (s0 + v + u) + quad;
          if (QX)
            xf[b][u] = c < xlim[b] ? *(const u32x4_t*)(codes + l16 * (g.K + 16) + 16 * c) : u32x4_t{0, 0, 0, 0};
          else
            xf[b][u] = *(const u32x4_t*)(c < xlim[b] ? xrow[b] + (int64_t)(s0 + v + u) * 64 : (const char*)kZero);
        }
#pragma unroll
      for (int u = 0; u < XU; ++u)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (I8)
            acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, wf[v + u]),
                                                           __builtin_bit_cast(i32x4_t, xf[b][u]), acc[b], 0, 0, 0);
          else
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wf[v + u]),
                                                             __builtin_bit_cast(bf16x8_t, xf[b][u]), acc[b], 0, 0, 0);
        }
    }
    if (s0 + SUN * SW < steps) load_w(s0 + SUN * SW);
  }
  // block layout: lane -> x row l16, register r -> weight row 4 quad + r
  typedef typename std::conditional<I8, int32_t, float>::type el_t;
  el_t* rd = (el_t*)red;  // [wave][16 NB rows][16]
#pragma unroll
  for (int b = 0; b < NB; ++b) *(acc_t*)(rd + ((wave * 16 * NB) + 16 * b + l16) * 16 + 4 * quad) = acc[b];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * 8; i += 64 * SW) {  // two weight rows a thread
    const int r = i >> 3, c = 2 * (i & 7), col = n0 + c;
    if (col >= g.N) continue;
    el_t v0 = 0, v1 = 0;
#pragma unroll
    for (int w = 0; w < SW; ++w) {
      v0 += rd[(w * 16 * NB + r) * 16 + c];
      v1 += rd[(w * 16 * NB + r) * 16 + c + 1];
    }
    float f0 = (float)v0, f1 = (float)v1;
    if (I8) {
      const int64_t t = QX ? 0 : source_row(g, p0 + r);
      const float xs = QX ? qscale[r] : t < 0 ? 0.0f : p.sc.x[t];
      const float* ws = p.sc.w + (int64_t)e * g.N + col;
      f0 = f0 * (xs * ws[0]) + (p.sc.bias ? p.sc.bias[col] : 0.0f);
      f1 = f1 * (xs * ws[1]) + (p.sc.bias ? p.sc.bias[col + 1] : 0.0f);
    }
    if (p.fp32) {
      float* o = (float*)p.y + (p0 + r) * g.ldy + col;
      o[0] = f0;
      o[1] = f1;
    } else {
      *(uint32_t*)((uint16_t*)p.y + (p0 + r) * g.ldy + col) = pack_bf16x2(f0, f1);
    }
  }
}

template <bool I8, bool QX>
__global__ __launch_bounds__(64 * SW) void k_op_skinny(SkinnyArgs p) {
  __shared__ float red[QX ? SW * 16 * 16 : SW * 64 * 16];
  __shared__ float qscale[QR];
  extern __shared__ u32x4_t codes[];  // QX: QR rows of K + 16 bytes
  const Groups& g = p.g;
  const int n0 = blockIdx.x * SN;
  int e = blockIdx.y;
  if (p.by_row) {
    // the expert of row blockIdx.y, taken by the workgroup of its first row
    const int64_t row = blockIdx.y;
    const int lane = threadIdx.x & 63;
    e = 0;
    for (int i = lane; i < (g.E + 63) / 64 * 64; i += 64)
      e += __builtin_popcountll(__ballot(i < g.E && g.offsets[i + 1] <= row));
    e = __builtin_amdgcn_readfirstlane(e);
    if (e >= g.E) return;
    if (group_range(g, e).lo != row) return;
  }
  const Range range = group_range(g, e);
  int64_t lo = range.lo;
  const int64_t hi = range.hi;
  while (lo < hi) {
    constexpr int MAXR = QX ? QR : 64;
    const int rows = (int)(hi - lo < MAXR ? hi - lo : MAXR);
    if (QX || rows <= 16)
      skinny_block<I8, 1, QX>(p, e, n0, lo, rows, red, (int8_t*)codes, qscale);
    else if (rows <= 32)
      skinny_block<I8, 2, false>(p, e, n0, lo, rows, red, nullptr, nullptr);
    else
      skinny_block<I8, 4, false>(p, e, n0, lo, rows, red, nullptr, nullptr);
    lo += rows;
    if (lo < hi) __syncthreads();  // the partial sums are read before they are overwritten
  }
}

}  // namespace

hipError_t launch_op_skinny(bool i8, bool quantize, const Groups& g, const void* x, const void* w, const Scales& sc, void* y,
                            bool fp32, hipStream_t s) {
  SkinnyArgs a{};
  a.g = g;
  a.x = (const char*)x;
  a.w = (const char*)w;
  a.sc = sc;
  a.y = y;
  a.fp32 = fp32;
  a.by_row = g.offsets && g.rows < g.E;
  const dim3 grid((unsigned)((g.N + SN - 1) / SN), (unsigned)(a.by_row ? g.rows : g.E));
  const Launch lc{s, nullptr, nullptr};
  if (quantize) return launch_shm(lc, k_op_skinny<true, true>, grid, dim3(64 * SW), (size_t)QR * (g.K + 16), a);
  if (i8) return launch(lc, k_op_skinny<true, false>, grid, dim3(64 * SW), a);
  return launch(lc, k_op_skinny<false, false>, grid, dim3(64 * SW), a);
}

}  // namespace moe
