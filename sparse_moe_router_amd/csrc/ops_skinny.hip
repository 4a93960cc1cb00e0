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
// its results' way through memory cost more.  Gated products take eight rows of
// each of the expert's two matrices, whose sums then meet in the same place.  The
// logits of few tokens against a vocabulary become a maximum and a sum of
// exponentials of each token and 16 columns, or their gradients, there.
#include <type_traits>

#include "ops_internal.h"
#include "ops_loss.h"
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
  uint16_t* pre;  // gated: the products themselves (NULL: not kept)
  int64_t ldp;
  LossTokens loss;  // logits
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

enum { PLAIN = 0, GATED_UNIT = 1, LOGITS = 2, LOGIT_GRADS = 3 };
// QX: x is bf16 and quantised here (rows <= QR, NB = 1).  GATED_UNIT: n0 counts the
// rows of each matrix; the block's rows 0..7 are of the first, 8..15 of the second.
template <bool I8, int NB, bool QX, int MODE>
__device__ __forceinline__ void skinny_block(const SkinnyArgs& p, int e, int n0, int64_t p0, int rows, float* red,
                                             int8_t* codes, float* qscale) {
  typedef typename std::conditional<I8, i32x4_t, f32x4_t>::type acc_t;
  constexpr int ES = I8 ? 1 : 2;
  constexpr bool GATED = MODE == GATED_UNIT;
  const Groups& g = p.g;
  const int lane = threadIdx.x & 63, l16 = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int KC = g.K * ES / 16;        // 16-byte chunks of a row
  const int steps = (KC + 3) / 4;      // 64-byte steps
  const int n = GATED ? n0 + (l16 & 7) : n0 + l16;
  const int64_t first = GATED ? ((int64_t)2 * e + (l16 >> 3)) * g.N : (int64_t)e * g.N;
  const char* wrow = p.w + (first + (n < g.N ? n : 0)) * g.K * ES + quad * 16;
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
  if constexpr (GATED) {
    for (int i = threadIdx.x; i < rows * 4; i += 64 * SW) {  // two features a thread
      const int r = i >> 2, c = 2 * (i & 3);
      float v[2][2] = {};
#pragma unroll
      for (int w = 0; w < SW; ++w)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          v[m][0] += rd[(w * 16 * NB + r) * 16 + 8 * m + c];
          v[m][1] += rd[(w * 16 * NB + r) * 16 + 8 * m + c + 1];
        }
      *(uint32_t*)((uint16_t*)p.y + (p0 + r) * g.ldy + n0 + c) =
          pack_bf16x2(silu(v[0][0]) * v[1][0], silu(v[0][1]) * v[1][1]);
      if (p.pre) {
        uint16_t* o = p.pre + (p0 + r) * p.ldp + n0 + c;
        *(uint32_t*)o = pack_bf16x2(v[0][0], v[0][1]);
        *(uint32_t*)(o + g.N) = pack_bf16x2(v[1][0], v[1][1]);
      }
    }
    return;
  }
  if constexpr (MODE == LOGITS || MODE == LOGIT_GRADS) {
    for (int i = threadIdx.x; i < (rows + 3) / 4 * 64; i += 64 * SW) {  // a column a thread, a token 16 lanes
      const int r = i >> 4, c = i & 15, col = n0 + c;
      if (r >= rows) continue;
      float z = 0.0f;
#pragma unroll
      for (int w = 0; w < SW; ++w) z += rd[(w * 16 * NB + r) * 16 + c];
      const int64_t t = p0 + r, hit = p.loss.target[t] - p.loss.v0;
      if constexpr (MODE == LOGITS) {
        if (col >= g.N) z = -INFINITY;
        if (hit == col) p.loss.hit[t] = z;
        float m = z;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
        float e = exp_from(z, m);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) e += __shfl_xor(e, d, 64);
        if (c == 0) p.loss.part[(int64_t)blockIdx.x * g.rows + t] = float2{m, e};
      } else {
        // all 16 columns: those past the vocabulary, which the products read with the last eight, are zeros
        const float w = scale_of(p.loss, t), e = __expf(z - p.loss.lse[t]);
        p.loss.d[t * p.loss.ldd + col] = (uint16_t)f32_to_bf16(w != 0.0f && col < g.N ? (hit == col ? e - 1.0f : e) : 0.0f);
      }
    }
    return;
  }
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

template <bool I8, bool QX, int MODE = PLAIN>
__global__ __launch_bounds__(64 * SW) void k_op_skinny(SkinnyArgs p) {
  __shared__ float red[QX ? SW * 16 * 16 : SW * 64 * 16];
  __shared__ float qscale[QR];
  extern __shared__ u32x4_t codes[];  // QX: QR rows of K + 16 bytes
  const Groups& g = p.g;
  const int n0 = blockIdx.x * (MODE == GATED_UNIT ? SN / 2 : SN);
  int e = blockIdx.y;
  Range range;
  if constexpr (MODE == LOGITS || MODE == LOGIT_GRADS) {
    // 64 tokens a workgroup row
    e = 0;
    range = limited(g, (int64_t)blockIdx.y * 64, (int64_t)blockIdx.y * 64 + 64);
  } else if (p.by_row) {
    // the expert of row blockIdx.y, taken by the workgroup of its first row; of up to 256 experts all
    // offsets are on their way at a time, and the expert's own are among them
    const int64_t row = blockIdx.y;
    const int lane = threadIdx.x & 63;
    const int32_t front = g.offsets[0];
    int32_t v[4];
    e = 0;
    for (int i0 = 0; i0 < g.E; i0 += 256) {
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = g.offsets[i0 + 64 * u + lane < g.E ? i0 + 64 * u + lane + 1 : g.E];
#pragma unroll
      for (int u = 0; u < 4; ++u) e += __builtin_popcountll(__ballot(i0 + 64 * u + lane < g.E && v[u] <= row));
    }
    e = __builtin_amdgcn_readfirstlane(e);
    if (e >= g.E) return;
    if (g.E <= 256) {
      auto at = [&](int i) {  // offsets[i + 1]
        const int32_t x = i < 64 ? v[0] : i < 128 ? v[1] : i < 192 ? v[2] : v[3];
        return __builtin_amdgcn_readlane(x, i & 63);
      };
      range = limited(g, e > 0 ? at(e - 1) : front, at(e));
    } else {
      range = group_range(g, e);
    }
    if (range.lo != row) return;
  } else {
    range = group_range(g, e);
  }
  int64_t lo = range.lo;
  const int64_t hi = range.hi;
  while (lo < hi) {
    constexpr int MAXR = QX ? QR : 64;
    const int rows = (int)(hi - lo < MAXR ? hi - lo : MAXR);
    if (QX || rows <= 16)
      skinny_block<I8, 1, QX, MODE>(p, e, n0, lo, rows, red, (int8_t*)codes, qscale);
    else if (rows <= 32)
      skinny_block<I8, 2, false, MODE>(p, e, n0, lo, rows, red, nullptr, nullptr);
    else
      skinny_block<I8, 4, false, MODE>(p, e, n0, lo, rows, red, nullptr, nullptr);
    lo += rows;
    if (lo < hi) __syncthreads();  // the partial sums are read before they are overwritten
  }
}

}  // namespace

hipError_t launch_gated_skinny(const Groups& g, const void* x, const void* w, void* h, void* pre, int64_t ldp,
                               hipStream_t s) {
  SkinnyArgs a{};
  a.g = g;
  a.x = (const char*)x;
  a.w = (const char*)w;
  a.y = h;
  a.pre = (uint16_t*)pre;
  a.ldp = ldp;
  a.by_row = g.offsets && g.rows < g.E;
  const dim3 grid((unsigned)((g.N + SN / 2 - 1) / (SN / 2)), (unsigned)(a.by_row ? g.rows : g.E));
  return launch(Launch{s, nullptr, nullptr}, k_op_skinny<false, false, GATED_UNIT>, grid, dim3(64 * SW), a);
}

hipError_t launch_loss_skinny(const Groups& g, const void* x, const void* w, const LossTokens& loss, bool grad,
                              hipStream_t s) {
  SkinnyArgs a{};
  a.g = g;
  a.x = (const char*)x;
  a.w = (const char*)w;
  a.loss = loss;
  const dim3 grid((unsigned)((g.N + SN - 1) / SN), (unsigned)((g.rows + 63) / 64));
  const Launch lc{s, nullptr, nullptr};
  return grad ? launch(lc, k_op_skinny<false, false, LOGIT_GRADS>, grid, dim3(64 * SW), a)
              : launch(lc, k_op_skinny<false, false, LOGITS>, grid, dim3(64 * SW), a);
}

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
