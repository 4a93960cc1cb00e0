// Row operators (gfx950, wave64): the norms before and after a block with its
// gate and residual sum, their gradients, and the 8-bit token quantiser.
//
//   block_norm    h = x r w,                        r = rsqrt(mean x^2 + eps)
//   block_merge   out = residual + a s(gate) y r w, then h = out r' w'
//   gradient of n = v r w for dn:  dv = r (dn w - (v r) mean(dn w v r)),
//                                  dw = sum over rows of dn v r
//   (in this order: r^3 of a row of zeros and a small eps is past fp32, and
//   that of a row of 1e15 below it)
//
// All are bound by HBM: a row is read once into registers (as it is stored,
// 16 bytes a lane a load), its sums go through wave shuffles (and LDS when
// several waves share the row), and every result is written once.  Weight
// gradients: each workgroup sums its rows in registers, a second launch adds
// the workgroups' sums in a fixed order.
#include <type_traits>

#include "ops_internal.h"
#include "quantize8.h"

namespace moe {
namespace {

// eight elements of a row, as stored
template <bool F32>
struct Raw8;
template <>
struct Raw8<false> {
  u32x4_t v;
  __device__ __forceinline__ void load(const void* p, int64_t i) { v = *(const u32x4_t*)((const uint16_t*)p + i); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_lo(v[j]);
      f[2 * j + 1] = bf16_hi(v[j]);
    }
  }
  // rounds f to the stored type
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const { *(u32x4_t*)((uint16_t*)p + i) = v; }
};
template <>
struct Raw8<true> {
  f32x4_t a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = *(const f32x4_t*)((const float*)p + i);
    b = *(const f32x4_t*)((const float*)p + i + 4);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = a[j];
      f[4 + j] = b[j];
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = f[j];
      b[j] = f[4 + j];
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    *(f32x4_t*)((float*)p + i) = a;
    *(f32x4_t*)((float*)p + i + 4) = b;
  }
};

__device__ __forceinline__ void load_weight(const void* w, bool f32, int col, float (&f)[8]) {
  if (f32) {
    Raw8<true> r;
    r.load(w, col);
    r.get(f);
  } else {
    Raw8<false> r;
    r.load(w, col);
    r.get(f);
  }
}

// sigmoid(z), and its derivative s(z) s(-z), from e = exp(-|z|): 1 - s(z) is
// never formed, which would lose the derivative of a wide open gate.
__device__ __forceinline__ float sigmoid(float z, float* slope = nullptr) {
  const float e = __expf(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
  if (slope) *slope = e * r * r;
  return z >= 0.0f ? r : z < 0.0f ? e * r : z;  // a NaN stays one
}

// Sums of NV values over the threads of one row: a wave (WPR = 1) or the whole
// workgroup of WPR waves; the same order in every call.
template <int WPR, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor(v[i], d, 64);
  if (WPR > 1) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) lds[wave * NV + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = 0.0f;
      for (int w = 0; w < WPR; ++w) v[i] += lds[w * NV + i];
    }
  }
}

// rows of a workgroup: one with WPR > 1, one a wave of four with WPR = 1
template <int WPR>
constexpr int kWaves = WPR == 1 ? 4 : WPR;

// Workgroups of a forward launch at most (threads of a launch stay below 2^32); rows past them are
// taken by the same workgroups in turn.
constexpr int64_t kMaxGroups = 1 << 20;
template <int WPR>
__device__ __forceinline__ int64_t first_row() {
  return WPR == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
}
template <int WPR>
__device__ __forceinline__ int64_t row_stride() {
  return (int64_t)gridDim.x * (WPR == 1 ? 4 : 1);
}
template <int WPR>
unsigned row_grid(int64_t rows) {
  const int64_t n = WPR == 1 ? (rows + 3) / 4 : rows;
  return (unsigned)(n < kMaxGroups ? n : kMaxGroups);
}

// Thread t of a row holds the 8-element chunks t, t + 64 WPR, ... below H / 8.
template <int WPR, int CPT, bool S32, bool MERGE>
__global__ __launch_bounds__(64 * kWaves<WPR>) void k_norm_fwd(NormArgs p) {
  __shared__ float lds[WPR > 1 ? WPR : 1];
  const int t = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int nc = p.H / 8;
  // the launch covers all rows unless there are more than kMaxGroups workgroups' worth
  for (int64_t row = first_row<WPR>(); row < p.rows; row += row_stride<WPR>()) {
    Raw8<S32> x[CPT];
    Raw8<false> y[CPT], gt[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int c = t + 64 * WPR * j;
      if (c < nc) {
        x[j].load(p.residual.data, row * p.residual.ld + 8 * c);
        if (MERGE) {
          y[j].load(p.y.data, row * p.y.ld + 8 * c);
          if (p.gate_mode == MOE_GATE_ELEMENT) gt[j].load(p.gate.data, row * p.gate.ld + 8 * c);
        }
      }
    }
    const float rh = 1.0f / (float)p.H;
    const void* wn = MERGE ? p.next_weight : p.weight;
    if (MERGE) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < CPT; ++j)
        if (t + 64 * WPR * j < nc) {
          float f[8];
          y[j].get(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss[0] += f[i] * f[i];
        }
      row_sum<WPR, 1>(ss, lds);
      float a = p.scale * rsqrtf(ss[0] * rh + p.eps);
      if (p.gate_mode == MOE_GATE_TOKEN)
        a *= sigmoid(__uint_as_float((uint32_t)((const uint16_t*)p.gate.data)[row] << 16));
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const int c = t + 64 * WPR * j;
        if (c < nc) {
          float f[8], o[8], w[8];
          y[j].get(f);
          x[j].get(o);
          load_weight(p.weight, p.weight32, 8 * c, w);
          if (p.gate_mode == MOE_GATE_ELEMENT) {
            float g[8];
            gt[j].get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += a * f[i] * w[i] * sigmoid(g[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += a * f[i] * w[i];
          }
          x[j].set(o);
          x[j].store(p.out.data, row * p.out.ld + 8 * c);
        }
      }
      if (!p.h.data) continue;
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < CPT; ++j)
      if (t + 64 * WPR * j < nc) {
        float f[8];
        x[j].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] += f[i] * f[i];
      }
    row_sum<WPR, 1>(ss, lds);
    const float r = rsqrtf(ss[0] * rh + p.eps);
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int c = t + 64 * WPR * j;
      if (c < nc) {
        float f[8], w[8];
        x[j].get(f);
        load_weight(wn, p.weight32, 8 * c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
        Raw8<false> o;
        o.set(f);
        o.store(p.h.data, row * p.h.ld + 8 * c);
      }
    }
  }
}

// Gradients.  Workgroup b takes the rows b * R, b * R + gridDim * R, ... (R rows
// at a time) and keeps its part of the weight gradients in registers.
template <int WPR, int CPT, bool S32, bool MERGE>
__global__ __launch_bounds__(64 * kWaves<WPR>) void k_norm_bwd(NormArgs p) {
  __shared__ float lds[WPR > 1 ? 3 * WPR : 1];
  __shared__ float comb[WPR == 1 ? 4 * 64 * 8 : 1];
  constexpr int R = WPR == 1 ? 4 : 1;
  const int t = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int wave = threadIdx.x >> 6;
  const int nc = p.H / 8;
  const float rh = 1.0f / (float)p.H;
  // block_norm_grad is the "next norm" half alone: out = x, dn = d_h, d_out = d_add
  const bool next = MERGE ? p.d_h.data != nullptr : true;
  const void* wn = MERGE ? p.next_weight : p.weight;
  // this thread's part of the weight gradients; with four chunks a thread in LDS ([2][H], each thread
  // its own columns), as the registers do not hold it beside the row
  constexpr bool LDS_SUMS = WPR == 8 && CPT == 4;
  extern __shared__ f32x4_t sums[];
  float aw[LDS_SUMS ? 1 : CPT][8], an[LDS_SUMS ? 1 : CPT][8];
  auto add = [&](int k, int j, const float(&f)[8]) {
    if (LDS_SUMS) {
      f32x4_t* at = sums + (k * p.H + 8 * (t + 64 * WPR * j)) / 4;
      at[0] += f32x4_t{f[0], f[1], f[2], f[3]};
      at[1] += f32x4_t{f[4], f[5], f[6], f[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) (k ? an : aw)[LDS_SUMS ? 0 : j][i] += f[i];
    }
  };
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (LDS_SUMS) {
      for (int k = 0; k < 2 && t + 64 * WPR * j < nc; ++k) {
        f32x4_t* at = sums + (k * p.H + 8 * (t + 64 * WPR * j)) / 4;
        at[0] = at[1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) aw[LDS_SUMS ? 0 : j][i] = an[LDS_SUMS ? 0 : j][i] = 0.0f;
    }
  }
  struct Row {
    Raw8<S32> v[CPT], d[CPT];
    Raw8<false> dh[CPT], y[CPT], gt[CPT];
  };
  auto load = [&](Row& q, int64_t row) {
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int c = t + 64 * WPR * j;
      if (c < nc && row < p.rows) {
        if (next) {
          q.v[j].load(p.out.data, row * p.out.ld + 8 * c);
          q.dh[j].load(p.d_h.data, row * p.d_h.ld + 8 * c);
        }
        if (p.d_out.data) q.d[j].load(p.d_out.data, row * p.d_out.ld + 8 * c);
        if (MERGE) {
          q.y[j].load(p.y.data, row * p.y.ld + 8 * c);
          if (p.gate_mode == MOE_GATE_ELEMENT) q.gt[j].load(p.gate.data, row * p.gate.ld + 8 * c);
        }
      }
    }
  };
  // the next row's loads are on their way while this one's sums are taken, where a thread's part
  // of a row is one chunk (two rows of two would not fit the registers)
  constexpr bool AHEAD = CPT == 1;
  const int64_t stride = (int64_t)gridDim.x * R, row0 = (int64_t)blockIdx.x * R + (WPR == 1 ? wave : 0);
  Row ahead;
  if (AHEAD) load(ahead, row0);
  for (int64_t row = row0; row < p.rows; row += stride) {
    Row cur;
    if (AHEAD) {
      cur = ahead;
      load(ahead, row + stride);
    } else {
      load(cur, row);
    }
    const Raw8<S32>(&v)[CPT] = cur.v;
    const Raw8<S32>(&d)[CPT] = cur.d;
    const Raw8<false>(&dh)[CPT] = cur.dh;
    const Raw8<false>(&y)[CPT] = cur.y;
    const Raw8<false>(&gt)[CPT] = cur.gt;
    // sums: v^2, d_h w' v, y^2
    float s1[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int c = t + 64 * WPR * j;
      if (c < nc) {
        float f[8];
        if (next) {
          float e[8], w[8];
          v[j].get(f);
          dh[j].get(e);
          load_weight(wn, p.weight32, 8 * c, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            s1[0] += f[i] * f[i];
            s1[1] += e[i] * w[i] * f[i];
          }
        }
        if (MERGE) {
          y[j].get(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) s1[2] += f[i] * f[i];
        }
      }
    }
    row_sum<WPR, 3>(s1, lds);
    const float rn = rsqrtf(s1[0] * rh + p.eps), mn = s1[1] * rh * rn;
    const float ry = rsqrtf(s1[2] * rh + p.eps);
    float gs = p.scale;  // the block output's factor where it is one for the whole row
    float gslope = 0.0f;
    if (MERGE && p.gate_mode == MOE_GATE_TOKEN) {
      gs *= sigmoid(__uint_as_float((uint32_t)((const uint16_t*)p.gate.data)[row] << 16), &gslope);
    }
    // D = d_out + gradient through the next norm; it is d_residual
    float s2[2] = {0.0f, 0.0f};  // sums: db w y, D b (db = the gradient of the normed y)
    float D[CPT][8];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int c = t + 64 * WPR * j;
      if (c < nc) {
        if (p.d_out.data)
          d[j].get(D[j]);
        else
#pragma unroll
          for (int i = 0; i < 8; ++i) D[j][i] = 0.0f;
        if (next) {
          float f[8], e[8], w[8];
          v[j].get(f);
          dh[j].get(e);
          load_weight(wn, p.weight32, 8 * c, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[i] *= rn;
            D[j][i] += rn * (e[i] * w[i] - f[i] * mn);
            e[i] *= f[i];
          }
          add(1, j, e);
        }
        Raw8<S32> o;
        o.set(D[j]);
        o.store(p.d_residual.data, row * p.d_residual.ld + 8 * c);
        if (MERGE) {
          float f[8], w[8], g[8];
          y[j].get(f);
          load_weight(p.weight, p.weight32, 8 * c, w);
          if (p.gate_mode == MOE_GATE_ELEMENT) {
            gt[j].get(g);
            float dg[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float slope;
              const float sg = sigmoid(g[i], &slope), b = f[i] * ry * w[i];
              dg[i] = p.scale * D[j][i] * b * slope;
              D[j][i] *= p.scale * sg;  // now db
            }
            Raw8<false> og;
            og.set(dg);
            og.store(p.d_gate.data, row * p.d_gate.ld + 8 * c);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              s2[1] += D[j][i] * (f[i] * ry * w[i]);
              D[j][i] *= gs;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            s2[0] += D[j][i] * w[i] * f[i];
            f[i] = D[j][i] * f[i] * ry;
          }
          add(0, j, f);
        }
      }
    }
    if (MERGE) {
      row_sum<WPR, 2>(s2, lds);
      if (p.gate_mode == MOE_GATE_TOKEN && t == 0)
        ((uint16_t*)p.d_gate.data)[row] = (uint16_t)f32_to_bf16(p.scale * s2[1] * gslope);
      const float my = s2[0] * rh * ry;
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const int c = t + 64 * WPR * j;
          if (c < nc) {
          float f[8], w[8];
          y[j].get(f);
          load_weight(p.weight, p.weight32, 8 * c, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = ry * (D[j][i] * w[i] - f[i] * ry * my);
          Raw8<false> o;
          o.set(f);
          o.store(p.d_y.data, row * p.d_y.ld + 8 * c);
        }
      }
    }
  }
  // this workgroup's sums: [0] of weight (merge), [1] of the next norm's weight
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.H;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k == 0 && !MERGE) continue;
    if (k == 1 && !next) continue;
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int c = t + 64 * WPR * j;
      if (WPR == 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) comb[(wave * 8 + i) * 64 + t] = (k ? an : aw)[LDS_SUMS ? 0 : j][i];
        __syncthreads();
        // wave w adds elements 2 w, 2 w + 1 of every chunk, in wave order
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float s = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) s += comb[(w * 8 + 2 * wave + i) * 64 + t];
          if (c < nc) part[(int64_t)k * p.H + 8 * c + 2 * wave + i] = s;
        }
      } else if (c < nc) {
        f32x4_t* to = (f32x4_t*)(part + (int64_t)k * p.H + 8 * c);
        if (LDS_SUMS) {
          to[0] = sums[(k * p.H + 8 * c) / 4];
          to[1] = sums[(k * p.H + 8 * c) / 4 + 1];
        } else {
          const float(&f)[8] = (k ? an : aw)[LDS_SUMS ? 0 : j];
          to[0] = f32x4_t{f[0], f[1], f[2], f[3]};
          to[1] = f32x4_t{f[4], f[5], f[6], f[7]};
        }
      }
    }
  }
}

// d_weight / d_next_weight: sums over the workgroups' parts, in a fixed order.
// A workgroup takes 64 columns; its 32 groups of 16 threads take every 32nd
// part each, 16 bytes a thread, eight loads in flight.
__global__ __launch_bounds__(512) void k_norm_reduce(const float* part, int groups, int H, float* d0, float* d1) {
  __shared__ f32x4_t lds[32][16];
  const int k = blockIdx.y;
  float* dst = k ? d1 : d0;
  if (!dst) return;
  const int cx = threadIdx.x & 15, gy = threadIdx.x >> 4;
  const int col = blockIdx.x * 64 + 4 * cx;  // H is a multiple of 8
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < H) {
    for (int g0 = gy; g0 < groups; g0 += 32 * 8) {
      f32x4_t v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int g = g0 + 32 * u;
        v[u] = g < groups ? *(const f32x4_t*)(part + ((int64_t)g * 2 + k) * H + col) : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
  }
  lds[gy][cx] = s;
  __syncthreads();
  if (gy == 0 && col < H) {
    f32x4_t r = lds[0][cx];
#pragma unroll
    for (int i = 1; i < 32; ++i) r += lds[i][cx];
    *(f32x4_t*)(dst + col) = r;
  }
}

// Codes and scales of token rows (quantize8).
template <int WPR, int CPT>
__global__ __launch_bounds__(64 * kWaves<WPR>) void k_quantize(int64_t rows, int K, int64_t ldx, const uint16_t* x,
                                                               int8_t* codes, float* scale) {
  __shared__ uint32_t lds[WPR > 1 ? WPR : 1];
  const int t = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int nc = K / 8;
  for (int64_t row = first_row<WPR>(); row < rows; row += row_stride<WPR>()) {
    u32x4_t v[CPT];
    uint32_t m = 0;  // the largest magnitude's bits
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int c = t + 64 * WPR * j;
      if (c < nc) {
        v[j] = *(const u32x4_t*)(x + row * ldx + 8 * c);
        const uint32_t o = max_magnitude(v[j]);
        m = m > o ? m : o;
      }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      const uint32_t o = __shfl_xor(m, d, 64);
      m = m > o ? m : o;
    }
    if (WPR > 1) {
      __syncthreads();  // the previous row's maximum has been read
      if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
      __syncthreads();
      m = lds[0];
      for (int w = 1; w < WPR; ++w) m = m > lds[w] ? m : lds[w];
    }
    const float big = __uint_as_float(m);
    if (t == 0) scale[row] = big / 127.0f;
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int c = t + 64 * WPR * j;
      if (c < nc) *(uint64_t*)(codes + row * K + 8 * c) = quantize8(v[j], big);
    }
  }
}

// Threads of a row: a wave where it holds the row in at most WAVE_CPT chunks a
// lane, else four or eight waves.  Few rows take four waves each, to shorten
// the one row's way.  WAVE_CPT: 4 for the forward norms (8192 x 2048 at 5 TB/s),
// 2 for the gradients, whose registers hold no more beside the sums, and for
// the quantiser (8192 x 2048 13.2 us by four waves, 15.7 by one; 4096 x 1024
// 5.8 and 5.1).
struct RowPlan {
  int wpr, cpt;
};
template <int WAVE_CPT>
RowPlan row_plan(int64_t rows, int H) {
  const int nc = H / 8;
  if (rows >= 1024 && nc <= 64 * WAVE_CPT) return {1, nc <= 64 ? 1 : nc <= 128 ? 2 : 4};
  if (nc <= 64) return {1, 1};
  if (nc <= 256) return {4, 1};
  if (nc <= 512) return {4, 2};
  if (nc <= 1024) return {8, 2};
  return {8, 4};
}

template <int WPR, int CPT, bool MERGE>
hipError_t fwd(const NormArgs& a, hipStream_t s) {
  const unsigned grid = row_grid<WPR>(a.rows);
  const Launch lc{s, nullptr, nullptr};
  if (a.stream32) return launch(lc, k_norm_fwd<WPR, CPT, true, MERGE>, dim3(grid), dim3(64 * kWaves<WPR>), a);
  return launch(lc, k_norm_fwd<WPR, CPT, false, MERGE>, dim3(grid), dim3(64 * kWaves<WPR>), a);
}
template <int WPR, int CPT, bool MERGE>
hipError_t bwd(const NormArgs& a, unsigned grid, hipStream_t s) {
  const Launch lc{s, nullptr, nullptr};
  const size_t shm = WPR == 8 && CPT == 4 ? (size_t)a.H * 8 : 0;  // its sums of the weight gradients
  if (a.stream32) return launch_shm(lc, k_norm_bwd<WPR, CPT, true, MERGE>, dim3(grid), dim3(64 * kWaves<WPR>), shm, a);
  return launch_shm(lc, k_norm_bwd<WPR, CPT, false, MERGE>, dim3(grid), dim3(64 * kWaves<WPR>), shm, a);
}

// calls f(WPR, CPT) with the plan's values as constants
template <int WAVE_CPT, class F>
hipError_t with_plan(int64_t rows, int H, F&& f) {
  const RowPlan r = row_plan<WAVE_CPT>(rows, H);
#define MOE_CASE(W, C) \
  if (r.wpr == W && r.cpt == C) return f(std::integral_constant<int, W>{}, std::integral_constant<int, C>{});
  MOE_CASE(1, 1)
  MOE_CASE(1, 2)
  if constexpr (WAVE_CPT == 4) {
    MOE_CASE(1, 4)
  }
  MOE_CASE(4, 1)
  MOE_CASE(4, 2)
  MOE_CASE(8, 2)
  MOE_CASE(8, 4)
#undef MOE_CASE
  return hipErrorInvalidValue;
}

}  // namespace

int norm_grad_groups(int64_t rows, int H) {
  const RowPlan r = row_plan<2>(rows, H);
  const int64_t units = r.wpr == 1 ? (rows + 3) / 4 : rows;
  const int64_t most = r.wpr < 8 ? 1024 : r.cpt == 2 ? 512 : 256;
  return (int)(units < most ? units : most);
}

hipError_t launch_norm_fwd(const NormArgs& a, bool merge, hipStream_t s) {
  return with_plan<4>(a.rows, a.H, [&](auto w, auto c) {
    return merge ? fwd<w(), c(), true>(a, s) : fwd<w(), c(), false>(a, s);
  });
}

hipError_t launch_norm_bwd(const NormArgs& a, bool merge, hipStream_t s) {
  const int groups = norm_grad_groups(a.rows, a.H);
  if (groups > 0) {
    const hipError_t e = with_plan<2>(a.rows, a.H, [&](auto w, auto c) {
      return merge ? bwd<w(), c(), true>(a, groups, s) : bwd<w(), c(), false>(a, groups, s);
    });
    if (e != hipSuccess) return e;
  }
  const Launch lc{s, nullptr, nullptr};
  return launch(lc, k_norm_reduce, dim3((a.H + 63) / 64, 2), dim3(512), (const float*)a.part, groups, a.H,
                merge ? a.d_weight : nullptr, merge ? a.d_next_weight : a.d_weight);
}

hipError_t launch_quantize_i8(int64_t rows, int K, int64_t ldx, const uint16_t* x, int8_t* codes, float* scale,
                              hipStream_t s) {
  return with_plan<2>(rows, K, [&](auto w, auto c) {
    constexpr int WPR = w(), CPT = c();
    const unsigned grid = row_grid<WPR>(rows);
    return launch(Launch{s, nullptr, nullptr}, k_quantize<WPR, CPT>, dim3(grid), dim3(64 * kWaves<WPR>), rows, K, ldx,
                  x, codes, scale);
  });
}

}  // namespace moe
