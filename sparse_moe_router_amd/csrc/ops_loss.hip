// Softmax cross entropy against a vocabulary (gfx950, wave64, MFMA):
//   z = x W^T (never stored),  lse[t] = log sum_v exp z[t][v],  loss[t] = lse[t] - z[t][target[t]]
//   d[t][v] = exp(z[t][v] - lse[t]) - (v == target[t]),  dx = d_loss d W,  dW = (d_loss d)^T x
// on the tiles of the grouped products (ops_tile.h).
//
// Forward: every 256 x 256 tile of z is reduced in its epilogue to a maximum
// and a sum of exponentials for each row, 8 bytes where z has 1024; a second
// launch joins the panels of a row.  Gradients: the vocabulary goes by in
// pieces; a piece's z is computed again, becomes d in bf16 in the epilogue, and d feeds the two
// gradient products of the piece while it is still in the last-level cache.
// dx is summed over the pieces in fp32; where its tiles are too few for the
// chip, a piece's reduction is cut into slices with sums of their own, which
// the last launch adds in a fixed order.
//
// d is rounded to bf16 without the token's d_loss: the mean's 1 / n is the same
// for all of them and so would be its rounding, an error of up to 2^-8 of whole
// gradients (dx and dW of 999 tokens were off by 0.28% of their norm; now 0.17%,
// the rounding of the results).  dx takes d_loss in fp32 with
// its last sum; dW takes the largest d_loss in its epilogue, and the token's
// share of that, exactly 1 for a mean, into the bf16 copy of x that it reads.
//
// 4096 tokens against 65536 x 2048: logits 900 to 946 us = 1.16 to 1.22 PFLOP/s (matrix units busy 69% at 1.6
// to 1.7 GHz), their gradients 2 x 511 to 528 = 1.04 to 1.08 (57% at 1.7 to 1.8 GHz: each
// tile has 128 KB to store), products 2 x 808 to 852 = 1.29 to 1.36 (75% at 1.7 GHz): power as much as the loop.
// 257 tokens against 32003 x 2048: 44 us, 131 MB of weights at 3 TB/s: the 32 steps of the one tile that a
// workgroup has, with two stages in flight, not the bytes.
#include "ops_loss.h"
#include "ops_paths.h"
#include "ops_sum.h"
#include "ops_tile.h"

namespace moe {
namespace {

constexpr float LOG2E = 1.44269504088896340736f;

// The value of lane i ^ 1, i ^ 2 of each four.
__device__ __forceinline__ float quad_xor1(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true));
}
__device__ __forceinline__ float quad_xor2(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true));
}

struct LseEpi {
  static constexpr bool kGated = false;
  LossTokens t;
  int64_t rows;  // of all tiles

  template <int RB0, int RB1, class ACC>
  __device__ __forceinline__ void tile(const TileArgs& p, const TileOut& o, ACC& acc, u32x4_t* lds) const {
    float* st = (float*)epi_stage(lds, o);
    const int side = o.lane & 3;  // four lanes a row, 16 columns each
    const int col = o.c0 + 64 * o.wn + 16 * side, n = p.g.N - col;
    const bool whole = o.c0 + TB <= p.g.N;  // uniform
    constexpr int NB = RB0 + RB1;
    float2 mine[NB][2];  // of the lane's row in each half block
    int b = 0;
    each_block<RB0, RB1>(o, acc, [&](int row0, const f32x16_t& a0, const f32x16_t& a1) __attribute__((always_inline)) {
      int64_t at[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = row0 + 16 * q + (o.lane >> 2);
        at[q] = row < o.rows ? t.target[o.p0 + row] - col : -1;
      }
      // both halves are read before either is reduced: their chains of exchanges overlap
      float v[2][16];
      const int row = o.lane >> 2;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        stage16(st, q, o.lane, a0, a1);
        wave_sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4_t x = *staged(st, row, 4 * side + i);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[q][4 * i + k] = x[k];
        }
        if (at[q] >= 0 && at[q] < 16 && at[q] < n)
          t.hit[o.p0 + row0 + 16 * q + row] = ((const float*)staged(st, row, 4 * side + ((int)at[q] >> 2)))[at[q] & 3];
        wave_sync();
      }
      if (!whole)
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
          for (int q = 0; q < 2; ++q) v[q][i] = i < n ? v[q][i] : -INFINITY;
      float m[2], s[2] = {0.0f, 0.0f}, shift[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        m[q] = v[q][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) m[q] = fmaxf(m[q], v[q][i]);
        m[q] = fmaxf(m[q], quad_xor1(m[q]));
        m[q] = fmaxf(m[q], quad_xor2(m[q]));
        // exp(v - m) = 2^(v log2(e) - m log2(e)); of -inf 0 even where all are
        shift[q] = -fmaxf(m[q], -2e38f) * LOG2E;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) s[q] += __builtin_amdgcn_exp2f(fmaf(v[q][i], LOG2E, shift[q]));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        s[q] += quad_xor1(s[q]);
        s[q] += quad_xor2(s[q]);
        mine[b][q] = float2{m[q], s[q]};
      }
      ++b;
    });
    bar();  // the stages are free
    float2* sums = (float2*)(lds + EPI_AT);  // [wn][256]
    b = 0;
    each_block<RB0, RB1>(o, acc, [&](int row0, const f32x16_t&, const f32x16_t&) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (side == 0) sums[o.wn * TB + row0 + 16 * q + (o.lane >> 2)] = mine[b][q];
      ++b;
    });
    wait_vm<63>();
    bar();
    if (o.tid >= o.rows) return;
    float m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, sums[w * TB + o.tid].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) s += sums[w * TB + o.tid].y * exp_from(sums[w * TB + o.tid].x, m);
    t.part[o.panel * rows + o.p0 + o.tid] = float2{m, s};
  }
};

template <bool CHAIN>
__global__ __launch_bounds__(512, 1) void k_loss_logits(TileArgs p, LseEpi epi) {
  __shared__ u32x4_t lds[10 * HU];
  if constexpr (CHAIN)
    row_chain<OP_NT>(p, lds, epi);
  else
    row_tile<OP_NT, false, GX_ROWS>(p, lds, epi);
}

// Joins the panels of JR rows, 256 / JR threads a row: 16 of many rows, 4 of fewer (257 rows of 126 panels
// 5.6 us with 16, 5.1 so), and 1 where the panels are those of the matrix-vector kernel.
template <int JR>
__global__ __launch_bounds__(256) void k_loss_join(LossTokens a, int64_t rows, int panels, float* loss, float* lse) {
  constexpr int TH = 256 / JR;
  __shared__ float2 lds[TH][JR];
  const int r = threadIdx.x % JR, j = threadIdx.x / JR;
  for (int64_t t0 = (int64_t)blockIdx.x * JR; t0 < rows; t0 += (int64_t)gridDim.x * JR) {
    const int64_t t = t0 + r;
    float m = -INFINITY, s = 0.0f;
    if (t < rows)
      for (int i = j; i < panels; i += TH) {
        const float2 q = a.part[i * rows + t];
        const float b = fmaxf(m, q.x);
        s = s * exp_from(m, b) + q.y * exp_from(q.x, b);
        m = b;
      }
    __syncthreads();  // the rows before have been read
    lds[j][r] = float2{m, s};
    for (int n = TH / 2; n > 0; n >>= 1) {
      __syncthreads();
      if (j < n) {
        const float2 p = lds[j][r], q = lds[j + n][r];
        const float b = fmaxf(p.x, q.x);
        lds[j][r] = float2{b, p.y * exp_from(p.x, b) + q.y * exp_from(q.x, b)};
      }
    }
    if (j != 0 || t >= rows) continue;
    const float l = lds[0][r].x + logf(lds[0][r].y);
    const int64_t g = a.target[t];
    if (lse) lse[t] = l;
    loss[t] = g >= 0 && g < a.V && g != a.ignore ? l - a.hit[t] : 0.0f;
  }
}

// The one of larger magnitude, the positive one of two alike (a NaN never).
__device__ __forceinline__ float larger(float a, float b) {
  return fabsf(b) > fabsf(a) || (fabsf(b) == fabsf(a) && b > a) ? b : a;
}

// scale[t] = d_loss[t], 0 for a token without a target; *most = the one of largest magnitude, with its
// sign, so that a d_loss that all tokens share is 1 of it.
template <int WAVES>
__device__ __forceinline__ float largest(float m, float* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = larger(m, __shfl_xor(m, d, 64));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
  for (int i = 0; i < WAVES; ++i) m = larger(m, lds[i]);
  return m;
}
__global__ __launch_bounds__(1024) void k_loss_scale(LossTokens a, int64_t rows, float* scale, float* most) {
  __shared__ float lds[16];
  float m = 0.0f;
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < rows; t += 1024) {
    const float v = scale_of(a, t);
    scale[t] = v;
    m = larger(m, v);
  }
  m = largest<16>(m, lds);
  if (threadIdx.x == 0) *most = m;
}

// out[t] = x[t] scale[t] / *most; zeros for a token without a part in the gradients.  Up to kFewTokens
// tokens every workgroup finds the largest d_loss itself, which costs less than a launch before it.
constexpr int kFewTokens = 2048;
template <bool FEW>
__global__ __launch_bounds__(256) void k_loss_rows(LossTokens a, const uint16_t* x, int64_t ldx, int64_t rows,
                                                   float* scale, float* most, int H, uint16_t* out) {
  __shared__ float lds[4];
  float m;
  if (FEW) {
    m = 0.0f;
    for (int64_t t = threadIdx.x; t < rows; t += 256) {
      const float v = scale_of(a, t);
      if (blockIdx.x == 0) scale[t] = v;
      m = larger(m, v);
    }
    m = largest<4>(m, lds);
    if (blockIdx.x == 0 && threadIdx.x == 0) *most = m;
  } else {
    m = *most;
  }
  if (!out) return;
  const int64_t n = rows * H;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
    const int64_t t = i / H;
    const float v = FEW ? scale_of(a, t) : scale[t], r = m != 0.0f ? v / m : v;
    const u32x4_t q = *(const u32x4_t*)(x + t * ldx + (i - t * H));
    u32x4_t o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = r != 0.0f ? pack_bf16x2(r * bf16_lo(q[j]), r * bf16_hi(q[j])) : 0u;
    *(u32x4_t*)(out + i) = o;
  }
}

struct GradEpi {
  static constexpr bool kGated = false;
  LossTokens t;

  template <int RB0, int RB1, class ACC>
  __device__ __forceinline__ void tile(const TileArgs& p, const TileOut& o, ACC& acc, u32x4_t* lds) const {
    float* st = (float*)epi_stage(lds, o);
    each_block<RB0, RB1>(o, acc, [&](int row0, const f32x16_t& a0, const f32x16_t& a1) __attribute__((always_inline)) {
      const int chunk = o.lane & 7, col = o.c0 + 64 * o.wn + 8 * chunk;
      const bool whole = o.c0 + TB <= p.g.N;  // uniform
      float l[4], w[4];
      int64_t hit[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row0 + i * 8 + (o.lane >> 3);
        const int64_t grow = o.p0 + (row < o.rows ? row : 0);
        hit[i] = t.target[grow] - t.v0 - col;
        l[i] = -t.lse[grow] * LOG2E;
        w[i] = scale_of(t, grow);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        stage16(st, q, o.lane, a0, a1);
        wave_sync();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = 2 * q + j, row = j * 8 + (o.lane >> 3);
          const f32x4_t x = *staged(st, row, 2 * chunk), y = *staged(st, row, 2 * chunk + 1);
          if (row0 + 16 * q + row >= o.rows || col >= p.g.N) continue;
          // nothing for a token without a part, whatever its logits; columns past the vocabulary, which
          // the products read with the last eight, are zeros
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            v[k] = w[i] != 0.0f ? __builtin_amdgcn_exp2f(fmaf(k < 4 ? x[k & 3] : y[k & 3], LOG2E, l[i])) : 0.0f;
          if (hit[i] >= 0 && hit[i] < 8 && w[i] != 0.0f)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] -= hit[i] == k ? 1.0f : 0.0f;
          if (!whole)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = col + k < p.g.N ? v[k] : 0.0f;
          *(u32x4_t*)(t.d + (o.p0 + row0 + 16 * q + row) * t.ldd + col) =
              u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
        }
        wave_sync();
      }
    });
  }
};

template <bool CHAIN>
__global__ __launch_bounds__(512, 1) void k_loss_grad(TileArgs p, GradEpi epi) {
  __shared__ u32x4_t lds[10 * HU];
  if constexpr (CHAIN)
    row_chain<OP_NT>(p, lds, epi);
  else
    row_tile<OP_NT, false, GX_ROWS>(p, lds, epi);
}

// Adds a tile to what earlier pieces left (add = 0: the first piece).  With dx given (one piece, one slice)
// the tile is dx already: times the token's d_loss and in its type.
struct SumEpi {
  static constexpr bool kGated = false;
  float* out;  // [rows][K] of the slice
  int add;
  void* dx;
  int64_t lddx;
  int dx32;
  const float* scale;

  template <int RB0, int RB1, class ACC>
  __device__ __forceinline__ void tile(const TileArgs& p, const TileOut& o, ACC& acc, u32x4_t* lds) const {
    float* st = (float*)epi_stage(lds, o);
    const int chunk = o.lane & 15, col = o.c0 + 128 * (chunk >> 3) + 32 * o.wn + 4 * (chunk & 7);
    each_block<RB0, RB1>(o, acc, [&](int row0, const f32x16_t& a0, const f32x16_t& a1) __attribute__((always_inline)) {
      f32x4_t was[8];
      bool in[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = row0 + i * 4 + (o.lane >> 4);
        in[i] = row < o.rows && col < p.g.K;
        was[i] = in[i] && add ? *(const f32x4_t*)(out + (o.p0 + row) * p.g.K + col) : f32x4_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        stage16(st, q, o.lane, a0, a1);
        wave_sync();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * q + j, row = j * 4 + (o.lane >> 4);
          if (!in[i]) continue;
          const int64_t grow = o.p0 + row0 + 16 * q + row;
          f32x4_t v = *staged(st, row, chunk);
          if (!dx) {
            *(f32x4_t*)(out + grow * p.g.K + col) = was[i] + v;
            continue;
          }
          const float a = scale[grow];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] *= a;
          if (dx32)
            *(f32x4_t*)((float*)dx + grow * lddx + col) = v;
          else
            *(uint2*)((uint16_t*)dx + grow * lddx + col) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
        wave_sync();
      }
    });
  }
};

// Both products of a piece in one launch: the tiles of dw fill the compute units that dx's, which are
// longer, leave.  dx: units (slice, row tile, panel) in eight equal runs, one for each XCD, whose L2 then
// serves a slice's rows of d and w again.
struct LossTiles {
  TileArgs dx, dw;
  SumEpi sum;
  int dx_units;  // a multiple of 8
  int slice, slices, row_tiles;
};
template <class EPI>
__global__ __launch_bounds__(512, 1) void k_loss_products(LossTiles a) {
  __shared__ u32x4_t lds[10 * HU];
  const int b = blockIdx.x;
  if (b >= a.dx_units) {
    wgrad_tile<GX_ROWS, EPI>(a.dw, b - a.dx_units, lds);
    return;
  }
  TileArgs p = a.dx;
  const int per = a.row_tiles * p.npan, all = a.slices * per, run = a.dx_units / 8, unit = (b & 7) * run + (b >> 3);
  if (unit >= all) return;
  const int slice = unit / per, tile = unit - slice * per, n0 = slice * a.slice;
  if (n0 >= p.g.N) return;  // the last piece has fewer
  p.a += (int64_t)n0 * 2;
  p.b += (int64_t)n0 * p.g.K * 2;
  p.g.N = p.g.N - n0 < a.slice ? p.g.N - n0 : a.slice;
  SumEpi sum = a.sum;
  sum.out += (int64_t)slice * p.g.rows * p.g.K;
  const int64_t p0 = (int64_t)(tile / p.npan) * TB;
  const int rows = (int)(p.g.rows - p0 < TB ? p.g.rows - p0 : TB);
  const TileJob job{0, p0, rows, 0, 0, tile % p.npan};
  if (rows > 128)
    tile_product<OP_NN, false, 2, 2, GX_ROWS, false, SumEpi>(p, job, lds, nullptr, sum);
  else if (rows > 64)
    tile_product<OP_NN, false, 2, 0, GX_ROWS, false, SumEpi>(p, job, lds, nullptr, sum);
  else
    tile_product<OP_NN, false, 1, 0, GX_ROWS, false, SumEpi>(p, job, lds, nullptr, sum);
}

// dx = the sum of its slices, times the token's d_loss.
__global__ __launch_bounds__(256) void k_loss_dx_sum(const float* part, int slices, int64_t n, int K, int64_t ldx,
                                                     const float* scale, void* dx, int fp32) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
    float v[8] = {};
    for (int s = 0; s < slices; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t q = *(const f32x4_t*)(part + s * n + i + 4 * h);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * h + k] += q[k];
      }
    const int64_t t = i / K, at = t * ldx + (i - t * K);
    const float a = scale[t];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= a;
    if (fp32) {
      *(f32x4_t*)((float*)dx + at) = f32x4_t{v[0], v[1], v[2], v[3]};
      *(f32x4_t*)((float*)dx + at + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
      *(u32x4_t*)((uint16_t*)dx + at) = u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
  }
}

// One launch of row tiles of one group.
template <class F, class EPI>
hipError_t launch_rows(const Launch& lc, F chained, F single, const TileArgs& t, const EPI& epi) {
  const int64_t units = row_tile_units(t.g, t.npan);
  if (takes_chain(t.g, units)) return launch(lc, chained, dim3((unsigned)kChainGroups), dim3(512), t, epi);
  return launch(lc, single, dim3((unsigned)units), dim3(512), t, epi);
}

Groups one_matrix(int64_t rows, int64_t ldx, int64_t ldy, int N, int K) {
  return Groups{rows, rows, ldx, ldy, 1, N, K, 1, nullptr, nullptr};
}

constexpr size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

static int loss_panels(int64_t rows, int V) {
  const int w = takes_matrix_vector_logits(rows, V) ? kSkinnyColumns : TB;
  return (V + w - 1) / w;
}

size_t loss_workspace(int64_t rows, int V) {
  return align256((size_t)loss_panels(rows, V) * rows * sizeof(float2)) + align256((size_t)rows * 4);
}

static LossTokens loss_tokens(const LossArgs& a) {
  LossTokens t{};
  t.target = a.target;
  t.ignore = a.ignore;
  t.V = a.V;
  t.lse = a.lse;
  t.d_loss = a.d_loss;
  return t;
}

hipError_t launch_loss(const LossArgs& a, void* workspace, hipStream_t s) {
  const int panels = loss_panels(a.rows, a.V);
  LossTokens tokens = loss_tokens(a);
  tokens.part = (float2*)workspace;
  tokens.hit = (float*)((char*)workspace + align256((size_t)panels * a.rows * sizeof(float2)));
  const Launch lc{s, nullptr, nullptr};
  TileArgs t{};
  t.g = one_matrix(a.rows, a.ldx, a.V, a.V, a.H);
  t.a = (const char*)a.x;
  t.b = (const char*)a.w;
  t.npan = panels;
  set_row_tiles(&t);
  const bool few = takes_matrix_vector_logits(a.rows, a.V);
  const hipError_t e = few ? launch_loss_skinny(t.g, a.x, a.w, tokens, false, s)
                           : launch_rows(lc, k_loss_logits<true>, k_loss_logits<false>, t, LseEpi{tokens, a.rows});
  if (e != hipSuccess) return e;
  const int each = few ? 1 : a.rows <= 2048 ? 4 : 16;
  const int64_t joins = (a.rows + each - 1) / each;
  return launch(lc, each == 1 ? k_loss_join<1> : each == 4 ? k_loss_join<4> : k_loss_join<16>, dim3((unsigned)(joins < (1 << 20) ? joins : 1 << 20)),
                dim3(256), tokens, a.rows, panels, a.loss, a.lse_out);
}

LossPlan loss_plan(int64_t rows, int V, int H) {
  LossPlan p;
  const int64_t all = (V + TB - 1) / TB * (int64_t)TB, most = kLossPieceBytes / 2 / (rows < 1 ? 1 : rows) / TB * TB;
  p.piece = (int)(most >= all ? all : most < kLossPieceColumns ? (kLossPieceColumns < all ? kLossPieceColumns : all) : most);
  const int first = p.piece < V ? p.piece : V;  // columns of the first piece
  const int64_t tiles = (rows < 1 ? 1 : (rows + TB - 1) / TB) * ((H + TB - 1) / TB);
  const int64_t pieces = (V + p.piece - 1) / p.piece;
  const int64_t units = ((first + TB - 1) / TB) * (int64_t)((H + TB - 1) / TB);  // tiles of dw
  const int64_t dx_size = rows * H * 4, dw_size = (int64_t)first * H * 4;
  // Slices of dx and parts of dw: those with which a piece's launch takes least (launch_steps), three
  // calls with dw to one without it (dx does not depend on whether dw is asked for).  Slices are written,
  // from the second piece on read too, and added up at the end.  Both gradients / dx alone in us with 1, 2,
  // 4, 8 and 16 slices: 200 tokens x 64000 columns of 2048 1171 / 1026, 674 / 570, 430 / 331, 293 / 216, 276
  // / 169; 999 x 32000 of 2048 666 / 623, 457 / 402, 369 / 289, 386 / 251, 421 / 279; 2000 x 32000 of 2048
  // 863 / 773, 713 / 557, 706 / 473, 739 / 496, 796 / 551; 4096 x 65536 of 2048 2709 / 2217, 2703 / 1862,
  // 2750 / 1896, 2852 / 1998, 3035 / 2179; 6000 x 32000 of 2048 1993 / 1440, 2259 / 1693, 2378 / 1681, 2495
  // / 1807, 2745 / 2050; with 1, 2, 4, 8 and 16 parts: 16000 x 1000 of 512 311, 189, 128, 100, 97.
  p.slices = p.splits = 1;
  int64_t least = 0;
  for (int n = 1; n <= 32 && (n == 1 || (first / n >= 128 && tiles * n <= kMostTiles)); n = next_parts(n)) {
    const int64_t steps = ((first + n - 1) / n + 63) / 64 + kTileSteps;
    const bool direct = n == 1 && pieces == 1;
    const int64_t sums = direct ? 0 : (pieces == 1 ? 1 : 2) * n * dx_size / kStepBytes;
    const int64_t alone = pieces * (launch_steps(tiles * n, steps, 0, 0) + sums) +
                          4 * (direct ? 0 : kLaunchSteps + n * dx_size / kStepBytes);
    for (int m = 1; m == 1 || (m <= rows / 256 && units * m <= kMostTiles); m = next_parts(m)) {
      const int64_t both = launch_steps(tiles * n, steps, units * m, rows / (64 * m) + kTileSteps) + sums +
                           (m > 1 ? kLaunchSteps + 2 * m * dw_size / kStepBytes : 0);
      const int64_t t = alone + 3 * pieces * both;
      if ((n == 1 && m == 1) || t < least) p.slices = n, p.splits = m, least = t;
    }
  }
  p.slice = ((first + p.slices - 1) / p.slices + 63) / 64 * 64;
  p.slices = (first + p.slice - 1) / p.slice;  // none of the first piece's is empty
  p.d_bytes = align256((size_t)rows * p.piece * 2);
  p.part_bytes = align256((size_t)p.slices * rows * H * 4);
  p.x_bytes = align256((size_t)rows * H * 2);
  p.dw_bytes = p.splits > 1 ? align256((size_t)p.splits * first * H * 4) : 0;
  p.bytes = p.d_bytes + p.part_bytes + p.x_bytes + p.dw_bytes + align256((size_t)rows * 4) + 256;
  return p;
}

hipError_t launch_loss_grad(const LossArgs& a, void* workspace, hipStream_t s) {
  const LossPlan plan = loss_plan(a.rows, a.V, a.H);
  uint16_t* d = (uint16_t*)workspace;
  float* part = (float*)((char*)workspace + plan.d_bytes);
  uint16_t* x = (uint16_t*)((char*)part + plan.part_bytes);
  float* dw_part = (float*)((char*)x + plan.x_bytes);
  float* most = (float*)((char*)dw_part + plan.dw_bytes);
  float* scale = most + 64;
  const Launch lc{s, nullptr, nullptr};
  const int64_t total = a.rows * a.H, groups = (total / 8 + 255) / 256;
  const dim3 each((unsigned)(groups < 1024 ? groups : 1024));
  LossTokens tokens = loss_tokens(a);
  tokens.d = d;
  tokens.ldd = plan.piece;
  if (a.rows > 0) {
    const bool few = a.rows <= kFewTokens;
    hipError_t e = hipSuccess;
    if (!few) e = launch(lc, k_loss_scale, dim3(1), dim3(1024), tokens, a.rows, scale, most);
    if (e == hipSuccess && (few || a.dw))
      e = launch(lc, few ? k_loss_rows<true> : k_loss_rows<false>, few && !a.dw ? dim3(1) : each, dim3(256), tokens,
                 (const uint16_t*)a.x, a.ldx, a.rows, scale, most, a.H, a.dw ? x : nullptr);
    if (e != hipSuccess) return e;
  }
  const bool direct = plan.slices == 1 && plan.piece >= a.V;
  for (int64_t v0 = 0; v0 < a.V; v0 += plan.piece) {
    const int n = (int)(a.V - v0 < plan.piece ? a.V - v0 : plan.piece);
    const char* w = (const char*)a.w + v0 * a.H * 2;
    TileArgs t{};
    t.g = one_matrix(a.rows, a.ldx, plan.piece, n, a.H);
    t.a = (const char*)a.x;
    t.b = w;
    t.npan = (n + TB - 1) / TB;
    set_row_tiles(&t);
    hipError_t e = hipSuccess;
    if (a.rows > 0) {
      tokens.v0 = (int)v0;
      e = takes_matrix_vector_logits(a.rows, n) ? launch_loss_skinny(t.g, a.x, w, tokens, true, s)
                                : launch_rows(lc, k_loss_grad<true>, k_loss_grad<false>, t, GradEpi{tokens});
      if (e != hipSuccess) return e;
    }
    LossTiles f{};
    f.dx = t;
    f.dx.a = (const char*)d;
    f.dx.npan = (a.H + TB - 1) / TB;
    f.sum = SumEpi{part, v0 > 0, direct ? a.dx : nullptr, a.lddx, (int)a.dx32, scale};
    f.slice = plan.slice;
    f.slices = plan.slices;
    f.row_tiles = (int)((a.rows + TB - 1) / TB);
    if (a.dx) f.dx_units = (plan.slices * f.row_tiles * f.dx.npan + 7) / 8 * 8;
    f.dw = t;
    f.dw.g.ldx = a.H;
    f.dw.a = (const char*)d;
    f.dw.b = (const char*)x;
    f.dw.nrow = (n + TB - 1) / TB;
    f.dw.npan = f.dx.npan;
    f.dw.splits = plan.splits;
    f.dw.factor = most;
    void* dw = a.dw ? (char*)a.dw + v0 * a.H * (a.dw32 ? 4 : 2) : nullptr;
    f.dw.out = plan.splits > 1 ? dw_part : dw;
    f.dw.fp32 = plan.splits > 1 || a.dw32;
    const int64_t units = f.dx_units + (a.dw ? wgrad_units(f.dw.g, plan.splits) : 0);
    // the factor comes with the sum of the parts, and where there are no tokens there is none
    e = launch(lc, plan.splits > 1 || a.rows == 0 ? k_loss_products<StoreEpi> : k_loss_products<ScaledEpi>,
               dim3((unsigned)units), dim3(512), f);
    if (e == hipSuccess && a.dw && plan.splits > 1)
      e = launch_sum_parts(plan.splits, SumOf{dw_part, (int64_t)n * a.H, dw}, SumOf{}, most, a.dw32, s);
    if (e != hipSuccess) return e;
  }
  if (!a.dx || a.rows == 0 || direct) return hipSuccess;
  return launch(lc, k_loss_dx_sum, each, dim3(256), (const float*)part, plan.slices, total, a.H, a.lddx,
                (const float*)scale, a.dx, (int)a.dx32);
}

}  // namespace moe
