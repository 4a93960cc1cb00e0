// Softmax cross entropy against a vocabulary (gfx950, wave64, MFMA):
//   z = x W^T (never stored),  lse[t] = log sum_v exp z[t][v],  loss[t] = lse[t] - z[t][target[t]]
//   d[t][v] = exp(z[t][v] - lse[t]) - (v == target[t]),  dx = d_loss d W,  dW = (d_loss d)^T x
// on the tiles of the grouped products (ops_tile.h).
//
// Forward: every 256 x 256 tile of z is reduced in its epilogue to a maximum
// and a sum of exponentials for each row, 8 bytes where z has 1024; a second
// launch joins the panels of a row.  Gradients: the vocabulary goes by in
// pieces; a piece's z is computed again (the same sums in the same order as in
// the forward call), becomes d in bf16 in the epilogue, and d feeds the two
// gradient products of the piece while it is still in the last-level cache.
// dx is summed over the pieces in fp32; where its tiles are too few for the
// chip, a piece's reduction is cut into slices with sums of their own, which
// the last launch adds in a fixed order.
//
// d is rounded to bf16 without the token's d_loss: the mean's 1 / n is the same
// for all of them and so would be its rounding, an error of up to 2^-8 of whole
// gradients (dx and dW of 999 tokens were off by 0.28% of their norm; now 0.23%,
// of which 0.17% is the rounding of the results).  dx takes d_loss in fp32 with
// its last sum; dW takes the largest d_loss in its epilogue, and the token's
// share of that, exactly 1 for a mean, into the bf16 copy of x that it reads.
#include "ops_tile.h"

namespace moe {
namespace {

constexpr int ST_LD = 68;  // floats from a staged row to the next: rows 16 bytes of banks apart

// 32 x 64 results of a wave, columns 0..31 of its block of the first column half, 32..63 of the second.
__device__ __forceinline__ void stage_block(float* st, int ld, const TileOut& o, const f32x16_t& a0, const f32x16_t& a1) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int at = block_row(r, o.lane) * ld + (o.lane & 31);
    st[at] = a0[r];
    st[at + 32] = a1[r];
  }
}

// exp(x - m), 0 where both are -inf.
__device__ __forceinline__ float exp_from(float x, float m) { return x == -INFINITY ? 0.0f : __expf(x - m); }

struct LseEpi {
  static constexpr bool kGated = false;
  const int64_t* target;
  int64_t rows;   // of all tiles
  float2* part;   // [panel][rows] maximum, sum of exp(z - maximum)
  float* hit;     // [rows] z at the target, where a tile has it

  template <int RB0, int RB1, class ACC>
  __device__ __forceinline__ void tile(const TileArgs& p, const TileOut& o, ACC& acc, u32x4_t* lds) const {
    float* st = (float*)lds + o.wave * (32 * ST_LD);
    float2* sums = (float2*)((float*)lds + 8 * 32 * ST_LD);  // [wn][256]
    const int side = o.lane & 1;                             // two lanes a row: one for each column half
    const int col = o.c0 + 64 * o.wn + 32 * side, n = p.g.N - col;
    each_block<RB0, RB1>(o, acc, [&](int row0, const f32x16_t& a0, const f32x16_t& a1) {
      const int row = row0 + (o.lane >> 1);
      const bool in = row < o.rows;
      const int64_t t = in ? target[o.p0 + row] - col : -1;
      stage_block(st, ST_LD, o, a0, a1);
      wave_sync();
      const float* at = st + (o.lane >> 1) * ST_LD + 32 * side;
      float v[32];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const f32x4_t q = *(const f32x4_t*)(at + 4 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * i + k] = 4 * i + k < n ? q[k] : -INFINITY;
      }
      if (t >= 0 && t < 32 && t < n) hit[o.p0 + row] = at[t];
      float m = v[0];
#pragma unroll
      for (int i = 1; i < 32; ++i) m = fmaxf(m, v[i]);
      m = fmaxf(m, __shfl_xor(m, 1, 64));
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) s += exp_from(v[i], m);
      s += __shfl_xor(s, 1, 64);
      if (side == 0) sums[o.wn * TB + row] = float2{m, s};
      wave_sync();
    });
    __syncthreads();
    if (o.tid >= o.rows) return;
    float m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, sums[w * TB + o.tid].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) s += sums[w * TB + o.tid].y * exp_from(sums[w * TB + o.tid].x, m);
    part[o.panel * rows + o.p0 + o.tid] = float2{m, s};
  }
};

__global__ __launch_bounds__(512, 1) void k_loss_logits(TileArgs p, LseEpi epi) {
  __shared__ u32x4_t lds[10 * HU];
  row_tile<OP_NT, false, GX_ROWS>(p, lds, epi);
}

// Joins the panels of 16 rows, 16 threads a row.
constexpr int JR = 16;
__global__ __launch_bounds__(JR * 16) void k_loss_join(const float2* part, const float* hit, const int64_t* target,
                                                       int64_t ignore, int64_t rows, int panels, int V, float* loss,
                                                       float* lse) {
  __shared__ float2 lds[16][JR];
  const int r = threadIdx.x % JR, j = threadIdx.x / JR;
  for (int64_t t0 = (int64_t)blockIdx.x * JR; t0 < rows; t0 += (int64_t)gridDim.x * JR) {
    const int64_t t = t0 + r;
    float m = -INFINITY, s = 0.0f;
    if (t < rows)
      for (int i = j; i < panels; i += 16) {
        const float2 q = part[i * rows + t];
        const float b = fmaxf(m, q.x);
        s = s * exp_from(m, b) + q.y * exp_from(q.x, b);
        m = b;
      }
    __syncthreads();  // the rows before have been read
    lds[j][r] = float2{m, s};
    __syncthreads();
    if (j != 0 || t >= rows) continue;
    for (int i = 1; i < 16; ++i) m = fmaxf(m, lds[i][r].x);
    s = 0.0f;
    for (int i = 0; i < 16; ++i) s += lds[i][r].y * exp_from(lds[i][r].x, m);
    const float l = m + logf(s);
    const int64_t g = target[t];
    if (lse) lse[t] = l;
    loss[t] = g >= 0 && g < V && g != ignore ? l - hit[t] : 0.0f;
  }
}

// The one of larger magnitude, the positive one of two alike (a NaN never).
__device__ __forceinline__ float larger(float a, float b) {
  return fabsf(b) > fabsf(a) || (fabsf(b) == fabsf(a) && b > a) ? b : a;
}

// scale[t] = d_loss[t], 0 for a token without a target; *most = the one of largest magnitude, with its
// sign, so that a d_loss that all tokens share is 1 of it.
__global__ __launch_bounds__(1024) void k_loss_scale(const float* d_loss, const int64_t* target, int64_t ignore, int V,
                                                     int64_t rows, float* scale, float* most) {
  __shared__ float lds[16];
  float m = 0.0f;
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < rows; t += 1024) {
    const int64_t g = target[t];
    const float a = g >= 0 && g < V && g != ignore ? d_loss[t] : 0.0f;
    scale[t] = a;
    m = larger(m, a);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = larger(m, __shfl_xor(m, d, 64));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < 16; ++i) m = larger(m, lds[i]);
  *most = m;
}

// out[t] = x[t] scale[t] / *most; zeros for a token without a part in the gradients.
__global__ __launch_bounds__(256) void k_loss_rows(const uint16_t* x, int64_t ldx, const float* scale, const float* most,
                                                   int64_t n, int H, uint16_t* out) {
  const float m = *most;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
    const int64_t t = i / H;
    const float a = scale[t], r = m != 0.0f ? a / m : a;
    const u32x4_t q = *(const u32x4_t*)(x + t * ldx + (i - t * H));
    u32x4_t o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = r != 0.0f ? pack_bf16x2(r * bf16_lo(q[j]), r * bf16_hi(q[j])) : 0u;
    *(u32x4_t*)(out + i) = o;
  }
}

struct GradEpi {
  static constexpr bool kGated = false;
  const int64_t* target;
  int v0;  // first column of the piece
  const float* lse;
  const float* scale;  // 0: the token has no part
  uint16_t* d;         // [rows][ldd]
  int64_t ldd;

  template <int RB0, int RB1, class ACC>
  __device__ __forceinline__ void tile(const TileArgs& p, const TileOut& o, ACC& acc, u32x4_t* lds) const {
    float* st = (float*)lds + o.wave * (32 * ST_LD);
    each_block<RB0, RB1>(o, acc, [&](int row0, const f32x16_t& a0, const f32x16_t& a1) {
      float l[4], w[4];
      int64_t t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row0 + i * 8 + (o.lane >> 3);
        const int64_t grow = o.p0 + (row < o.rows ? row : 0);
        t[i] = target[grow];
        l[i] = lse[grow];
        w[i] = scale[grow];
      }
      stage_block(st, ST_LD, o, a0, a1);
      wave_sync();
      const int at = (o.lane & 7) * 8, col = o.c0 + 64 * o.wn + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i * 8 + (o.lane >> 3);
        const f32x4_t* s = (const f32x4_t*)(st + row * ST_LD + at);
        const f32x4_t x = s[0], y = s[1];
        if (row0 + row >= o.rows || col >= p.g.N) continue;
        const int64_t hit = t[i] - v0 - col;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float e = __expf((k < 4 ? x[k & 3] : y[k & 3]) - l[i]);
          // nothing for a token without a part, whatever its logits; columns past the vocabulary, which
          // the products read with the last eight, are zeros
          v[k] = w[i] != 0.0f && col + k < p.g.N ? (hit == k ? e - 1.0f : e) : 0.0f;
        }
        *(u32x4_t*)(d + (o.p0 + row0 + row) * ldd + col) = u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
      }
      wave_sync();
    });
  }
};

__global__ __launch_bounds__(512, 1) void k_loss_grad(TileArgs p, GradEpi epi) {
  __shared__ u32x4_t lds[10 * HU];
  row_tile<OP_NT, false, GX_ROWS>(p, lds, epi);
}

// Adds a tile to what earlier pieces left (add = 0: the first piece).
struct SumEpi {
  static constexpr bool kGated = false;
  float* out;  // [rows][K] of the slice
  int add;

  template <int RB0, int RB1, class ACC>
  __device__ __forceinline__ void tile(const TileArgs& p, const TileOut& o, ACC& acc, u32x4_t* lds) const {
    float* st = (float*)lds + o.wave * (32 * ST_LD);
    const int at = (o.lane & 15) * 4, col = o.c0 + 128 * (at >> 5) + 32 * o.wn + (at & 31);
    each_block<RB0, RB1>(o, acc, [&](int row0, const f32x16_t& a0, const f32x16_t& a1) {
      f32x4_t was[8];
      bool in[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = row0 + i * 4 + (o.lane >> 4);
        in[i] = row < o.rows && col < p.g.K;
        was[i] = in[i] && add ? *(const f32x4_t*)(out + (o.p0 + row) * p.g.K + col) : f32x4_t{0, 0, 0, 0};
      }
      stage_block(st, ST_LD, o, a0, a1);
      wave_sync();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = i * 4 + (o.lane >> 4);
        const f32x4_t v = *(const f32x4_t*)(st + row * ST_LD + at);
        if (in[i]) *(f32x4_t*)(out + (o.p0 + row0 + row) * p.g.K + col) = was[i] + v;
      }
      wave_sync();
    });
  }
};

// One slice of a piece's reduction a workgroup row.
__global__ __launch_bounds__(512, 1) void k_loss_dx(TileArgs p, SumEpi epi, int slice) {
  __shared__ u32x4_t lds[10 * HU];
  const int n0 = (int)blockIdx.y * slice;
  if (n0 >= p.g.N) return;
  p.a += (int64_t)n0 * 2;
  p.b += (int64_t)n0 * p.g.K * 2;
  p.g.N = p.g.N - n0 < slice ? p.g.N - n0 : slice;
  epi.out += (int64_t)blockIdx.y * p.g.rows * p.g.K;
  row_tile<OP_NN, false, GX_ROWS>(p, lds, epi);
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

Groups one_matrix(int64_t rows, int64_t ldx, int64_t ldy, int N, int K) {
  return Groups{rows, rows, ldx, ldy, 1, N, K, 1, nullptr, nullptr};
}

constexpr size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t loss_workspace(int64_t rows, int V) {
  const int panels = (V + TB - 1) / TB;
  return align256((size_t)panels * rows * sizeof(float2)) + align256((size_t)rows * 4);
}

hipError_t launch_loss(const LossArgs& a, void* workspace, hipStream_t s) {
  const int panels = (a.V + TB - 1) / TB;
  float2* part = (float2*)workspace;
  float* hit = (float*)((char*)workspace + align256((size_t)panels * a.rows * sizeof(float2)));
  TileArgs t{};
  t.g = one_matrix(a.rows, a.ldx, a.V, a.V, a.H);
  t.a = (const char*)a.x;
  t.b = (const char*)a.w;
  t.npan = panels;
  const Launch lc{s, nullptr, nullptr};
  hipError_t e = launch(lc, k_loss_logits, dim3((unsigned)row_tile_units(t.g, panels)), dim3(512), t,
                        LseEpi{a.target, a.rows, part, hit});
  if (e != hipSuccess) return e;
  const int64_t joins = (a.rows + JR - 1) / JR;
  return launch(lc, k_loss_join, dim3((unsigned)(joins < (1 << 20) ? joins : 1 << 20)), dim3(JR * 16), (const float2*)part,
                (const float*)hit, a.target, a.ignore, a.rows, panels, a.V, a.loss, a.lse_out);
}

LossPlan loss_plan(int64_t rows, int V, int H) {
  LossPlan p;
  const int64_t all = (V + TB - 1) / TB * (int64_t)TB, most = kLossPieceBytes / 2 / (rows < 1 ? 1 : rows) / TB * TB;
  p.piece = (int)(most >= all ? all : most < kLossPieceColumns ? (kLossPieceColumns < all ? kLossPieceColumns : all) : most);
  const int first = p.piece < V ? p.piece : V;  // columns of the first piece
  const int64_t tiles = (rows + TB - 1) / TB * ((H + TB - 1) / TB);
  // slices: the fewest that fill the chip's 256 workgroups best, of at least 512 columns each
  p.slices = 1;
  double best = 1e30;
  for (int n = 1; n <= 32 && (n == 1 || first / n >= 512); ++n) {
    const double waves = (double)((tiles * n + 255) / 256) / n + 0.01 * n;
    if (waves < best) best = waves, p.slices = n;
  }
  p.slice = ((first + p.slices - 1) / p.slices + 63) / 64 * 64;
  p.slices = (first + p.slice - 1) / p.slice;  // none of the first piece's is empty
  p.d_bytes = align256((size_t)rows * p.piece * 2);
  p.part_bytes = align256((size_t)p.slices * rows * H * 4);
  p.x_bytes = align256((size_t)rows * H * 2);
  p.bytes = p.d_bytes + p.part_bytes + p.x_bytes + align256((size_t)rows * 4) + 256;
  return p;
}

hipError_t launch_loss_grad(const LossArgs& a, void* workspace, hipStream_t s) {
  const LossPlan plan = loss_plan(a.rows, a.V, a.H);
  uint16_t* d = (uint16_t*)workspace;
  float* part = (float*)((char*)workspace + plan.d_bytes);
  uint16_t* x = (uint16_t*)((char*)part + plan.part_bytes);
  float* most = (float*)((char*)x + plan.x_bytes);
  float* scale = most + 64;
  const Launch lc{s, nullptr, nullptr};
  const int64_t total = a.rows * a.H, groups = (total / 8 + 255) / 256;
  const dim3 each((unsigned)(groups < 8192 ? groups : 8192));
  if (a.rows > 0) {
    hipError_t e = launch(lc, k_loss_scale, dim3(1), dim3(1024), a.d_loss, a.target, a.ignore, a.V, a.rows, scale, most);
    if (e == hipSuccess && a.dw)
      e = launch(lc, k_loss_rows, each, dim3(256), (const uint16_t*)a.x, a.ldx, (const float*)scale, (const float*)most,
                 total, a.H, x);
    if (e != hipSuccess) return e;
  }
  for (int64_t v0 = 0; v0 < a.V; v0 += plan.piece) {
    const int n = (int)(a.V - v0 < plan.piece ? a.V - v0 : plan.piece);
    const char* w = (const char*)a.w + v0 * a.H * 2;
    TileArgs t{};
    t.g = one_matrix(a.rows, a.ldx, plan.piece, n, a.H);
    t.a = (const char*)a.x;
    t.b = w;
    t.npan = (n + TB - 1) / TB;
    hipError_t e = hipSuccess;
    if (a.rows > 0) {
      e = launch(lc, k_loss_grad, dim3((unsigned)row_tile_units(t.g, t.npan)), dim3(512), t,
                 GradEpi{a.target, (int)v0, a.lse, scale, d, (int64_t)plan.piece});
      if (e != hipSuccess) return e;
    }
    if (a.dx && a.rows > 0) {
      TileArgs u = t;
      u.a = (const char*)d;
      u.npan = (a.H + TB - 1) / TB;
      e = launch(lc, k_loss_dx, dim3((unsigned)row_tile_units(u.g, u.npan), (unsigned)plan.slices), dim3(512), u,
                 SumEpi{part, v0 > 0}, plan.slice);
      if (e != hipSuccess) return e;
    }
    if (a.dw) {
      Groups g = t.g;
      g.ldx = a.H;
      e = launch_op_tile(OP_TN, false, g, d, x, Scales{}, (char*)a.dw + v0 * a.H * (a.dw32 ? 4 : 2), a.dw32, s,
                         a.rows > 0 ? most : nullptr);
      if (e != hipSuccess) return e;
    }
  }
  if (!a.dx || a.rows == 0) return hipSuccess;
  return launch(lc, k_loss_dx_sum, each, dim3(256), (const float*)part, plan.slices, total, a.H, a.lddx,
                (const float*)scale, a.dx, (int)a.dx32);
}

}  // namespace moe
