// Backward pass of a gated feed-forward block for few rows (gfx950, wave64):
// bound by the weights read and the gradients written, not by the products.
//   dh[p] = dy[p] W_d,  (d[p], h[p]) from dh and the kept products     k_few_gate
//   dx[p] = d[p] W_gu,  dW_gu = d^T x[row],  dW_d = dy^T h             k_few_products
// A matrix tile would wait for its whole reduction with one row in 64 at work.
// Here a row's product with a matrix is spread over all of the chip: a
// workgroup takes 128 columns (16 lanes of 16 bytes) and 64 rows of the matrix
// at a time, whose sums meet in LDS in a fixed order.  A weight gradient is an
// outer product for each row of the group, in registers, and is written once.
// d and h stay fp32 between the two launches: with few rows their roundings
// would not average out.
//
// One row and one expert of 512 x 2048: 15.6 us (tiles 40); in a trace k_few_gate 9.2, four workgroups of which each goes
// through 2048 rows of 256 bytes, and k_few_products 7.1.  8 rows over 8 experts of 1024 x 2048: 44 us (68), in a trace
// 14.1 + 34.2; 32 rows 14.6 + 46.7, all of them of one expert 14.2 + 47.7.  22 x 2 over 182 of 1016 x 400, most of them
// without rows: the gradients' 444 MB.
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int FT = 1024;               // threads
constexpr int FC = 128;                // columns of a row's product
constexpr int FN = 64, FK = 512;       // rows and columns of a weight gradient's tile

// The expert of row p; -1: none.
__device__ __forceinline__ int expert_of(const Groups& g, int64_t p) {
  if (!g.offsets) return 0;
  const int lane = threadIdx.x & 63;
  int e = 0;
  for (int i = 0; i < g.E; i += 64)
    e += __builtin_popcountll(__ballot(i + lane < g.E && g.offsets[i + lane < g.E ? i + lane + 1 : g.E] <= p));
  e = __builtin_amdgcn_readfirstlane(e);
  if (e >= g.E) return -1;
  const Range r = group_range(g, e);
  return r.lo <= p && p < r.hi ? e : -1;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void eight(const uint16_t* p, float (&f)[8]) {
  const u32x4_t q = *(const u32x4_t*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(q[i]), f[2 * i + 1] = bf16_hi(q[i]);
}
__device__ __forceinline__ void eight(const float* p, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = ((const f32x4_t*)p)[i >> 2][i & 3];
}

// sum over j < n of v[j] w[j][c0 + t], for the threads t < 128 (columns past `cols`: 0)
template <class V>
__device__ __forceinline__ float row_product(const V* v, const uint16_t* w, int n, int cols, int c0, float (*lds)[FC]) {
  constexpr int U = 8, SLOTS = FT / (FC / 8);
  const int at = threadIdx.x % (FC / 8), slot = threadIdx.x / (FC / 8), c = c0 + 8 * at;
  float acc[8] = {};
  if (c < cols)
    for (int j0 = slot; j0 < n; j0 += U * SLOTS) {
      u32x4_t q[U];
      float a[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * SLOTS;
        q[u] = u32x4_t{0, 0, 0, 0};
        a[u] = 0.0f;
        if (j < n) {
          q[u] = *(const u32x4_t*)(w + (int64_t)j * cols + c);
          a[u] = to_float(v[j]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2 * i] = fmaf(a[u], bf16_lo(q[u][i]), acc[2 * i]);
          acc[2 * i + 1] = fmaf(a[u], bf16_hi(q[u][i]), acc[2 * i + 1]);
        }
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    acc[i] += __shfl_xor(acc[i], 16, 64);
    acc[i] += __shfl_xor(acc[i], 32, 64);
  }
  if ((threadIdx.x & 63) < FC / 8)
#pragma unroll
    for (int i = 0; i < 8; ++i) lds[threadIdx.x >> 6][8 * at + i] = acc[i];
  __syncthreads();
  float s = 0.0f;
  if (threadIdx.x < FC)
#pragma unroll
    for (int k = 0; k < FT / 64; ++k) s += lds[k][threadIdx.x];
  return s;
}

struct FewArgs {
  Groups g;  // of x and w_gate_up: N = 2 I
  int I, H;
  const uint16_t *dy, *x, *w_gate_up, *w_down, *pre;
  int64_t ld_dy, ldp, ld_dx;
  float *d, *h;  // [rows][2 I], [rows][I]
  uint16_t* dx;
  void *dw_gate_up, *dw_down;
  int dw32;
  int dx_units, gu_units;
};

__global__ __launch_bounds__(FT) void k_few_gate(FewArgs a) {
  __shared__ float lds[FT / 64][FC];
  const int64_t p = blockIdx.y;
  const int e = expert_of(a.g, p), c = blockIdx.x * FC + threadIdx.x;
  if (e < 0) return;
  const float dh = row_product(a.dy + p * a.ld_dy, a.w_down + (int64_t)e * a.H * a.I, a.H, a.I, blockIdx.x * FC, lds);
  if (threadIdx.x >= FC || c >= a.I) return;
  const float z = to_float(a.pre[p * a.ldp + c]), u = to_float(a.pre[p * a.ldp + a.I + c]);
  // sigmoid(z) and sigmoid(-z) from exp(-|z|): neither is formed as a difference
  const float x = __expf(-fabsf(z)), q = __builtin_amdgcn_rcpf(1.0f + x);
  const float s = z >= 0.0f ? q : x * q, t = z >= 0.0f ? x * q : q;
  a.d[p * 2 * a.I + c] = dh * u * (s * (1.0f + z * t));
  a.d[p * 2 * a.I + a.I + c] = dh * (z * s);
  a.h[p * a.I + c] = z * s * u;
}

// dw[n][k] = sum over the group's rows of a[p][n] b[row(p)][k]: 64 x 512 of them, a wave four n, a lane eight k
template <class A, class B, bool GATHER>
__device__ __forceinline__ void outer(const FewArgs& f, int unit, const A* a, int64_t lda, int N, const B* b, int64_t ldb,
                                      int K, void* dw) {
  const int npan = (K + FK - 1) / FK, nrow = (N + FN - 1) / FN, e = unit / (npan * nrow), tile = unit - e * npan * nrow;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = tile / npan * FN + wave * 4, k = tile % npan * FK + (threadIdx.x & 63) * 8;
  if (e >= f.g.E || n0 >= N || k >= K) return;
  const Range r = group_range(f.g, e);
  float acc[4][8] = {};
  for (int64_t p = r.lo; p < r.hi; ++p) {
    const int64_t t = GATHER ? source_row(f.g, p) : p;
    if (t < 0) continue;
    float v[8];
    eight(b + t * ldb + k, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m = to_float(a[p * lda + (n0 + i < N ? n0 + i : n0)]);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(m, v[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n0 + i >= N) continue;
    const int64_t at = ((int64_t)e * N + n0 + i) * K + k;
    if (f.dw32) {
      f32x4_t* o = (f32x4_t*)((float*)dw + at);
      o[0] = f32x4_t{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
      o[1] = f32x4_t{acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
    } else {
      *(u32x4_t*)((uint16_t*)dw + at) = u32x4_t{pack_bf16x2(acc[i][0], acc[i][1]), pack_bf16x2(acc[i][2], acc[i][3]),
                                                pack_bf16x2(acc[i][4], acc[i][5]), pack_bf16x2(acc[i][6], acc[i][7])};
    }
  }
}

__global__ __launch_bounds__(FT) void k_few_products(FewArgs a) {
  __shared__ float lds[FT / 64][FC];
  int b = blockIdx.x;
  if (b < a.dx_units) {
    const int npan = (a.g.K + FC - 1) / FC, c0 = b % npan * FC, c = c0 + threadIdx.x;
    const int64_t p = b / npan;
    const int e = expert_of(a.g, p);
    if (e < 0) return;
    const float v = row_product(a.d + p * 2 * a.I, a.w_gate_up + (int64_t)e * 2 * a.I * a.g.K, 2 * a.I, a.g.K, c0, lds);
    if (threadIdx.x < FC && c < a.g.K) a.dx[p * a.ld_dx + c] = (uint16_t)f32_to_bf16(v);
    return;
  }
  b -= a.dx_units;
  if (b < a.gu_units)
    outer<float, uint16_t, true>(a, b, a.d, 2 * (int64_t)a.I, 2 * a.I, a.x, a.g.ldx, a.g.K, a.dw_gate_up);
  else
    outer<uint16_t, float, false>(a, b - a.gu_units, a.dy, a.ld_dy, a.H, a.h, a.I, a.I, a.dw_down);
}

int64_t outer_units(const FfnArgs& a, int64_t N, int64_t K) { return a.g.E * ((N + FN - 1) / FN) * ((K + FK - 1) / FK); }

}  // namespace

hipError_t launch_few_rows(const FfnArgs& f, const void* w_down, const void* pre, int64_t ldp, float* d, float* h,
                           hipStream_t s) {
  FewArgs a{};
  a.g = f.g;
  a.I = f.I;
  a.H = f.H;
  a.dy = (const uint16_t*)f.dy;
  a.x = (const uint16_t*)f.x;
  a.w_gate_up = (const uint16_t*)f.w_gate_up;
  a.w_down = (const uint16_t*)w_down;
  a.pre = (const uint16_t*)pre;
  a.ld_dy = f.ld_dy;
  a.ldp = ldp;
  a.ld_dx = f.ld_dx;
  a.d = d;
  a.h = h;
  a.dx = (uint16_t*)f.dx;
  a.dw_gate_up = f.dw_gate_up;
  a.dw_down = f.dw_down;
  a.dw32 = f.dw32;
  a.dx_units = (int)(f.g.rows * ((f.g.K + FC - 1) / FC));
  a.gu_units = (int)outer_units(f, f.g.N, f.g.K);
  const Launch lc{s, nullptr, nullptr};
  const hipError_t e = launch(lc, k_few_gate, dim3((unsigned)((f.I + FC - 1) / FC), (unsigned)f.g.rows), dim3(FT), a);
  if (e != hipSuccess) return e;
  // at most 2^28 weights: fewer than 2^20 units of either product
  const unsigned units = (unsigned)(a.dx_units + a.gu_units + outer_units(f, f.H, f.I));
  return launch(lc, k_few_products, dim3(units), dim3(FT), a);
}

}  // namespace moe
