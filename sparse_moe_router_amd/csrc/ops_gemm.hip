// Grouped matrix-matrix products (gfx950, wave64, MFMA, fp32 or int32
// accumulation):
//   NT  y[p][n]     = sum_k x[row(p)][k] w[e][n][k]   (bf16, or int8 codes)
//   NN  dx[p][k]    = sum_n dy[p][n] w[e][n][k]
//   TN  dw[e][n][k] = sum_p dy[p][n] x[row(p)][k]
// over the ragged groups of rows of each expert.
//
// One 8-wave workgroup computes one output tile of up to 256 x 256 over the
// whole reduction.  Operands travel straight from global memory into LDS
// rings (global->LDS transfers of 16 bytes a lane, whole cache lines), steps
// of 64 reduction elements (128 of int8) ahead of the MFMAs.  An operand
// whose reduction runs along memory (NT both, NN the rows dy) is staged as
// [256 rows][128 bytes] and read as it lies; one whose reduction runs across
// rows (NN the weights, TN both) is staged as [64 rows][512 bytes] and read
// with the transposing LDS read, so no operand is ever transposed in memory.
//
// Which rows a workgroup has comes from the group offsets on the device: each
// wave scans them itself (a few loads and a wave scan) instead of waiting for
// a map made by a launch of its own.
#include <type_traits>

#include "ops_internal.h"

namespace moe {
namespace {

constexpr int TB = kOpTile;        // tile edge
constexpr int SU = TB * 8;         // 16-byte units of one stage (32 KB)
constexpr int DA = 2, DB = 3;      // stages of the two rings

// where transfers of rows, columns or reduction steps past the end read zeros
__device__ __align__(16) const uint32_t kZero[4] = {0, 0, 0, 0};

typedef __attribute__((__vector_size__(4 * sizeof(int16_t)))) int16_t i16x4_t;

struct TileArgs {
  Groups g;
  const char* a;
  const char* b;
  Scales sc;
  void* out;
  int fp32;
  int npan;    // tiles along the second output dimension
  int nrow;    // TN: tiles along n
};

__device__ __forceinline__ void dma(const char* src, u32x4_t* dst) {
  __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));  // vmcnt(N) lgkmcnt(0)
}
__device__ __forceinline__ void bar() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The row tile and panel of workgroup (xcd, local): group, first row, rows.  A
// group of c rows has ceil(c / 256) tiles of equal height (a multiple of 32);
// the units (tile, panel), panels of a tile in a row, are cut into eight equal
// runs, one for each XCD.  Lane l scans the groups [l * per, (l + 1) * per);
// every wave does the same scan.
struct RowTile {
  int e;
  int64_t p0;
  int rows;
  int panel;
};
__device__ __forceinline__ bool find_tile(const Groups& g, int xcd, int64_t local, int npan, RowTile* out) {
  const int lane = threadIdx.x & 63;
  int e = 0;
  int64_t lo = 0, c = g.rows, i;
  int64_t mine = 0, incl = 0, total;
  const int per = (g.E + 63) / 64;
  if (!g.offsets) {
    total = (c + TB - 1) / TB;
  } else {
    for (int j = 0; j < per; ++j) {
      const int ge = lane * per + j;
      if (ge < g.E) {
        int64_t a, b;
        group_range(g, ge, &a, &b);
        mine += (b - a + TB - 1) / TB;
      }
    }
    incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    total = __shfl(incl, 63, 64);
  }
  const int64_t run = (total * npan + 7) / 8, unit = xcd * run + local;
  if (local >= run || unit >= total * npan) return false;
  const int64_t t = unit / npan;
  i = t;
  if (g.offsets) {
    const int src = __builtin_ctzll(__ballot(incl > t));
    i -= __shfl(incl - mine, src, 64);
    for (int j = 0; j < per; ++j) {
      int64_t b;
      e = src * per + j;
      group_range(g, e, &lo, &b);  // the unit exists, so a group below E holds it
      c = b - lo;
      const int64_t n = (c + TB - 1) / TB;
      if (i < n) break;
      i -= n;
    }
  }
  const int64_t nt = (c + TB - 1) / TB;
  const int64_t h = ((c + nt - 1) / nt + 31) / 32 * 32;
  const int64_t p0 = lo + i * h;
  out->e = __builtin_amdgcn_readfirstlane(e);
  out->p0 = ((int64_t)__builtin_amdgcn_readfirstlane((int)(p0 >> 32)) << 32) |
            (uint32_t)__builtin_amdgcn_readfirstlane((int)p0);
  out->rows = __builtin_amdgcn_readfirstlane((int)(c - i * h < h ? c - i * h : h));
  out->panel = __builtin_amdgcn_readfirstlane((int)(unit - t * npan));
  return true;
}

// One output tile.  Wave w = 4 rg + cg: columns [64 cg, +64) in two blocks of
// 32, rows in the 32-row blocks rb = rg, rg + 2, ... below NRB.
template <OpKind KIND, bool I8, int NRB>
__device__ __forceinline__ void tile_product(const TileArgs& p, int e, int64_t p0, int rows, int64_t len, int r0t,
                                             int panel, u32x4_t* const (&ra)[DA], u32x4_t* const (&rb_)[DB]) {
  constexpr bool AT = KIND == OP_TN, BT = KIND != OP_NT;  // operand reduces across its rows
  constexpr int NRH = (NRB + 1) / 2;
  constexpr int ES = I8 ? 1 : 2;           // bytes an element
  typedef typename std::conditional<I8, i32x16_t, f32x16_t>::type acc_t;
  const Groups& g = p.g;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cg = wave & 3, rg = wave >> 2;
  const int lr = lane >> 3;
  const char* zero = (const char*)kZero;

  // output tile: rows of `ncols`-wide out starting at (row base, c0)
  const int ncols = KIND == OP_NT ? g.N : g.K;
  const int c0 = panel * TB;
  // reduction length in elements; steps of 128 bytes (64 rows where it runs across rows)
  const int64_t red = KIND == OP_NT ? g.K : KIND == OP_NN ? g.N : len;
  constexpr int BKE = I8 ? 128 : 64;
  const int nsteps = (int)((red + BKE - 1) / BKE);

  // ---- transfers.  Along-memory operand: transfer i of the wave fills stage
  // rows 8 blk .. +8 (blk = wave * n + i), lane -> row lane/8, chunk
  // position lane%8, source chunk (lane%8) ^ ((row/2) % 8), the swizzle that
  // spreads 16 consecutive rows' reads over all banks.  Across-rows operand:
  // transfer i fills stage rows 2 blk, +1 (512 bytes each), lane -> row
  // lane/32, chunk position lane%32, source chunk pos ^ 4 (row % 4): the four
  // rows a transposing read takes together lie in different 64-byte parts.
  // A lane's transfers of steps >= lim read zeros.
  const char* asrc[4];
  int alim[4];
  int64_t astep;
  if (!AT) {
    astep = 128;
    const int64_t ld = KIND == OP_NT ? g.ldx : g.ldy;
#pragma unroll
    for (int i = 0; i < NRH; ++i) {
      const int blk = wave * NRH + i, row = blk * 8 + lr;
      const int q = (lane & 7) ^ ((row >> 1) & 7);
      int64_t src = -1;
      if (row < rows) src = KIND == OP_NT ? source_row(g, p0 + row) : p0 + row;
      const int64_t rest = red - (int64_t)q * (16 / ES);  // elements from this chunk on
      asrc[i] = p.a + (src < 0 ? 0 : src) * ld * ES + q * 16;
      alim[i] = src < 0 || rest <= 0 ? 0 : (int)((rest + BKE - 1) / BKE);
    }
  } else {
    astep = (int64_t)64 * g.ldy * 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (wave * 4 + i) * 2 + half;
      const int col = r0t * TB + (l32 ^ (4 * (row & 3))) * 8;
      asrc[i] = p.a + ((p0 + row) * g.ldy + col) * 2;
      alim[i] = col >= g.N || row >= len ? 0 : (int)((len - row + 63) / 64);
    }
  }
  const char* bsrc[4];
  int blim[4];
  int64_t bstep;
  int bcol = 0;
  if (!BT) {
    bstep = 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (wave * 4 + i) * 8 + lr;
      const int q = (lane & 7) ^ ((row >> 1) & 7);
      const int n = c0 + row;
      const int64_t rest = red - (int64_t)q * (16 / ES);
      bsrc[i] = p.b + (((int64_t)e * g.N + (n < g.N ? n : 0)) * g.K) * ES + q * 16;
      blim[i] = n >= g.N || rest <= 0 ? 0 : (int)((rest + BKE - 1) / BKE);
    }
  } else if (KIND == OP_NN) {
    bstep = (int64_t)64 * g.K * 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (wave * 4 + i) * 2 + half;
      const int col = c0 + (l32 ^ (4 * (row & 3))) * 8;
      bsrc[i] = p.b + (((int64_t)e * g.N + row) * g.K + col) * 2;
      blim[i] = col >= g.K || row >= g.N ? 0 : (g.N - row + 63) / 64;
    }
  } else {
    bstep = (int64_t)64 * g.ldx * 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (wave * 4 + i) * 2 + half;
      const int col = c0 + (l32 ^ (4 * (row & 3))) * 8;
      bcol = col;
      bsrc[i] = p.b + (g.perm ? (int64_t)col * 2 : ((p0 + row) * g.ldx + col) * 2);
      blim[i] = col >= g.K || row >= len ? 0 : (int)((len - row + 63) / 64);
    }
  }
  (void)bcol;
  auto load_a = [&](int st, int s) {
#pragma unroll
    for (int i = 0; i < (AT ? 4 : NRH); ++i)
      dma(s < alim[i] ? asrc[i] + s * astep : zero, ra[st] + (wave * (AT ? 4 : NRH) + i) * 64);
  };
  // TN with a permutation: the rows of x that the lane's transfers of step s read
  auto gather = [&](int64_t (&idx)[4], int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = (int64_t)s * 64 + (wave * 4 + i) * 2 + half;
      idx[i] = s < blim[i] ? source_row(g, p0 + r) : -1;
    }
  };
  auto load_b = [&](int st, int s, const int64_t (&idx)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const char* src = zero;
      if (KIND == OP_TN && g.perm) {
        if (idx[i] >= 0) src = bsrc[i] + idx[i] * g.ldx * 2;
      } else if (s < blim[i]) {
        src = bsrc[i] + s * bstep;
      }
      dma(src, rb_[st] + (wave * 4 + i) * 64);
    }
  };

  acc_t acc[NRH][2];
#pragma unroll
  for (int j = 0; j < NRH; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c) acc[j][c] = (acc_t){};

  // ---- operand reads: sub-step kk, lane half h take the reduction elements
  // 32 h + 8 kk .. +8 of a step (int8: 64 h + 16 kk .. +16) on both operands.
  auto read_along = [&](const u32x4_t* st, int row32, int kk) -> u32x4_t {
    return st[(row32 + l32) * 8 + ((4 * half + kk) ^ ((l32 >> 1) & 7))];
  };
  const int ti = lane & 15, tsub = (lane >> 4) & 1;
  auto read_across = [&](const u32x4_t* st, int col32, int kk) -> u32x4_t {
    // two transposing reads of 4 rows each; lane ti of 16 supplies row ti/4, columns 4 (ti%4) .. +4
    const int row = 32 * half + 8 * kk + (ti >> 2);
    const int q = (col32 / 8 + 2 * tsub + ((ti & 3) >> 1)) ^ (4 * (ti >> 2));
    const char* at = (const char*)(st + row * 32 + q) + 8 * (ti & 1);
    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)at);
    const i16x4_t hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(at + 4 * 512));
    u32x4_t r;
    const uint64_t l64 = __builtin_bit_cast(uint64_t, lo), h64 = __builtin_bit_cast(uint64_t, hi);
    r[0] = (uint32_t)l64;
    r[1] = (uint32_t)(l64 >> 32);
    r[2] = (uint32_t)h64;
    r[3] = (uint32_t)(h64 >> 32);
    return r;
  };

  if (nsteps > 0) {
    int64_t idx[2][4];
    if (KIND == OP_TN && g.perm) {
      gather(idx[0], 0);
      gather(idx[1], 1);
    }
    load_b(0, 0, idx[0]);
    load_b(1, 1, idx[1]);
    load_a(0, 0);
    if (KIND == OP_TN && g.perm) gather(idx[0], 2);
    for (int s0 = 0; s0 < nsteps; s0 += DA * DB) {
#pragma unroll
      for (int u = 0; u < DA * DB; ++u) {
        const int s = s0 + u;
        if (s >= nsteps) break;  // uniform
        // own transfers of step s done (at s = 0 all; else after them only
        // B step s + 1's four were issued), then everyone's
        if (s == 0)
          wait_vm<0>();
        else
          wait_vm<4>();
        bar();
        if (KIND == OP_TN && g.perm) gather(idx[(u + 1) & 1], s + 3);
        load_a((u + 1) % DA, s + 1);
        load_b((u + 2) % DB, s + 2, idx[u & 1]);
        const u32x4_t* sa = ra[u % DA];
        const u32x4_t* sb = rb_[u % DB];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          u32x4_t af[NRH], bf[2];
#pragma unroll
          for (int j = 0; j < NRH; ++j) {
            const int rb = 2 * j + rg;
            if (NRB == 1 && rg == 1) continue;
            af[j] = AT ? read_across(sa, 32 * rb, kk) : read_along(sa, 32 * rb, kk);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int cb = 64 * cg + 32 * c;
            bf[c] = BT ? read_across(sb, cb, kk) : read_along(sb, cb, kk);
          }
#pragma unroll
          for (int j = 0; j < NRH; ++j) {
            if (NRB == 1 && rg == 1) continue;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if constexpr (I8)
                acc[j][c] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, af[j]),
                                                                  __builtin_bit_cast(i32x4_t, bf[c]), acc[j][c], 0, 0, 0);
              else
                acc[j][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, af[j]),
                                                                    __builtin_bit_cast(bf16x8_t, bf[c]), acc[j][c], 0,
                                                                    0, 0);
            }
          }
        }
      }
    }
  }
  // transfers of steps past the end have landed and every wave has read its
  // last operands before the rings are used again
  wait_vm<0>();
  bar();

  // ---- epilogue.  Block layout: lane -> column lane%32, register r -> row
  // 8 (r/4) + 4 (lane/32) + r%4.
  const int nrows = KIND == OP_TN ? (g.N - r0t * TB < TB ? g.N - r0t * TB : TB) : rows;
  const int64_t ldo = KIND == OP_NT ? g.ldy : KIND == OP_NN ? g.ldx : g.K;
  const int64_t row_base = KIND == OP_TN ? (int64_t)e * g.N + (int64_t)r0t * TB : p0;
  const int wc0 = c0 + 64 * cg;
  float* s_scale = (float*)ra[1];  // I8: the rows' scales
  if (I8) {
    if (tid < rows) {
      const int64_t t = source_row(g, p0 + tid);
      s_scale[tid] = t < 0 ? 0.0f : p.sc.x[t];
    }
    __syncthreads();
  }
  float ws[2] = {1.0f, 1.0f}, bi[2] = {0.0f, 0.0f};
  if (I8) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = wc0 + 32 * c + l32;
      if (n < ncols) {
        ws[c] = p.sc.w[(int64_t)e * g.N + n];
        if (p.sc.bias) bi[c] = p.sc.bias[n];
      }
    }
  }
  if (wc0 >= ncols || (NRB == 1 && rg == 1)) return;
  uint16_t* stage = (uint16_t*)ra[0] + wave * (32 * 64);  // 4 KB a wave
#pragma unroll
  for (int j = 0; j < NRH; ++j) {
    const int rb = 2 * j + rg;
    if (32 * rb >= nrows) break;  // uniform
    float v[2][16];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if constexpr (I8) {
          const int row = 32 * rb + 8 * (r >> 2) + 4 * half + (r & 3);
          v[c][r] = (float)acc[j][c][r] * (s_scale[row] * ws[c]) + bi[c];
        } else {
          v[c][r] = acc[j][c][r];
        }
      }
    if (p.fp32) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * rb + 8 * (r >> 2) + 4 * half + (r & 3);
        float* orow = (float*)p.out + (row_base + row) * ldo + wc0 + l32;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (row < nrows && wc0 + 32 * c + l32 < ncols) orow[32 * c] = v[c][r];
      }
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 8 * (r >> 2) + 4 * half + (r & 3);
#pragma unroll
        for (int c = 0; c < 2; ++c) stage[row * 64 + 32 * c + l32] = (uint16_t)f32_to_bf16(v[c][r]);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int c = lane; c < 32 * 8; c += 64) {
        const int row = c >> 3, q = c & 7;
        const int grow = 32 * rb + row, col = wc0 + 8 * q;
        if (grow < nrows && col < ncols)
          *(u32x4_t*)((uint16_t*)p.out + (row_base + grow) * ldo + col) = *(const u32x4_t*)(stage + row * 64 + 8 * q);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  }
}

// Row-tiled products (NT, NN).  Workgroup b runs on XCD b % 8; a row tile's
// panels stay on one XCD, whose L2 then serves the tile's rows again.
template <OpKind KIND, bool I8>
__global__ __launch_bounds__(512, 1) void k_op_rows(TileArgs p) {
  __shared__ u32x4_t sA0[SU], sA1[SU], sB0[SU], sB1[SU], sB2[SU];  // 160 KB
  u32x4_t* const ra[DA] = {sA0, sA1};
  u32x4_t* const rb[DB] = {sB0, sB1, sB2};
  RowTile tl;
  if (!find_tile(p.g, blockIdx.x & 7, blockIdx.x >> 3, p.npan, &tl)) return;
  const int panel = tl.panel;
  const int nb = (tl.rows + 31) >> 5;
  if (nb <= 1)
    tile_product<KIND, I8, 1>(p, tl.e, tl.p0, tl.rows, 0, 0, panel, ra, rb);
  else if (nb <= 2)
    tile_product<KIND, I8, 2>(p, tl.e, tl.p0, tl.rows, 0, 0, panel, ra, rb);
  else if (nb <= 4)
    tile_product<KIND, I8, 4>(p, tl.e, tl.p0, tl.rows, 0, 0, panel, ra, rb);
  else if (nb <= 6)
    tile_product<KIND, I8, 6>(p, tl.e, tl.p0, tl.rows, 0, 0, panel, ra, rb);
  else
    tile_product<KIND, I8, 8>(p, tl.e, tl.p0, tl.rows, 0, 0, panel, ra, rb);
}

// Weight gradients (TN): a workgroup per expert and 256 x 256 tile of dw.
__global__ __launch_bounds__(512, 1) void k_op_wgrad(TileArgs p) {
  __shared__ u32x4_t sA0[SU], sA1[SU], sB0[SU], sB1[SU], sB2[SU];
  u32x4_t* const ra[DA] = {sA0, sA1};
  u32x4_t* const rb[DB] = {sB0, sB1, sB2};
  // an expert's tiles follow one another on one XCD: they share dy and x
  const int per = p.nrow * p.npan;
  const int run = (p.g.E * per + 7) / 8, unit = (int)(blockIdx.x & 7) * run + (int)(blockIdx.x >> 3);
  if (unit >= p.g.E * per) return;
  const int e = unit / per, tile = unit % per;
  int64_t lo, hi;
  group_range(p.g, e, &lo, &hi);
  tile_product<OP_TN, false, 8>(p, e, lo, 0, hi - lo, tile / p.npan, tile % p.npan, ra, rb);
}

}  // namespace

int64_t op_tile_units(OpKind kind, const Groups& g) {
  const int64_t pn = (g.N + TB - 1) / TB, pk = (g.K + TB - 1) / TB;
  const int64_t tiles = kind == OP_TN ? g.E * pn : (g.rows + TB - 1) / TB + (g.offsets ? (g.E < g.rows ? g.E : g.rows) : 0);
  return (tiles * (kind == OP_NT ? pn : pk) + 7) / 8 * 8;
}

hipError_t launch_op_tile(OpKind kind, bool i8, const Groups& g, const void* a, const void* b, const Scales& sc,
                          void* out, bool fp32, hipStream_t s) {
  TileArgs t{};
  t.g = g;
  t.a = (const char*)a;
  t.b = (const char*)b;
  t.sc = sc;
  t.out = out;
  t.fp32 = fp32;
  t.nrow = (g.N + TB - 1) / TB;
  t.npan = ((kind == OP_NT ? g.N : g.K) + TB - 1) / TB;
  const unsigned grid = (unsigned)op_tile_units(kind, g);
  const Launch lc{s, nullptr, nullptr};
  if (kind == OP_TN) return launch(lc, k_op_wgrad, dim3(grid), dim3(512), t);
  if (kind == OP_NN) return launch(lc, k_op_rows<OP_NN, false>, dim3(grid), dim3(512), t);
  if (i8) return launch(lc, k_op_rows<OP_NT, true>, dim3(grid), dim3(512), t);
  return launch(lc, k_op_rows<OP_NT, false>, dim3(grid), dim3(512), t);
}

}  // namespace moe
