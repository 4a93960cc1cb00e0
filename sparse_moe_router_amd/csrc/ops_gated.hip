// Gated products (gfx950, wave64, MFMA):
//   h = silu(x G^T) * (x U^T)                        G, U the two halves of an expert's weights
//   d_gate = dh u s (1 + g (1 - s)), d_up = dh g s, h = g s u     with s = sigmoid(g), dh = dy W
// over the ragged groups of rows of each expert, on the tiles of the grouped
// products (ops_tile.h).
//
// Forward: a tile is 256 rows x 128 features of both matrices; a wave holds
// the same columns of the two products in the same registers, so the
// activation needs no exchange and neither product reaches memory (unless the
// backward pass wants them: then rounded to bf16 beside h).  Backward: the
// gradient of h never leaves the registers; the tile's gate and up values are
// fetched while the accumulators go through LDS, and the two gradients and h,
// which the weight gradient of the next projection reads, leave together.
//
// Forward: 4096 tokens x 8 over 256 experts of 512 x 2048: 218 us, bound by the stream of the weights (1124
// MB in and out at 5.2 TB/s; two kernels would write and read another 134 MB).  With the products kept, 2501
// x 4 rows over 60 skewed experts of 1000 x 1416: 136 us for 407 MB; rows of 2832 bytes start off the cache
// lines, which two steps then share (rows of 2816 bytes: 112).  Backward: 8192 x 2 rows over 16 experts of
// 1024 x 2048: 111 to 131 us; 288 tiles are two rounds of 256 workgroups (matrix units busy 28% at 2.0 GHz).
#include "ops_tile.h"

namespace moe {
namespace {

constexpr int GATED_COLS = TB / 2;  // features of a tile

struct GatedEpi {
  static constexpr bool kGated = true;
  uint16_t* h;
  int64_t ldh;
  uint16_t* pre;  // or NULL
  int64_t ldp;

  template <int RB0, int RB1, class ACC>
  __device__ __forceinline__ void tile(const TileArgs& p, const TileOut& o, ACC& acc, u32x4_t* lds) const {
    const int n = p.g.N, col0 = o.c0 + 32 * o.wn;
    uint16_t* st = (uint16_t*)epi_stage(lds, o);  // 32 rows x 32 columns, of h, or of gate and up
    // 16 bytes a lane from the stage's part `from` to columns `at` of out
    auto put = [&](int row0, int from, uint16_t* out, int64_t ld, int at0) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = i * 64 + o.lane, row = c >> 2, at = (c & 3) * 8;
        if (row0 + row < o.rows && col0 + at < n)
          *(u32x4_t*)(out + (o.p0 + row0 + row) * ld + at0 + col0 + at) = *(const u32x4_t*)(st + from + row * 32 + at);
      }
    };
    each_block<RB0, RB1>(o, acc, [&](int row0, const f32x16_t& g, const f32x16_t& u) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        st[block_row(r, o.lane) * 32 + (o.lane & 31)] = (uint16_t)f32_to_bf16(silu(g[r]) * u[r]);
      wave_sync();
      put(row0, 0, h, ldh, 0);
      wave_sync();
      if (!pre) return;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int at = block_row(r, o.lane) * 32 + (o.lane & 31);
        st[at] = (uint16_t)f32_to_bf16(g[r]);
        st[1024 + at] = (uint16_t)f32_to_bf16(u[r]);
      }
      wave_sync();
      put(row0, 0, pre, ldp, 0);
      put(row0, 1024, pre, ldp, n);
      wave_sync();
    });
  }
};

struct GatedGradEpi {
  static constexpr bool kGated = false;
  const uint16_t* pre;
  int64_t ldp;
  uint16_t* d_pre;
  int64_t ldd;
  uint16_t* h;
  int64_t ldh;

  // dh of eight elements to d_gate, d_up and h, from g and u as stored
  __device__ __forceinline__ static void gate_grad(const float (&dh)[8], u32x4_t g, u32x4_t u, u32x4_t* dg, u32x4_t* du,
                                                   u32x4_t* h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a[2], b[2], v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float z = k ? bf16_hi(g[i]) : bf16_lo(g[i]), w = k ? bf16_hi(u[i]) : bf16_lo(u[i]), d = dh[2 * i + k];
        // sigmoid(z) and sigmoid(-z) from e = exp(-|z|): neither is formed as a difference
        const float e = __expf(-fabsf(z)), q = __builtin_amdgcn_rcpf(1.0f + e);
        const float s = z >= 0.0f ? q : e * q, t = z >= 0.0f ? e * q : q;
        a[k] = d * w * (s * (1.0f + z * t));
        b[k] = d * (z * s);
        v[k] = z * s * w;
      }
      (*dg)[i] = pack_bf16x2(a[0], a[1]);
      (*du)[i] = pack_bf16x2(b[0], b[1]);
      (*h)[i] = pack_bf16x2(v[0], v[1]);
    }
  }

  template <int RB0, int RB1, class ACC>
  __device__ __forceinline__ void tile(const TileArgs& p, const TileOut& o, ACC& acc, u32x4_t* lds) const {
    const int n = p.g.K;
    float* st = (float*)epi_stage(lds, o);
    each_block<RB0, RB1>(o, acc, [&](int row0, const f32x16_t& a0, const f32x16_t& a1) __attribute__((always_inline)) {
      // columns 0..31 of the stage: the wave's block of the first half, 32..63: of the second
      const int chunk = o.lane & 7, col = o.c0 + 128 * (chunk >> 2) + 32 * o.wn + (chunk & 3) * 8;
      u32x4_t g[4], u[4];
      bool in[4];
      int64_t grow[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i * 8 + (o.lane >> 3);
        grow[i] = o.p0 + row0 + row;
        in[i] = row0 + row < o.rows && col < n;
        g[i] = u[i] = u32x4_t{0, 0, 0, 0};
        if (in[i]) {
          g[i] = *(const u32x4_t*)(pre + grow[i] * ldp + col);
          u[i] = *(const u32x4_t*)(pre + grow[i] * ldp + n + col);
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        stage16(st, q, o.lane, a0, a1);
        wave_sync();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = 2 * q + k, row = k * 8 + (o.lane >> 3);
          const f32x4_t x = *staged(st, row, 2 * chunk), y = *staged(st, row, 2 * chunk + 1);
          const float dh[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
          u32x4_t dg, du, v;
          gate_grad(dh, g[i], u[i], &dg, &du, &v);
          if (!in[i]) continue;
          *(u32x4_t*)(d_pre + grow[i] * ldd + col) = dg;
          *(u32x4_t*)(d_pre + grow[i] * ldd + n + col) = du;
          *(u32x4_t*)(h + grow[i] * ldh + col) = v;
        }
        wave_sync();
      }
    });
  }
};

template <int GX>
__global__ __launch_bounds__(512, 1) void k_gated(TileArgs p, GatedEpi epi) {
  __shared__ u32x4_t lds[10 * HU];
  row_tile<OP_NT, false, GX>(p, lds, epi);
}

__global__ __launch_bounds__(512, 1) void k_gated_grad(TileArgs p, GatedGradEpi epi) {
  __shared__ u32x4_t lds[10 * HU];
  row_tile<OP_NN, false, GX_ROWS>(p, lds, epi);
}

}  // namespace

int64_t gated_units(const Groups& g) { return row_tile_units(g, (g.N + GATED_COLS - 1) / GATED_COLS); }

hipError_t launch_gated(const Groups& g, const void* x, const void* w, void* h, void* pre, int64_t ldp, hipStream_t s) {
  TileArgs t{};
  t.g = g;
  t.a = (const char*)x;
  t.b = (const char*)w;
  t.npan = (g.N + GATED_COLS - 1) / GATED_COLS;
  set_row_tiles(&t);
  const GatedEpi epi{(uint16_t*)h, g.ldy, (uint16_t*)pre, ldp};
  const dim3 gr((unsigned)gated_units(g)), bl(512);
  const Launch lc{s, nullptr, nullptr};
  return rows_far(g, 2) ? launch(lc, k_gated<GX_FAR>, gr, bl, t, epi) : launch(lc, k_gated<GX_ROWS>, gr, bl, t, epi);
}

hipError_t launch_gated_grad(const Groups& g, const void* dy, const void* w, const void* pre, int64_t ldp, void* d_pre,
                             int64_t ldd, void* h, int64_t ldh, hipStream_t s) {
  TileArgs t{};
  t.g = g;
  t.a = (const char*)dy;
  t.b = (const char*)w;
  t.npan = (g.K + TB - 1) / TB;
  set_row_tiles(&t);
  const GatedGradEpi epi{(const uint16_t*)pre, ldp, (uint16_t*)d_pre, ldd, (uint16_t*)h, ldh};
  return launch(Launch{s, nullptr, nullptr}, k_gated_grad, dim3((unsigned)op_tile_units(OP_NN, g)), dim3(512), t, epi);
}

}  // namespace moe
